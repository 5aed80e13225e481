"""GPU tests of the 4-bit cache's handle when its block table is replaced: calls go by the new table, captured steps by the
one that they were captured with."""
import numpy as np
import pytest
import torch

from tests.parity_util import bf16_dev, f32_dev
from tests.test_gpu_kv4 import _i32, _kv, _ok, _outputs, _params, _qs

pytestmark = pytest.mark.gpu


def test_replacing_the_block_table():
    import learned_block_sparse_warp_b200 as sas
    B, Hkv, d, L = 2, 2, 128, 512
    p = _params(B, 8, Hkv, d, L, 3)
    k, v = (bf16_dev(x) for x in _kv(B, Hkv, L, d, seed=1))
    cl, (q, s) = _i32([512, 300]), _qs(p, seed=2)
    qd, sd = bf16_dev(q), f32_dev(s)
    tables = [torch.from_numpy(np.random.default_rng(i).permutation(40)[:16].reshape(B, 8).astype(np.int32)).cuda() for i in (1, 2)]
    cache = sas.empty_kv4_cache(p, n_pages=40, block_table=tables[0].clone())
    cache.k.zero_(), cache.v.zero_()
    sas.sas_kv4_write(p, cache, k, v, cl, cl)
    first, captured, again = (_outputs(p) for _ in range(3))
    sas.decode_step_fused_kv4(p, qd, cache, cl, sd, first)
    graph = sas.DecodeGraph.kv4(p, qd, cache, cl, sd, 2, captured, fused=True)

    cache.block_table = tables[1].clone()
    filler = [torch.full((B, 8), -1, dtype=torch.int32, device="cuda") for _ in range(64)]  # would take a freed table's place
    cache.k.zero_(), cache.v.zero_()
    sas.sas_kv4_write(p, cache, k, v, cl, cl)
    sas.decode_step_fused_kv4(p, qd, cache, cl, sd, again)
    _ok()
    assert all(torch.equal(first[x], again[x]) for x in ("o", "lse_o", "idx"))  # the same sequences on other pages
    used = [set(t[0].tolist()) | set(t[1, :5].tolist()) for t in tables]
    assert all((cache.k[page] != 0).any().item() == (page in used[1]) for page in used[0] | used[1])

    other = sas.Kv4Cache(p, cache.k, cache.v, tables[0])
    sas.sas_kv4_write(p, other, k, v, cl, cl)
    graph.replay()
    _ok()
    assert all(torch.equal(first[x], captured[x]) for x in ("o", "lse_o", "idx"))
    del filler

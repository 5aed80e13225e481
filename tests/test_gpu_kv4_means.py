"""GPU: block means over the 4-bit cache of keys at the ends of bf16's range."""
import numpy as np
import pytest
import torch

import oracle.kv4_oracle as KV
from synth.workloads import bf16_round
from tests.parity_util import host
from tests.test_gpu_kv4 import Store, _i32, _ok, _params

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [1e-39, 1e-30, 1.0, 3e36, 1.6e38])
def test_means_at_the_ends_of_the_range(scale, d):
    """A mean of finite keys is finite. 64 products and their sums are rounded to fp32, of codes and minima apart: 2^-17 of
    the mean of s code + |m|, and 64 * 2^-150 where they are subnormal; then a rounding to bf16, or 2^-134."""
    import learned_block_sparse_warp_b200 as sas
    B, H, T = 2, 2, 320
    lens = [320, 200]
    p = _params(B, H, H, d, T)
    g = np.random.default_rng(d)
    k = bf16_round((g.uniform(-1, 1, (B, H, T, d)) * scale).astype(np.float32))
    k[:, 1] = np.abs(k[:, 1])  # a head whose values add up
    st = Store(p, True, seed=1)
    st.write(k, k, lens, lens)
    st.handle()
    km = torch.full((B, H, T // 64, d), 7.0, dtype=torch.bfloat16, device="cuda")
    sas.sas_kv4_block_mean_keys(p, st.cache, T, _i32(lens), km, _i32(lens))
    _ok()
    got = host(km).astype(np.float64)
    for b in range(B):
        for h in range(H):
            codes, step, low = KV._raw(st.rows("k", b, h), "k")
            part, m = codes * np.repeat(KV._bf16_value(step), 32, -1), np.repeat(KV._bf16_value(low), 32, -1)
            for blk in range(lens[b] // 64):
                ref, mag = (part + m)[blk].mean(0), (part + np.abs(m))[blk].mean(0)
                assert np.all(np.isfinite(got[b, h, blk])), (b, h, blk)
                tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -17 * mag + 2.0 ** -134 + 64 * 2.0 ** -150
                assert np.all(np.abs(got[b, h, blk] - ref) <= tol), (b, h, blk)
            assert np.all(got[b, h, lens[b] // 64:] == 7.0)

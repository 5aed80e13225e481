"""GPU: the codes that sas_kv4_write stores at half-way points, bit for bit, of groups whose values differ in size by up to
2^120 (x - m is no fp32 number there, and the definition is that of the exact x - m)."""
import numpy as np
import pytest
import torch

from tests.parity_util import bf16_dev
from tests.test_gpu_kv4 import Store, _i32, _ok, _params
from tests.test_kv4_codes_host import half_way_groups

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [64, 37])  # whole tiles, and parts of them
@pytest.mark.parametrize("d", [64, 128])
def test_codes_at_half_way_points(d, T):
    import learned_block_sparse_warp_b200 as sas
    p = _params(1, 2, 2, d, 128)
    st = Store(p, False, seed=1)
    k, v = (half_way_groups(seed, 2 * 64 * d // 32).reshape(1, 2, 64, d)[:, :, :T].copy() for seed in (d, d + 1))
    sas.sas_kv4_write(p, st.cache, bf16_dev(k), bf16_dev(v), _i32([64 + T if T == 64 else 41 + T]))
    _ok()
    st.write(k, v, [64 + T if T == 64 else 41 + T], [T])
    st.same()

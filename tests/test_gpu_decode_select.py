"""GPU test of the decode select (one CTA per row of up to 2048 history blocks) on rows with ties and special scores.

The order is that of the scores, with -0 equal to +0 and NaN under every number; ties go to the lower block. The picks
have to be equal. LSE(s): fp32 exponentials and at most 8 + 5 + 8 additions in fp32, 64 * 2^-24 relative to 1 + |lse|.
"""
import numpy as np
import pytest
import torch

from tests.parity_util import f32_dev, host
from tests.test_gpu_kv4 import _i32, _ok, _params, _sas, _score_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["normal", "same", "few", "special", "close", "outlier", "magnitudes"])
@pytest.mark.parametrize("NB", [1, 2, 33, 256, 257, 1000, 2047, 2048])
def test_picks_are_the_highest_scores_and_outputs_are_optional(NB, kind):
    sas = _sas()
    g = np.random.default_rng(NB + 1)
    B, H = 5, 2
    s = _score_rows(kind, (B, H, NB), g)
    lens = [64 * NB, 1, 64 * NB - 63, *(int(x) for x in g.integers(1, 64 * NB + 1, 2))]
    cl, sd = _i32(lens), f32_dev(s)
    for K in (1, 16, 255, 700, 2048):
        p = _params(B, H, H, 64, 64 * NB, K)
        want = np.full((B, H, K), -1, np.int32)
        for b, L in enumerate(lens):
            c = (L - 1) // 64
            for h in range(H):
                row = s[b, h, :c].astype(np.float64)
                order = np.lexsort((np.arange(c), -np.where(np.isnan(row), 0.0, row), np.isnan(row)))[:K]
                want[b, h, :len(order)] = np.sort(order)
        idx, lse = torch.full((B, H, K), -7, dtype=torch.int32, device="cuda"), torch.full((B, H), -7.0, device="cuda")
        sas.sas_topk_select(p, sd, idx, lse, cache_len=cl)
        alone, lse_alone = torch.full_like(idx, -7), torch.full_like(lse, -7.0)
        sas.sas_topk_select(p, sd, alone, None, cache_len=cl)
        sas.sas_gate_lse(p, sd, lse_alone, cache_len=cl)
        _ok()
        assert np.array_equal(idx.cpu().numpy(), want), (NB, K, kind)
        assert torch.equal(alone, idx)
        assert torch.equal(lse_alone.view(torch.int32), lse.view(torch.int32))
    with np.errstate(all="ignore"):
        for b, L in enumerate(lens):
            row = s[b, :, :(L - 1) // 64].astype(np.float64)
            if row.shape[1] == 0:
                assert np.all(host(lse)[b] == -np.inf)
            elif np.all(np.isfinite(row)):
                top = row.max(-1, keepdims=True)
                ref = np.log(np.exp(row - top).sum(-1)) + top[:, 0]
                assert np.all(np.abs(host(lse)[b] - ref) <= 64 * 2.0 ** -24 * (1 + np.abs(ref)))

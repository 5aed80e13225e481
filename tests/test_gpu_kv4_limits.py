"""GPU tests of the 4-bit KV cache's decode at the limits of its numbers, against the fp64 oracle.

The bounds are derived before any run, beside each test; dz, the error of a logit, is that of test_gpu_kv4.
"""
import numpy as np
import pytest
import torch

import oracle.kv4_oracle as KV
import oracle.sas_oracle as O
from synth.workloads import bf16_round
from tests.parity_util import host
from tests.test_gpu_kv4 import Store, _kv, _params, _qs, _run, _zero_past

pytestmark = pytest.mark.gpu


def _row(p, st, lens, b, h, s):
    """Of a row that attends to every block: K and V values, |s code| + |m| of both, and the V steps, by token."""
    toks = np.arange(lens[b])
    out = []
    for side in "kv":
        codes, step, low = (x.reshape(p.seq_len, -1)[toks] for x in KV._raw(st.rows(side, b, h), side))
        stp = np.repeat(KV._bf16_value(step), 32, -1)
        m = np.repeat(KV._bf16_value(low), 32, -1)
        out.append((stp * codes + m, stp * codes + np.abs(m)))
    return out


@pytest.mark.parametrize("form", ["fused", "split"])
@pytest.mark.parametrize("grow", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [30.0, 300.0, 1e4, 1e6, 1e15])
def test_very_large_logits(scale, d, grow, form):
    """Queries and keys large together, so that the logits pass 2^17, 2^27 and 2^100, over V steps that stay and that grow.

    Where the largest logit leads the next by more than 2 dz + 100, every other weight is below e^-100 and o is that
    token's V: bf16 (2^-8 of it), and four fp32 roundings and the merge's weights on s code and |m| (2^-20). Most rows
    are such: of 1000 normal logits the largest two lie about sigma / 4 apart, and dz is 2^-18 * 128 / 11 * sigma or so.
    In every row o is a mean of V values: at most the largest, and 2^-7 for P, P*s and bf16.
    """
    B, Hq, Hkv, T = 3, 24, 3, 1024
    lens = [1024, 1000, 70]
    p = _params(B, Hq, Hkv, d, T, 16)
    st = Store(p, False, seed=1, fill=0xFF)
    k, v = _kv(B, Hkv, T, d, seed=7)
    if grow:
        v = bf16_round((v * np.exp2(np.arange(T) / 51.2)[None, None, :, None]).astype(np.float32))
    st.write(bf16_round((k * np.float32(scale)).astype(np.float32)), v, lens, lens)
    st.handle()
    q, s = _qs(p, seed=8, scale=scale)
    out = _run(p, st, q, lens, s, 3, form)
    o, lse = host(out["o"]).astype(np.float64), host(out["lse_o"]).astype(np.float64)
    alone = 0
    for b in range(B):
        for h in range(Hkv):
            (kk, ka), (vv, va) = _row(p, st, lens, b, h, s)
            for hq in range(8 * h, 8 * h + 8):
                z = kk @ q[b, hq].astype(np.float64) / np.sqrt(d)
                dz = 2.0 ** -18 * (ka @ np.abs(q[b, hq]).astype(np.float64)).max() / np.sqrt(d)
                top, second = np.argsort(z)[[-1, -2]]
                ref = O.logsumexp(z)
                assert abs(lse[b, hq] - ref) <= dz + 2.0 ** -20 * (1 + abs(ref)), (b, hq)
                assert np.all(np.isfinite(o[b, hq])), (b, hq)
                assert np.all(np.abs(o[b, hq]) <= (1 + 2.0 ** -7) * va.max(0)), (b, hq)
                if z[top] - z[second] > 2 * dz + 100:
                    alone += 1
                    assert np.all(np.abs(o[b, hq] - vv[top]) <= 2.0 ** -8 * np.abs(vv[top]) + 2.0 ** -20 * va[top]), (b, hq)
    assert alone >= (0.8 if scale >= 300 else 0.3) * B * Hq

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


def _outside_bounds(p, st, lens, q, lam):
    """o of the gate outside the softmax over every block, with log-gates lam [B, Hkv, NB] and the current block's 0, and
    the bound of its error. Per token, P = p g / (largest p g) and P*s are rounded to 11 bits (1.05 * 2^-10 of p g s code
    together), P is dropped or cut below 2^-33 of the largest, and steps 2^-16 under the row's largest are not resolved
    (2^-13 of it times the sum of p g). Logits are off by dz, log-gates by 2^-20 (1 + 2 |lam|): the products
    (s - lse) * log2 e and lse are fp32. o is rounded to bf16."""
    B, G, d = p.batch, p.group, p.head_dim
    ref, tol = np.zeros((B, p.n_q_heads, d)), np.zeros((B, p.n_q_heads, d))
    for b in range(B):
        c = (lens[b] - 1) // 64
        for h in range(p.n_kv_heads):
            (kk, ka), (vv, va) = _row(p, st, lens, b, h, None)
            g = np.exp(np.append(np.repeat(lam[b, h, :c], 64), np.zeros(lens[b] - 64 * c)))
            top = max(KV._bf16_value(KV._raw(st.rows("v", b, h), "v")[1].reshape(p.seq_len, -1)[:lens[b]]).max(), 0)
            for hq in range(h * G, h * G + G):
                qv = q[b, hq].astype(np.float64)
                z = kk @ qv / np.sqrt(d)
                w = np.exp(z - O.logsumexp(z)) * g
                dz = 2.0 ** -18 * (ka @ np.abs(qv)).max() / np.sqrt(d) + 2.0 ** -20 * (1 + 2 * np.abs(lam[b, h, :c]).max())
                ref[b, hq] = w @ vv
                tol[b, hq] = (2.0 ** -8 * np.abs(ref[b, hq]) + (1.05 * 2.0 ** -10 + 2 * dz) * (w @ va)
                              + (15 * len(z) * 2.0 ** -33 * w.max() + 2.0 ** -13 * w.sum()) * top)
    return ref, tol


@pytest.mark.parametrize("form", ["fused", "split"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("gap", [5.0, 22.0, 60.0])
def test_outside_gate_with_the_mass_where_gates_are_small(gap, d, form):
    """One block has the gate, by a score `gap` above the others', and like the current one next to no attention: o is
    made of picks whose gates are e^-gap, as exact next to its own size as any other row."""
    B, Hkv, T = 2, 2, 512
    lens = [512, 300]
    p = _params(B, 8, Hkv, d, T, 8, O.GATE_SOFTMAX_OUTSIDE)
    st = Store(p, True, seed=4, fill=0xFF)
    k, v = _kv(B, Hkv, T, d, seed=9)
    for b, L in enumerate(lens):
        k[b, :, :64] -= 90 / np.sqrt(d)
        k[b, :, 64 * ((L - 1) // 64):] -= 90 / np.sqrt(d)
    st.write(bf16_round(k), v, lens, lens)
    st.handle()
    q, s = _qs(p, seed=10, scale=0.2)
    q = bf16_round(q + np.float32(1))  # the suppressed blocks' logits are about 90 lower
    s[..., 0] += np.float32(gap)
    lam = np.stack([[s[b, h].astype(np.float64) - O.logsumexp(s[b, h, :(lens[b] - 1) // 64].astype(np.float64))
                     for h in range(Hkv)] for b in range(B)])
    ref, tol = _outside_bounds(p, st, lens, q, lam)
    assert np.abs(ref).max() < 4 * np.exp(2 - gap)  # the rows are what they are meant to be
    o = host(_run(p, st, q, lens, s, 3, form)["o"]).astype(np.float64)
    worst = (np.abs(o - ref) / tol).max()
    assert worst <= 1, f"{worst:.3g} of the bound"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shift", [-30.0, 3.0, 12.0, 40.0])
def test_outside_gate_under_another_rows_lse(shift, d):
    """sas_decode_kv4 takes the LSE from its caller: one that is `shift` below the row's own makes the weights that much
    larger, up to e^40, and o with them."""
    import learned_block_sparse_warp_b200 as sas
    B, Hkv, T = 2, 2, 512
    lens = [512, 300]
    p = _params(B, 8, Hkv, d, T, 8, O.GATE_SOFTMAX_OUTSIDE)
    st = Store(p, False, seed=4, fill=0xFF)
    k, v = _kv(B, Hkv, T, d, seed=11)
    st.write(k, v, lens, lens)
    st.handle()
    q, s = _qs(p, seed=12)
    out = _run(p, st, q, lens, s, 3, "split")
    lse = out["lse_s"].double().cpu().numpy()
    out["lse_s"] -= shift
    lam = s.astype(np.float64) - host(out["lse_s"]).astype(np.float64)[..., None]
    assert np.allclose(lam.max(), (s - lse[..., None]).max() + shift, atol=0.1)
    ref, tol = _outside_bounds(p, st, lens, q, lam)
    qd, cl, sd = (torch.from_numpy(x).cuda() for x in (q, np.array(lens, np.int32), s))
    sas.sas_decode_kv4(p, qd.bfloat16(), st.cache, cl, sd, out["idx"], out["lse_s"], 3, out["o_part"], out["lse_part"])
    sas.sas_decode_combine(p, 3, out["o_part"], out["lse_part"], out["o"], out["lse_o"])
    torch.cuda.synchronize()
    assert sas.sas_get_device_error() == 0
    worst = (np.abs(host(out["o"]).astype(np.float64) - ref) / tol).max()
    assert worst <= 1, f"{worst:.3g} of the bound"


@pytest.mark.parametrize("form", ["fused", "split"])
@pytest.mark.parametrize("gate", [O.GATE_LOG_SOFTMAX, O.GATE_LOG_SIGMOID, O.GATE_LOGIT, O.GATE_SOFTMAX_OUTSIDE])
@pytest.mark.parametrize("d", [64, 128])
def test_a_masked_history_leaves_the_current_block(d, gate, form):
    """Scores that are all -inf close every gate, whatever its form: the current block alone is attended to, or with the
    gate outside the softmax only its values count. The bound is _outside_bounds' with the picks' weights at 0."""
    B, Hkv, T = 2, 2, 512
    lens = [512, 300]
    p = _params(B, 8, Hkv, d, T, 8, gate)
    st = Store(p, True, seed=4, fill=0xFF)
    k, v = _kv(B, Hkv, T, d, seed=13)
    st.write(k, v, lens, lens)
    st.handle()
    q, s = _qs(p, seed=14)
    s[:] = -np.inf
    out = _run(p, st, q, lens, s, 3, form)
    assert np.all(host(out["lse_s"]) == -np.inf)
    o, lse = host(out["o"]).astype(np.float64), host(out["lse_o"]).astype(np.float64)
    for b, L in enumerate(lens):
        cur = np.arange(L) >= 64 * ((L - 1) // 64)
        for hq in range(8):
            (kk, ka), (vv, va) = _row(p, st, lens, b, hq // 4, s)
            steps = KV._bf16_value(KV._raw(st.rows("v", b, hq // 4), "v")[1].reshape(T, -1)[:L])
            qv = q[b, hq].astype(np.float64)
            z = kk @ qv / np.sqrt(d)
            dz = 2.0 ** -18 * (ka @ np.abs(qv)).max() / np.sqrt(d)
            ref = O.logsumexp(z) if gate == O.GATE_SOFTMAX_OUTSIDE else O.logsumexp(z[cur])
            w = np.exp(z - ref) * cur
            assert abs(lse[b, hq] - ref) <= dz + 2.0 ** -20 * (1 + abs(ref))
            tol = (2.0 ** -8 * np.abs(w @ vv) + (1.05 * 2.0 ** -10 + 2 * dz) * (w @ va)
                   + (15 * L * 2.0 ** -33 * w.max() + 2.0 ** -13 * w.sum()) * steps.max())
            assert np.all(np.abs(o[b, hq] - w @ vv) <= tol), (b, hq)

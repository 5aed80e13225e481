"""GPU parity of the 4-bit KV cache: write, read, block means and decode against the fp64 oracle.

Tolerances, before any run. Records are compared bit for bit: the step is two IEEE fp32 operations and a rounding,
and the codes are those of the exact x - m.
  read   one rounding to bf16 (2^-8 of the value) after one to fp32.
  means  64 fp32 additions (64 * 2^-24 of the largest partial sum, at most the sum of |k|) and a rounding to bf16.
  decode the logits z are fp32 sums of at most 34 tensor-core accumulations, each off by 2^-23 of the largest partial
         sum, so dz = 2^-18 * scale * sum |q| (s code + |m|). lse adds exp2 and log2 errors: dz + 2^-20 (1 + |lse|).
         o: bf16 (2^-8 |o|); p and p*s in 11 bits (2 * 2^-11 sum p s code, with 5% room for second-order terms);
         p below 2^-24 and steps 2^-18 under the largest are dropped (n 2^-24 + 2^-14) max(s) 15; the logits (2 dz sum p |v|).
"""
import numpy as np
import pytest
import torch

import oracle.kv4_oracle as KV
import oracle.sas_oracle as O
from synth.workloads import bf16_round
from tests.parity_util import assert_idx_equal, bf16_dev, f32_dev, host

pytestmark = pytest.mark.gpu

GATES = [O.GATE_NONE, O.GATE_LOG_SOFTMAX, O.GATE_LOG_SIGMOID, O.GATE_LOGIT, O.GATE_SOFTMAX_OUTSIDE]
INDEX = 6  # SAS_ERR_DEVICE_INDEX


def _sas():
    import learned_block_sparse_warp_b200 as sas
    return sas


def _i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def _params(B, Hq, Hkv, d, Lmax, K=4, gate=O.GATE_NONE, **kw):
    return _sas().Params(batch=B, n_q_heads=Hq, n_kv_heads=Hkv, head_dim=d, seq_len=Lmax, top_k=K, gate_mode=gate, **kw)


def _ok():
    torch.cuda.synchronize()
    assert _sas().sas_get_device_error() == 0


class Store:
    """A cache on both sides: records on the host, by (sequence, head, block) or page, and the library's handle."""

    def __init__(self, p, paged, seed, fill=0xA5):
        g = np.random.default_rng(seed)
        self.p, B, H, NB = p, p.batch, p.n_kv_heads, p.n_blocks
        self.table = g.permutation(B * NB + 3)[: B * NB].reshape(B, NB).astype(np.int32) if paged else None
        shape = (B * NB + 3, H, 40 * p.head_dim) if paged else (B, H, NB, 40 * p.head_dim)
        self.rec = {s: np.full(shape, fill, np.uint8) for s in "kv"}
        self.handle()

    def handle(self):
        t = None if self.table is None else torch.from_numpy(self.table).cuda()
        self.dev = {s: torch.from_numpy(self.rec[s]).cuda() for s in "kv"}
        self.cache = _sas().Kv4Cache(self.p, self.dev["k"], self.dev["v"], t)

    def rows(self, side, b, h):
        """Records [NB, 40 d] of one sequence's head (a copy)."""
        r = self.rec[side]
        return r[b, h].copy() if self.table is None else r[self.table[b], h].copy()

    def put(self, side, b, h, rows):
        if self.table is None:
            self.rec[side][b, h] = rows
        else:
            self.rec[side][self.table[b], h] = rows

    def write(self, k, v, lens, new):
        """The oracle's sas_kv4_write."""
        for side, x in (("k", k), ("v", v)):
            for b in range(self.p.batch):
                for h in range(self.p.n_kv_heads if new[b] else 0):
                    rows = self.rows(side, b, h)
                    KV.pack_into(rows, side, *KV.quantise(x[b, h, :new[b]]), lens[b] - new[b])
                    self.put(side, b, h, rows)

    def dense(self, side):
        """Values [B, Hkv, Lmax, d] in fp64."""
        with np.errstate(all="ignore"):
            return np.stack([np.stack([KV.unpack(self.rows(side, b, h), side).reshape(self.p.seq_len, -1)
                                       for h in range(self.p.n_kv_heads)]) for b in range(self.p.batch)])

    def same(self):
        for s in "kv":
            got = self.dev[s].cpu().numpy()
            bad = np.argwhere(got != self.rec[s])
            assert bad.size == 0, f"{s}: {len(bad)} bytes differ, first at {bad[0].tolist()}"


def _kv(B, H, T, d, seed, scale=1.0):
    g = np.random.default_rng(seed)
    loud = np.where(np.arange(d) % 21 == 5, 4.0, 1.0)
    k = g.standard_normal((B, H, T, d)) * loud + 0.5 * g.standard_normal((1, H, 1, d))
    return bf16_round((k * scale).astype(np.float32)), bf16_round((g.standard_normal((B, H, T, d)) * scale).astype(np.float32))


# ---------------------------------------------------------------------------------------------------------------
# write and read
# ---------------------------------------------------------------------------------------------------------------
SHAPES = [  # B, Hkv, d, Lmax, T, cache_len, new_len
    (1, 1, 64, 64, 1, [1], None),
    (3, 2, 128, 256, 1, [256, 17, 64], None),
    (2, 3, 128, 512, 512, [512, 512], None),
    (3, 2, 64, 320, 77, [77, 320, 141], [77, 1, 30]),
    (4, 1, 128, 256, 130, [131, 0, 200, 255], [130, 0, 67, 2]),
    (2, 8, 64, 1024, 1000, [1001, 1000], [1000, 333]),
]


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("B,H,d,Lmax,T,lens,new", SHAPES)
def test_write_is_bit_exact_and_read_returns_it(B, H, d, Lmax, T, lens, new, paged):
    sas = _sas()
    p = _params(B, H, H, d, Lmax)
    st = Store(p, paged, seed=T + d)
    k, v = _kv(B, H, T, d, seed=T)
    kd, vd = bf16_dev(k), bf16_dev(v)
    n = [T] * B if new is None else new
    sas.sas_kv4_write(p, st.cache, kd, vd, _i32(lens), None if new is None else _i32(new))
    _ok()
    st.write(k, v, lens, n)
    st.same()  # and every byte of other tokens is as it was
    ko, vo = torch.full_like(kd, 7.0), torch.full_like(vd, 7.0)
    sas.sas_kv4_read(p, st.cache, ko, vo, _i32(lens), None if new is None else _i32(new))
    _ok()
    for side, got, x in (("k", host(ko), k), ("v", host(vo), v)):
        ref = KV.values(*KV.quantise(x))
        for b in range(B):
            err = np.abs(got[b, :, :n[b]] - ref[b, :, :n[b]])
            assert np.all(err <= (2.0 ** -8 + 2.0 ** -23) * np.abs(ref[b, :, :n[b]]) + 2.0 ** -133)
            assert np.all(got[b, :, n[b]:] == 7.0)  # rows behind a sequence's tokens stay
    one = torch.full_like(kd, 7.0)
    sas.sas_kv4_read(p, st.cache, None, one, _i32(lens), None if new is None else _i32(new))
    assert torch.equal(one, vo)
    one.fill_(7.0)
    sas.sas_kv4_read(p, st.cache, one, None, _i32(lens), None if new is None else _i32(new))
    assert torch.equal(one, ko)


@pytest.mark.parametrize("d", [64, 128])
def test_token_by_token_equals_one_write(d):
    sas = _sas()
    p = _params(2, 2, 2, d, 128)
    k, v = _kv(2, 2, 83, d, seed=5)
    a, b = Store(p, True, seed=1), Store(p, True, seed=1)
    sas.sas_kv4_write(p, a.cache, bf16_dev(k), bf16_dev(v), _i32([83, 83]))
    for i in range(83):
        sas.sas_kv4_write(p, b.cache, bf16_dev(k[:, :, i:i + 1]), bf16_dev(v[:, :, i:i + 1]), _i32([i + 1, i + 1]))
    _ok()
    assert torch.equal(a.dev["k"], b.dev["k"]) and torch.equal(a.dev["v"], b.dev["v"])


@pytest.mark.parametrize("scale", [1e-41, 1e-36, 1e-20, 1e20, 1e38])
def test_write_over_the_range_of_bf16(scale):
    """From steps below 2^-126, which are stored as 0, to ranges above the largest float, which read as NaN."""
    sas = _sas()
    p = _params(1, 2, 2, 128, 64)
    g = np.random.default_rng(3)
    x = bf16_round((g.uniform(-2.5, 2.5, (1, 2, 64, 128)) * scale).astype(np.float32))
    st = Store(p, False, seed=2)
    sas.sas_kv4_write(p, st.cache, bf16_dev(x), bf16_dev(x), _i32([64]))
    _ok()
    st.write(x, x, [64], [64])
    st.same()


def test_groups_with_nan_infinity_ties_and_constants():
    sas = _sas()
    p = _params(1, 1, 1, 64, 64)
    x = np.zeros((1, 1, 64, 64), np.float32)
    g = np.random.default_rng(8)
    x[0, 0, :, :32] = bf16_round(g.integers(-16, 17, (64, 32)).astype(np.float32) * 0.5)  # many half-way values
    x[0, 0, :, 0], x[0, 0, :, 1] = -8.0, 7.0
    x[0, 0, 0, 40], x[0, 0, 1, 41], x[0, 0, 2, 42], x[0, 0, 3, 32:] = np.nan, np.inf, -np.inf, -2.5
    x[0, 0, 4, 50], x[0, 0, 5, 3] = -0.0, np.nan
    st = Store(p, False, seed=2)
    xd = bf16_dev(x)
    sas.sas_kv4_write(p, st.cache, xd, xd, _i32([64]))
    out = torch.empty_like(xd)
    sas.sas_kv4_read(p, st.cache, out, None, _i32([64]))
    _ok()
    ref = KV.values(*KV.quantise(x))
    got = host(out)
    assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.isnan(got).sum() == 4 * 32
    # rows that hold an 8.0 have the step bf16(16/15), whose levels are no bf16: reading is one rounding, at most
    # 2^-8 of the value. The records themselves are compared bit for bit.
    ok = ~np.isnan(ref)
    assert np.all(np.abs(got[ok] - ref[ok]) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(ref[ok]))
    st.write(x, x, [64], [64])
    st.same()


def test_bad_lengths_and_pages_leave_the_cache_alone():
    sas = _sas()
    B, T, Lmax = 6, 4, 128
    p = _params(B, 1, 1, 64, Lmax)
    st = Store(p, True, seed=4)
    k, v = _kv(B, 1, T, 64, seed=1)
    st.table[0, 1] = 1000  # a page past the pool
    st.table[5, 0] = -1
    st.handle()
    lens, new = [66, 129, 3, 10, 10, 4], [4, 4, 4, 5, -1, 4]  # 0: half of it in the bad page; 1..4: broken lengths
    out = torch.full((B, 1, T, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: sas.sas_kv4_write(p, st.cache, bf16_dev(k), bf16_dev(v), _i32(lens), _i32(new)),
                 lambda: sas.sas_kv4_read(p, st.cache, out, None, _i32(lens), _i32(new))):
        call()
        torch.cuda.synchronize()
        assert sas.sas_get_device_error() == INDEX
    rows = st.rec["k"][st.table[0, :1], 0]
    for side, x in (("k", k), ("v", v)):
        rows = st.rec[side][st.table[0, :1], 0]
        KV.pack_into(rows, side, *KV.quantise(x[0, 0, :2]), 62)
        st.rec[side][st.table[0, :1], 0] = rows
    st.same()
    got = host(out)
    assert np.all(got[0, 0, 2:] == 7.0) and np.all(got[1:] == 7.0) and np.all(got[0, 0, :2] != 7.0)


# ---------------------------------------------------------------------------------------------------------------
# block means
# ---------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("B,H,d,Lmax,T,lens,new", [
    (1, 2, 128, 512, 512, [512], None),
    (4, 3, 64, 256, 1, [64, 65, 256, 1], None),
    (5, 1, 128, 640, 200, [200, 640, 63, 128, 77], [200, 129, 63, 0, 65]),
])
def test_block_means(B, H, d, Lmax, T, lens, new, paged):
    sas = _sas()
    p = _params(B, H, H, d, Lmax)
    st = Store(p, paged, seed=T)
    k, v = _kv(B, H, Lmax, d, seed=9)
    st.write(k, v, lens, lens)
    st.handle()
    km = torch.full((B, H, Lmax // 64, d), 7.0, dtype=torch.bfloat16, device="cuda")
    sas.sas_kv4_block_mean_keys(p, st.cache, T, _i32(lens), km, None if new is None else _i32(new))
    _ok()
    got, vals = host(km), st.dense("k")
    for b in range(B):
        n = T if new is None else new[b]
        for m in range(Lmax // 64):
            if lens[b] - n < 64 * (m + 1) <= lens[b]:
                x = vals[b, :, 64 * m: 64 * m + 64]
                ref, mag = x.mean(1), np.abs(x).mean(1)
                assert np.all(np.abs(got[b, :, m] - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -17 * mag)
            else:
                assert np.all(got[b, :, m] == 7.0)


# ---------------------------------------------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------------------------------------------
def _filled(p, paged, seed, lens, scale=1.0):
    """A cache with lens tokens; 0xFF (NaN steps and minima) in every byte that no token has written."""
    st = Store(p, paged, seed, fill=0xFF)
    k, v = _kv(p.batch, p.n_kv_heads, p.seq_len, p.head_dim, seed, scale)
    st.write(k, v, lens, lens)
    st.handle()
    return st


def _qs(p, seed, scale=1.0):
    g = np.random.default_rng(seed + 100)
    q = bf16_round((g.standard_normal((p.batch, p.n_q_heads, p.head_dim)) * scale).astype(np.float32))
    s = (g.standard_normal((p.batch, p.n_kv_heads, p.n_blocks)) * np.sqrt(2)).astype(np.float32)
    return q, s


def _zero_past(x, lens):
    x = x.copy()
    for b, L in enumerate(lens):
        x[b, :, L:] = 0.0
    return x


def _reference(p, st, q, lens, s):
    """The oracle's step on the cache's values, and the bounds of o and lse (see the top of the file)."""
    kd, vd = _zero_past(st.dense("k"), lens), _zero_past(st.dense("v"), lens)
    cl = np.array(lens, np.int32)
    ref = O.decode(q, kd, vd, cl, s.astype(np.float64), p.top_k, gate_mode=p.gate_mode, n_split=1)
    B, Hq, d, G = p.batch, p.n_q_heads, p.head_dim, p.group
    scale = 1.0 / np.sqrt(d)
    tol_o, tol_l = np.zeros((B, Hq, d)), np.zeros((B, Hq))
    for b in range(B):
        L, c = lens[b], (lens[b] - 1) // 64
        for h in range(p.n_kv_heads):
            sel = [int(m) for m in ref["idx"][b, h] if m >= 0]
            toks = np.concatenate([np.arange(64 * m, 64 * m + 64) for m in sel] + [np.arange(64 * c, L)])
            lam = np.zeros(len(toks))
            if sel:
                lam[: 64 * len(sel)] = np.repeat(O.log_gate(s[b, h, :c].astype(np.float64), sel, p.gate_mode), 64)
            bias, w = O._gate_placement(lam, p.gate_mode)
            parts = {}
            for side in "kv":
                codes, step, low = KV._raw(st.rows(side, b, h), side)
                codes, step, low = (x.reshape(p.seq_len, -1)[toks] for x in (codes, step, low))
                stp = np.repeat(KV._bf16_value(step), 32, -1)
                parts[side] = stp * codes, np.abs(np.repeat(KV._bf16_value(low), 32, -1)), stp
            for g in range(G):
                hq = h * G + g
                z = scale * (kd[b, h, toks] @ q[b, hq]) + bias
                lse = O.logsumexp(z)
                pr = np.exp(z - lse) * w
                dz = 2.0 ** -18 * (scale * ((parts["k"][0] + parts["k"][1]) @ np.abs(q[b, hq])).max() + np.abs(bias).max())
                top = parts["v"][2].max()
                tol_l[b, hq] = dz + 2.0 ** -20 * (1 + abs(lse))
                tol_o[b, hq] = (2.0 ** -8 * np.abs(ref["o"][b, hq]) + 1.05 * 2.0 ** -10 * (pr @ parts["v"][0])
                                + (len(toks) * 2.0 ** -24 + 2.0 ** -14) * 15 * top
                                + 2 * dz * (pr @ (parts["v"][0] + parts["v"][1])))
    return ref, tol_o, tol_l


def _outputs(p, n_split=None):
    sas = _sas()
    return sas.empty_decode_outputs(p, n_split or 1)


def _check(out, ref, tol_o, tol_l, lse_s=True):
    assert_idx_equal(out["idx"].cpu().numpy(), ref["idx"])
    if lse_s:
        got = host(out["lse_s"])
        fin = np.isfinite(ref["lse_s"])
        assert np.array_equal(np.isfinite(got), fin) and np.all(np.abs(got[fin] - ref["lse_s"][fin]) < 1e-4)
    o, lse = host(out["o"]), host(out["lse_o"])
    worst = np.abs(lse - ref["lse"]) / tol_l
    assert np.all(worst <= 1), f"lse_o: {worst.max():.3g} of its bound"
    worst = np.abs(o - ref["o"]) / tol_o
    assert np.all(worst <= 1), f"o: {worst.max():.3g} of its bound"


def _run(p, st, q, lens, s, n_split, form):
    sas = _sas()
    out = _outputs(p, n_split)
    if form == "fused":
        sas.decode_step_fused_kv4(p, bf16_dev(q), st.cache, _i32(lens), f32_dev(s), out)
    else:
        sas.decode_step_kv4(p, bf16_dev(q), st.cache, _i32(lens), f32_dev(s), n_split, out)
    _ok()
    return out


DECODE = [  # B, Hq, Hkv, d, Lmax, K, n_split, lens
    (4, 32, 8, 128, 2048, 16, 17, [2048, 1, 1000, 1999]),
    (3, 8, 8, 64, 1024, 4, 2, [64, 65, 1024]),
    (2, 10, 2, 128, 4096, 8, 3, [4096, 4033]),
    (2, 16, 2, 128, 1024, 32, 33, [1024, 130]),   # K above the history: every block, G = 8
    (1, 4, 1, 64, 512, 2, 1, [300]),
    (2, 6, 2, 128, 8192, 64, 5, [8192, 5000]),    # G = 3
    (40, 8, 8, 64, 512, 4, 1, None),
    (1, 7, 1, 128, 64, 1, 2, [17]),               # one block: no history
]


@pytest.mark.parametrize("form", ["fused", "split"])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("B,Hq,Hkv,d,Lmax,K,n_split,lens", DECODE)
def test_decode_parity(B, Hq, Hkv, d, Lmax, K, n_split, lens, paged, form):
    lens = lens or list(np.random.default_rng(B).integers(1, Lmax + 1, B))
    p = _params(B, Hq, Hkv, d, Lmax, K)
    st = _filled(p, paged, seed=K + d, lens=lens)
    q, s = _qs(p, seed=K)
    _check(_run(p, st, q, lens, s, n_split, form), *_reference(p, st, q, lens, s))


@pytest.mark.parametrize("form", ["fused", "split"])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("d", [64, 128])
def test_decode_gates(d, gate, form):
    p = _params(3, 12, 3, d, 1024, 5, gate)
    lens = [1024, 333, 20]
    st = _filled(p, True, seed=d + gate, lens=lens)
    q, s = _qs(p, seed=gate)
    _check(_run(p, st, q, lens, s, 3, form), *_reference(p, st, q, lens, s))


@pytest.mark.parametrize("form", ["fused", "split"])
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 33, 48, 63, 64, 65, 127, 129])
def test_decode_every_tail(L, form):
    """Current blocks that end inside a tile, at its edge and after one token."""
    p = _params(2, 8, 2, 128, 192, 2)
    lens = [L, 192 - L]
    st = _filled(p, True, seed=L, lens=lens)
    q, s = _qs(p, seed=L)
    _check(_run(p, st, q, lens, s, 2, form), *_reference(p, st, q, lens, s))


@pytest.mark.parametrize("form", ["fused", "split"])
@pytest.mark.parametrize("scale", [1e-25, 1e-8, 1e-4, 300.0, 1e8, 1e25])
def test_decode_over_a_wide_range_of_values(scale, form):
    """K, V far from 1, the queries scaled the other way."""
    p = _params(2, 8, 2, 128, 512, 3)
    lens = [512, 200]
    st = _filled(p, False, seed=11, lens=lens, scale=scale)
    q, s = _qs(p, seed=12, scale=1.0 / scale)
    _check(_run(p, st, q, lens, s, 2, form), *_reference(p, st, q, lens, s))


@pytest.mark.parametrize("form", ["fused", "split"])
def test_decode_growing_values_and_sharp_softmax(form):
    """V steps that grow by 2^20 along the cache (the running scale has to follow), and logits far apart."""
    p = _params(1, 8, 1, 128, 1024, 15)
    st = Store(p, False, seed=1, fill=0xFF)
    k, v = _kv(1, 1, 1024, 128, seed=2, scale=3.0)
    v = bf16_round((v * np.exp2(np.arange(1024) / 51.2)[None, None, :, None]).astype(np.float32))
    st.write(k, v, [1024], [1024])
    st.handle()
    q, s = _qs(p, seed=3, scale=4.0)
    _check(_run(p, st, q, [1024], s, 4, form), *_reference(p, st, q, [1024], s))


@pytest.mark.parametrize("form", ["fused", "split"])
def test_decode_nan_stays_in_its_channels(form):
    """A NaN in V reaches the outputs of its 32 channels of the KV head's queries alone; one in K the whole row."""
    p = _params(1, 8, 2, 128, 256, 8)
    st = Store(p, False, seed=1, fill=0xFF)
    k, v = _kv(1, 2, 256, 128, seed=2)
    v[0, 0, 70, 33] = np.nan
    st.write(k, v, [256], [256])
    st.handle()
    q, s = _qs(p, seed=3)
    out = _run(p, st, q, [256], s, 2, form)
    nan = np.isnan(host(out["o"]))
    assert nan[0, :4, 32:64].all() and nan.sum() == 4 * 32
    assert np.isfinite(host(out["lse_o"])).all()
    k[0, 1, 9, 1] = np.inf
    st.write(k, v, [256], [256])
    st.handle()
    out = _run(p, st, q, [256], s, 2, form)
    assert np.isnan(host(out["o"])[0, 4:]).all() and np.isnan(host(out["lse_o"])[0, 4:]).all()
    assert np.isfinite(host(out["lse_o"])[0, :4]).all()


def test_decode_ties_take_the_lowest_blocks():
    p = _params(4, 16, 4, 64, 4096, 16, O.GATE_LOG_SOFTMAX)
    lens = [4096, 4000, 1500, 700]
    st = _filled(p, True, seed=1, lens=lens)
    q, _ = _qs(p, seed=1)
    s = np.random.default_rng(4).choice(np.array([-1.0, 0.5, 2.0], np.float32), size=(4, 4, 64))
    ref = _reference(p, st, q, lens, s)
    for form in ("fused", "split"):
        _check(_run(p, st, q, lens, s, 4, form), *ref)


def test_split_partials_match_the_oracle():
    """The partials themselves, empty splits among them, on the contract of sas_decode."""
    sas = _sas()
    p = _params(3, 8, 2, 128, 1024, 12)
    lens = [1024, 70, 400]
    st = _filled(p, True, seed=6, lens=lens)
    q, s = _qs(p, seed=6)
    out = _run(p, st, q, lens, s, 5, "split")
    _, tol_o, tol_l = _reference(p, st, q, lens, s)
    kd, vd = _zero_past(st.dense("k"), lens), _zero_past(st.dense("v"), lens)
    ref = O.decode(q, kd, vd, np.array(lens, np.int32), s.astype(np.float64), 12, n_split=5)
    lp, fin = host(out["lse_part"]), np.isfinite(ref["lse_part"])
    assert np.array_equal(np.isfinite(lp), fin) and np.all(lp[~fin] == -np.inf)
    assert np.all(np.abs(lp - np.where(fin, ref["lse_part"], 0))[fin] <= 2.0 ** -12)
    got = host(out["o_part"])
    assert np.all(got[~fin] == 0) and np.abs(got - ref["o_part"]).max() < 2.0 ** -7
    again = _outputs(p, 5)
    sas.decode_step_kv4(p, bf16_dev(q), st.cache, _i32(lens), f32_dev(s), 5, again)
    assert all(torch.equal(again[k], out[k]) for k in out)  # no atomics: the same bits


def test_many_blocks_per_split_and_full_scope():
    p = _params(1, 2, 1, 64, 64 * 300, 2048)
    lens = [64 * 300 - 5]
    st = _filled(p, False, seed=6, lens=lens)
    q, s = _qs(p, seed=6)
    _check(_run(p, st, q, lens, s, 40, "split"), *_reference(p, st, q, lens, s))


@pytest.mark.parametrize("d", [64, 128])
def test_outputs_that_are_small_next_to_their_terms(d):
    """Attention over a whole cache of 65536 tokens: o is a mean of many values, 200 times smaller than sum p s code
    and sum p |m| that it is made of, and keeps what rounding P and P*s leaves of it.

    Bound of the root mean square of o's error over the channels, before any run. Two roundings to 11 bits, each off by
    2^-11/sqrt(3) of p s code at most, in root mean square, and of one token independent of another's:
    sqrt(2/3) 2^-11 sqrt(sum (p s code)^2). The sums of a warp's 64 tiles, each cut off by half of 2^-23 of a partial
    sum, on average half the last one: 64 * 2^-25 sum p s code. The minima, the merges, sum p and the logits, in fp32 and
    rounded to nearest: 2^-22 of the sums, and 2^-20 (a weight's relative error) of a term each.
    """
    T = 65536
    p = _params(1, 36, 18, d, T, T // 64)  # 18 KV heads: CTAs enough without clusters, 16 blocks a warp
    g = np.random.default_rng(d)
    st = Store(p, False, seed=1, fill=0)
    n = (T // 64, 64)
    for side in "kv":
        step = KV._bf16_bits((0.18 + 0.2 * g.random((*n, d // 32))).astype(np.float32))
        low = KV._bf16_bits((-KV._bf16_value(step) * (7.5 + 1.5 * g.standard_normal(step.shape))).astype(np.float32))
        st.put(side, 0, 0, KV.pack(g.integers(0, 16, (*n, d)).astype(np.uint8), step, low, side))
    st.handle()
    q, s = _qs(p, seed=d)
    out = _run(p, st, q, [T], s, 17, "split")
    codes, step, low = (x.reshape(T, -1) for x in KV._raw(st.rows("v", 0, 0), "v"))
    term = codes * np.repeat(KV._bf16_value(step), 32, -1)
    v = term + np.repeat(KV._bf16_value(low), 32, -1)
    k = KV.unpack(st.rows("k", 0, 0), "k").reshape(T, d)
    lp, op = host(out["lse_part"])[0], host(out["o_part"])[0]  # the fp32 partials: o itself is rounded to bf16
    for h in range(2):
        z = k @ q[0, h].astype(np.float64) / np.sqrt(d)
        pr = np.exp(z - O.logsumexp(z))
        w = np.exp(lp[h].astype(np.float64) - O.logsumexp(lp[h].astype(np.float64)))
        err = (w[:, None] * op[h]).sum(0) - pr @ v
        rms = lambda x: np.sqrt(np.mean(x ** 2))
        sums = rms(pr @ term) + rms(pr @ (v - term))
        squares = np.sqrt(np.mean(pr ** 2 @ term ** 2))
        bound = np.sqrt(2 / 3) * 2.0 ** -11 * squares + (64 * 2.0 ** -25 + 2.0 ** -22) * sums + 2.0 ** -20 * squares
        print(f"head {h}: error {rms(err):.3g}, bound {bound:.3g}, o {rms(pr @ v):.3g}")
        assert rms(err) <= bound


@pytest.mark.parametrize("form", ["fused", "split"])
def test_bad_lengths_indices_and_pages_are_reported(form):
    sas = _sas()
    p = _params(2, 4, 1, 64, 256, 2)
    st = _filled(p, True, seed=6, lens=[256, 256])
    q, s = _qs(p, seed=6)
    good = _run(p, st, q, [256, 256], s, 1, form)
    out = _outputs(p, 1)
    step = ((lambda L: sas.decode_step_fused_kv4(p, bf16_dev(q), st.cache, _i32(L), f32_dev(s), out)) if form == "fused"
            else (lambda L: sas.decode_step_kv4(p, bf16_dev(q), st.cache, _i32(L), f32_dev(s), 1, out)))
    step([256, 5000])  # clamped to 256
    torch.cuda.synchronize()
    assert sas.sas_get_device_error() == INDEX
    if form == "split":  # sas_topk_select gives such a row no picks: the current block alone is left
        good["idx"][1] = -1
        sas.sas_decode_kv4(p, bf16_dev(q), st.cache, _i32([256, 256]), None, good["idx"], None, 1, good["o_part"], good["lse_part"])
        sas.sas_decode_combine(p, 1, good["o_part"], good["lse_part"], good["o"], good["lse_o"])
        _ok()
    assert all(torch.equal(out[k], good[k]) for k in ("o", "idx"))
    st.table[1, 3] = 10 ** 6  # the current block of sequence 1 is left out
    st.handle()
    step([256, 256])
    torch.cuda.synchronize()
    assert sas.sas_get_device_error() == INDEX and sas.sas_get_device_error() == 0
    assert torch.equal(out["o"][0], good["o"][0]) and torch.isfinite(out["o"]).all()
    st.table[1] = -1  # nothing is left of sequence 1
    st.handle()
    step([256, 256])
    torch.cuda.synchronize()
    assert sas.sas_get_device_error() == INDEX
    assert torch.all(out["o"][1] == 0) and torch.all(out["lse_o"][1] == -np.inf)
    assert torch.equal(out["o"][0], good["o"][0])


def test_split_leaves_out_a_pick_past_the_history():
    sas = _sas()
    p = _params(1, 4, 1, 128, 512, 3)
    st = _filled(p, False, seed=6, lens=[400])
    q, s = _qs(p, seed=6)
    out = _outputs(p, 2)
    got = []
    for idx in ([1, 3, 7], [1, 3, -1]):
        out["idx"].copy_(_i32(idx).view(1, 1, 3))
        sas.sas_decode_kv4(p, bf16_dev(q), st.cache, _i32([400]), None, out["idx"], None, 2, out["o_part"], out["lse_part"])
        torch.cuda.synchronize()
        assert sas.sas_get_device_error() == (INDEX if idx[2] == 7 else 0)
        got.append((out["o_part"].clone(), out["lse_part"].clone()))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


# ---------------------------------------------------------------------------------------------------------------
# as they are used
# ---------------------------------------------------------------------------------------------------------------
def test_records_past_four_gigabytes():
    """Pages whose byte offsets pass 32 bits: written, read, summarised and attended to."""
    sas = _sas()
    n_pages = 110000  # 8 heads x 5120 B: 4.5 GB each of K and V
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    p = _params(1, 8, 8, 128, 192, 2)
    table = _i32([n_pages - 1, 54000, n_pages - 2]).view(1, 3)
    cache = sas.empty_kv4_cache(p, n_pages=n_pages, block_table=table)
    small = Store(p, False, seed=1)
    k, v = _kv(1, 8, 192, 128, seed=1)
    q, s = _qs(p, seed=1)
    outs = []
    for c in (cache, small.cache):
        ko, vo = (torch.empty((1, 8, 192, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        km = torch.empty((1, 8, 3, 128), dtype=torch.bfloat16, device="cuda")
        out, split = _outputs(p, 1), _outputs(p, 1)
        sas.sas_kv4_write(p, c, bf16_dev(k), bf16_dev(v), _i32([192]))
        sas.sas_kv4_read(p, c, ko, vo, _i32([192]))
        sas.sas_kv4_block_mean_keys(p, c, 192, _i32([192]), km)
        sas.decode_step_fused_kv4(p, bf16_dev(q), c, _i32([192]), f32_dev(s), out)
        sas.decode_step_kv4(p, bf16_dev(q), c, _i32([192]), f32_dev(s), 1, split)
        _ok()
        outs.append([ko, vo, km, out["o"], out["lse_o"], split["o"], split["lse_o"]])
    assert all(torch.equal(a, b) for a, b in zip(*outs))


@pytest.mark.parametrize("paged", [False, True])
def test_serving_loop(paged):
    """Prompts in two chunks, means, then steps that write a token, score, select, attend: the path end to end."""
    sas = _sas()
    B, Hq, Hkv, d, Lmax, K = 2, 8, 2, 128, 512, 3
    p = _params(B, Hq, Hkv, d, Lmax, K)
    st = Store(p, paged, seed=3, fill=0xFF)
    lens = [250, 61]
    k, v = _kv(B, Hkv, Lmax, d, seed=4)
    km = torch.zeros((B, Hkv, Lmax // 64, d), dtype=torch.bfloat16, device="cuda")
    km_ref = np.zeros((B, Hkv, Lmax // 64, d))
    at = [0, 0]
    for new in ([150, 61], [100, 0]):
        at = [a + n for a, n in zip(at, new)]
        T = max(new)
        ck, cv = np.zeros((B, Hkv, T, d), np.float32), np.zeros((B, Hkv, T, d), np.float32)
        for b in range(B):
            ck[b, :, :new[b]], cv[b, :, :new[b]] = k[b, :, at[b] - new[b]:at[b]], v[b, :, at[b] - new[b]:at[b]]
        sas.sas_kv4_write(p, st.cache, bf16_dev(ck), bf16_dev(cv), _i32(at), _i32(new))
        sas.sas_kv4_block_mean_keys(p, st.cache, T, _i32(at), km, _i32(new))
        st.write(ck, cv, at, new)
    out = _outputs(p, 2)
    sd = torch.zeros((B, Hkv, Lmax // 64), dtype=torch.float32, device="cuda")
    for step in range(8):
        lens = [L + 1 for L in lens]
        tk = np.stack([k[b, :, lens[b] - 1:lens[b]] for b in range(B)])
        tv = np.stack([v[b, :, lens[b] - 1:lens[b]] for b in range(B)])
        q, _ = _qs(p, seed=step)
        sas.decode_step_scored_kv4(p, bf16_dev(q), bf16_dev(tk), bf16_dev(tv), st.cache, km, _i32(lens), sd, 2, out)
        _ok()
        st.write(tk, tv, lens, [1] * B)
        st.same()
        dense = st.dense("k")
        for b in range(B):
            for m in range(lens[b] // 64):
                km_ref[b, :, m] = dense[b, :, 64 * m:64 * m + 64].mean(1)
        got_km = host(km)
        assert np.all(np.abs(got_km - km_ref) <= 2.0 ** -8 * np.abs(km_ref) + 2.0 ** -15)
        s_got = host(sd).astype(np.float32)
        s_ref = O.decode_scores(q, got_km, lens)
        live = np.isfinite(s_ref)
        assert np.all(np.abs(s_got - np.where(live, s_ref, 0))[live] < 1e-4)
        _check(out, *_reference(p, st, q, lens, s_got))
    # the separate attention and the one launch agree on the scores that the selector wrote
    fused = _outputs(p, 1)
    sas.decode_step_fused_kv4(p, bf16_dev(q), st.cache, _i32(lens), sd, fused)
    _ok()
    _check(fused, *_reference(p, st, q, lens, s_got))


def test_read_back_feeds_the_dense_forward():
    """The prompt read back is a valid input of the training forward, and decode agrees with its last row."""
    sas = _sas()
    p = _params(1, 4, 2, 128, 256, 8)
    st = Store(p, True, seed=1)
    k, v = _kv(1, 2, 256, 128, seed=7)
    sas.sas_kv4_write(p, st.cache, bf16_dev(k), bf16_dev(v), _i32([256]))
    ko, vo = (torch.empty((1, 2, 256, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    sas.sas_kv4_read(p, st.cache, ko, vo, _i32([256]))
    g = np.random.default_rng(1)
    qf = bf16_dev(bf16_round(g.standard_normal((1, 4, 256, 128)).astype(np.float32)))
    s = f32_dev(g.standard_normal((1, 2, 4, 4)).astype(np.float32))
    out = sas.empty_prefill_outputs(p, backward=False)
    sas.prefill_step(p, qf, ko, vo, s, None, out, backward=False)
    dec = _outputs(p, 1)
    sas.decode_step_fused_kv4(p, qf[:, :, -1].contiguous(), st.cache, _i32([256]), s[:, :, -1].contiguous(), dec)
    _ok()
    # the forward rounds K, V and P to bf16: three roundings of 2^-8 over |values| up to the row's sum of p |v|
    assert (dec["o"].float() - out["o"][:, :, -1].float()).abs().max() < 2e-2


def test_graph_replay_other_stream_and_two_graphs():
    """A captured write + step replays fresh inputs; two graphs over one cache and a side stream give the same."""
    sas = _sas()
    p = _params(2, 8, 2, 128, 512, 3)
    lens0 = [300, 64]
    st = _filled(p, True, seed=2, lens=lens0)
    k, v = _kv(2, 2, 4, 128, seed=6)
    kd, vd = bf16_dev(k[:, :, :1]), bf16_dev(v[:, :, :1])
    q, s = _qs(p, seed=5)
    qd, sd, cl = bf16_dev(q), f32_dev(s), _i32(lens0)
    outs = [_outputs(p, 1), _outputs(p, 2)]

    def fused():
        sas.sas_kv4_write(p, st.cache, kd, vd, cl)
        sas.decode_step_fused_kv4(p, qd, st.cache, cl, sd, outs[0])

    def split():
        sas.decode_step_kv4(p, qd, st.cache, cl, sd, 2, outs[1])

    graphs = []
    for f in (fused, split):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            f()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side, capture_error_mode="thread_local"):
            f()
        graphs.append(g)
    st.write(k[:, :, :1], v[:, :, :1], lens0, [1, 1])  # the eager warm-up wrote position lens0 - 1
    lens = lens0
    for i in range(1, 4):
        lens = [L + 1 for L in lens]
        kd.copy_(bf16_dev(k[:, :, i:i + 1]))
        vd.copy_(bf16_dev(v[:, :, i:i + 1]))
        q, s = _qs(p, seed=20 + i)
        qd.copy_(bf16_dev(q))
        sd.copy_(f32_dev(s))
        cl.copy_(_i32(lens))
        for g in graphs:
            g.replay()
        _ok()
        st.write(k[:, :, i:i + 1], v[:, :, i:i + 1], lens, [1, 1])
        st.same()
        ref = _reference(p, st, q, lens, s)
        for out in outs:
            _check(out, *ref)


def test_optional_outputs_and_refusals_of_the_binding():
    sas = _sas()
    p = _params(1, 4, 2, 128, 256, 3)
    st = _filled(p, False, seed=2, lens=[256])
    q, s = _qs(p, seed=5)
    full = _run(p, st, q, [256], s, 1, "fused")
    o = torch.empty_like(full["o"])
    sas.sas_decode_fused_kv4(p, bf16_dev(q), st.cache, _i32([256]), f32_dev(s), o)
    _ok()
    assert torch.equal(o, full["o"])
    k = torch.zeros((1, 2, 1, 128), dtype=torch.bfloat16, device="cuda")
    cl = _i32([1])
    for bad in (k.float(), k[:, :, :, ::2], torch.zeros((1, 2, 128, 2), device="cuda", dtype=torch.bfloat16).transpose(2, 3),
                k.cpu(), torch.zeros((1, 3, 1, 128), device="cuda", dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            sas.sas_kv4_write(p, st.cache, bad, bad, cl)
    with pytest.raises(ValueError):
        sas.sas_kv4_write(p, st.cache, k, k, cl.long())
    with pytest.raises(ValueError):
        sas.sas_kv4_read(p, st.cache, None, None, cl)
    with pytest.raises(ValueError):  # another sequence length than the cache's
        sas.sas_kv4_write(_params(1, 4, 2, 128, 512, 3), st.cache, k, k, cl)
    with pytest.raises(ValueError):
        sas.Kv4Cache(p, st.dev["k"], st.dev["v"][:, :, :, :-1])
    with pytest.raises(sas.SasError):
        sas.sas_kv4_write(p, st.cache, k.expand(1, 2, 300, 128).contiguous(), k.expand(1, 2, 300, 128).contiguous(), cl)


# ---------------------------------------------------------------------------------------------------------------
# what could go wrong
# ---------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("d", [64, 128])
def test_write_windows_at_every_offset(d):
    """Windows that begin and end at each of a tile's 16 tokens, in the middle of a block and across two."""
    sas = _sas()
    p = _params(16, 2, 2, d, 192)
    for T in (1, 15, 16, 35, 80):
        st = Store(p, True, seed=T)
        k, v = _kv(16, 2, T, d, seed=T)
        lens = [T + 23 + off for off in range(16)]
        sas.sas_kv4_write(p, st.cache, bf16_dev(k), bf16_dev(v), _i32(lens))
        _ok()
        st.write(k, v, lens, [T] * 16)
        st.same()


def _score_rows(kind, shape, g):
    s = (g.standard_normal(shape) * np.sqrt(2)).astype(np.float32)
    if kind == "same":
        s[:] = 0.75
    elif kind == "few":
        s = g.choice(np.array([-1.0, -0.0, 0.0, 2.0], np.float32), shape)
    elif kind == "special":
        s = g.choice(np.array([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-40, 3.4e38, -3.4e38, 1.0], np.float32), shape)
    elif kind == "close":  # neighbours in fp32
        s = (1.0 + g.integers(0, 40, shape) * 2.0 ** -23).astype(np.float32)
    elif kind == "outlier":
        s[..., 0], s[..., -1] = 3e38, -3e38
    elif kind == "magnitudes":
        s = (s * np.exp2(g.integers(-120, 120, shape))).astype(np.float32)
    return s


@pytest.mark.parametrize("kind", ["normal", "same", "few", "special", "close", "outlier", "magnitudes"])
@pytest.mark.parametrize("NB", [1, 2, 5, 33, 128, 129, 512, 513, 2048])
def test_one_launch_selection_is_the_select_kernels(NB, kind):
    sas = _sas()
    g = np.random.default_rng(NB)
    s = _score_rows(kind, (3, 2, NB), g)
    lens = [64 * NB, 64 * max(NB - 1, 1), int(g.integers(1, 64 * NB + 1))]
    cl, sd = _i32(lens), f32_dev(s)
    for K in sorted({1, 3, 32, 64, 255, min(NB, 255)}):
        p = _params(3, 2, 2, 64, 64 * NB, K)
        cache = sas.empty_kv4_cache(p)
        cache.k.zero_(), cache.v.zero_()
        q = torch.ones((3, 2, 64), dtype=torch.bfloat16, device="cuda")
        out = _outputs(p)
        sas.decode_step_fused_kv4(p, q, cache, cl, sd, out)
        idx, lse = torch.empty_like(out["idx"]), torch.empty_like(out["lse_s"])
        sas.sas_topk_select(p, sd, idx, lse, cache_len=cl)
        _ok()
        assert torch.equal(out["idx"], idx), (NB, K, kind)
        a, b = host(out["lse_s"]), host(lse)
        same = (a == b) | (np.isnan(a) & np.isnan(b))
        # a sum of up to 2048 fp32 terms in another order, each side off by log2(2048) + 16 roundings at most
        with np.errstate(invalid="ignore"):
            near = np.abs(a - b) <= 64 * 2.0 ** -24 * (1 + np.abs(b))
        assert np.all(same | near), (NB, K, kind)
        assert torch.all(out["o"] == 0)


@pytest.mark.parametrize("gate", [O.GATE_LOG_SIGMOID, O.GATE_LOGIT])
@pytest.mark.parametrize("form", ["fused", "split"])
def test_gates_that_close_leave_the_current_block(gate, form):
    """Every pick's gate is 0 (log g = -inf): rows of whole splits are empty, and the current block stands alone."""
    p = _params(2, 8, 2, 128, 1024, 9, gate)
    lens = [1024, 700]
    st = _filled(p, True, seed=3, lens=lens)
    q, s = _qs(p, seed=3)
    s[0] = -np.inf
    s[1, :, ::2] = -np.inf
    out = _run(p, st, q, lens, s, 5, form)
    # the same picks and the same outputs as of gates of e^-200, which are below every rounding here
    _check(out, *_reference(p, st, q, lens, np.where(np.isfinite(s), s, np.float32(-200.0))), lse_s=False)
    if form == "split":
        lp = host(out["lse_part"])
        assert np.all(lp[0, :, 1:] == -np.inf) and torch.all(out["o_part"][0, :, 1:] == 0)


@pytest.mark.parametrize("form", ["fused", "split"])
@pytest.mark.parametrize("qs,ks,vs", [(1e33, 1e-33, 1.0), (1e-30, 1e30, 1.0), (1.0, 1.0, 1e37), (1.0, 1.0, 1e-36)])
def test_decode_at_the_ends_of_the_range(qs, ks, vs, form):
    p = _params(2, 8, 2, 128, 512, 3)
    lens = [512, 77]
    st = Store(p, False, seed=5, fill=0xFF)
    k, _ = _kv(2, 2, 512, 128, seed=5, scale=ks)
    _, v = _kv(2, 2, 512, 128, seed=6, scale=vs)
    st.write(k, v, lens, lens)
    st.handle()
    q, s = _qs(p, seed=7, scale=qs)
    _check(_run(p, st, q, lens, s, 2, form), *_reference(p, st, q, lens, s))


def test_merge_has_the_same_bits_for_few_and_many_rows():
    """sas_decode_combine spreads few rows over more warps; a row's result does not depend on that, nor on NaN next to it."""
    sas = _sas()
    for d in (64, 128):
        for n in (1, 9, 33, 64):
            g = torch.Generator(device="cuda").manual_seed(n)
            few, many = _params(8, 32, 8, d, 4096, 64), _params(9, 32, 8, d, 4096, 64)  # 256 and 288 rows
            o_part = torch.randn((9, 32, n, d), device="cuda", generator=g)
            lse_part = 3 * torch.randn((9, 32, n), device="cuda", generator=g)
            lse_part[1, 3, 0] = -np.inf
            lse_part[2, 5] = -np.inf
            lse_part[4, 6, n - 1] = np.nan
            o_part[4, 6, n - 1] = np.nan
            res = []
            for p in (few, many):
                o = torch.empty((p.batch, 32, d), dtype=torch.bfloat16, device="cuda")
                lse = torch.empty((p.batch, 32), dtype=torch.float32, device="cuda")
                sas.sas_decode_combine(p, n, o_part[:p.batch].contiguous(), lse_part[:p.batch].contiguous(), o, lse)
                res.append((o, lse))
            _ok()
            assert torch.equal(res[0][0].view(torch.int16), res[1][0][:8].view(torch.int16))
            a, b = res[0][1], res[1][1][:8]
            assert torch.equal(torch.nan_to_num(a, nan=7.0), torch.nan_to_num(b, nan=7.0))
            assert torch.isnan(res[0][0][4, 6]).all() and torch.isnan(a[4, 6]) and torch.isnan(a).sum() == 1
            assert torch.all(res[0][0][2, 5] == 0) and a[2, 5] == -np.inf


def test_two_streams_at_once():
    """Steps of two batches on two streams, none waiting for the other, give what each gives alone."""
    sas = _sas()
    runs = []
    for seed, (d, Lmax, K) in ((1, (128, 2048, 8)), (2, (64, 1024, 5))):
        p = _params(3, 12, 3, d, Lmax, K, O.GATE_LOG_SOFTMAX)
        lens = [Lmax, Lmax // 2 + 5, 70]
        st = _filled(p, True, seed=seed, lens=lens)
        q, s = _qs(p, seed=seed)
        alone = (_run(p, st, q, lens, s, 2, "fused"), _run(p, st, q, lens, s, 2, "split"))
        runs.append((p, st, bf16_dev(q), _i32(lens), f32_dev(s), alone, [_outputs(p, 2) for _ in range(2)], torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for p, st, q, cl, s, alone, outs, stream in runs:
            sas.decode_step_fused_kv4(p, q, st.cache, cl, s, outs[0], stream=stream)
            sas.decode_step_kv4(p, q, st.cache, cl, s, 2, outs[1], stream=stream)
    _ok()
    for p, st, q, cl, s, alone, outs, stream in runs:
        for want, got in zip(alone, outs):
            assert all(torch.equal(want[k], got[k]) for k in ("o", "lse_o", "idx", "lse_s"))


def test_captured_steps():
    """DecodeGraph.kv4: the three steps, replayed on new inputs, are the eager ones."""
    sas = _sas()
    p = _params(2, 8, 2, 128, 512, 3)
    lens = [300, 64]
    st = _filled(p, True, seed=2, lens=lens)
    q, s = _qs(p, seed=5)
    qd, sd, cl = bf16_dev(q), f32_dev(s), _i32(lens)
    km = torch.zeros((2, 2, 8, 128), dtype=torch.bfloat16, device="cuda")
    sas.sas_kv4_block_mean_keys(p, st.cache, 300, cl, km, cl)
    k, v = _kv(2, 2, 3, 128, seed=6)
    kd, vd = bf16_dev(k[:, :, :1]), bf16_dev(v[:, :, :1])
    outs = [_outputs(p, 2) for _ in range(3)]
    s3 = torch.zeros_like(sd)
    graphs = [sas.DecodeGraph.kv4(p, qd, st.cache, cl, sd, 2, outs[0], fused=True),
              sas.DecodeGraph.kv4(p, qd, st.cache, cl, sd, 2, outs[1]),
              sas.DecodeGraph.kv4(p, qd, st.cache, cl, s3, 2, outs[2], kmean=km, k_new=kd, v_new=vd)]
    for i in range(3):
        q, s = _qs(p, seed=30 + i)
        cl.copy_(_i32([L + i for L in lens]))
        for dst, src in ((qd, q), (kd, k[:, :, i:i + 1]), (vd, v[:, :, i:i + 1])):
            dst.copy_(bf16_dev(src))
        sd.copy_(f32_dev(s))
        for g in reversed(graphs):  # the scored one first: it writes the token that all of them read
            g.replay()
        want = [_outputs(p, 2) for _ in range(3)]
        sas.decode_step_fused_kv4(p, qd, st.cache, cl, sd, want[0])
        sas.decode_step_kv4(p, qd, st.cache, cl, sd, 2, want[1])
        sas.decode_step_scored_kv4(p, qd, kd, vd, st.cache, km, cl, torch.zeros_like(s3), 2, want[2])
        _ok()
        for a, b in zip(want, outs):
            assert all(torch.equal(a[x], b[x]) for x in ("o", "lse_o", "idx", "lse_s"))
    with pytest.raises(ValueError):
        sas.decode_step_scored_kv4(p, qd, bf16_dev(k), bf16_dev(v), st.cache, km, cl, s3, 2, outs[2])

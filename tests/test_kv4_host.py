"""The 4-bit KV cache without a GPU: its oracle's own checks, and what the C ABI and the binding refuse."""
import ctypes

import numpy as np
import pytest
import torch

import learned_block_sparse_warp_b200 as sas
import oracle.kv4_oracle as KV
from learned_block_sparse_warp_b200 import Params, lib, sas_kv4_cache
from synth.workloads import bf16_round

OK, INVALID, UNSUPPORTED = 0, 1, 2
A = 0x7F0000000000  # aligned fake address; only ever handed to calls that reject their arguments


# ---------------------------------------------------------------------------------------------------------------
# the oracle
# ---------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("scale", [1e-30, 1e-3, 1.0, 1e4, 1e30])
def test_every_value_is_within_half_a_step(scale):
    x = bf16_round((np.random.default_rng(1).standard_normal((50, 128)) * scale).astype(np.float32))
    codes, step, low = KV.quantise(x)
    s = np.repeat(KV._bf16_value(step), 32, axis=-1)
    assert codes.min() == 0 and codes.max() == 15
    assert np.all(np.abs(KV.values(codes, step, low) - x) <= 0.5 * s * (1 + 1e-12))


def test_half_way_values_go_up():
    x = np.zeros((1, 64))
    x[0, :3], x[0, 32:35] = [15.0, 0.5, 2.5], [-8.0, 7.0, -7.5]  # s = 1 in both groups
    codes, step, low = KV.quantise(x)
    assert KV._bf16_value(step).tolist() == [[1.0, 1.0]] and KV._bf16_value(low).tolist() == [[0.0, -8.0]]
    assert codes[0, :4].tolist() == [15, 1, 3, 0] and codes[0, 32:36].tolist() == [0, 15, 1, 8]


def test_groups_without_a_step():
    x = np.zeros((1, 128))
    x[0, :32], x[0, 32], x[0, 64], x[0, 96] = 3.25, np.nan, -np.inf, 1e-39
    codes, step, low = KV.quantise(x)
    v = KV.values(codes, step, low)
    assert np.all(v[0, :32] == 3.25) and np.isnan(v[0, 32:96]).all() and np.all(v[0, 96:] == 0.0)
    assert np.all(step == 0) and np.all(codes == 0)


@pytest.mark.parametrize("side", ["k", "v"])
@pytest.mark.parametrize("d", [64, 128])
def test_pack_and_unpack_are_inverse(d, side):
    g = np.random.default_rng(d)
    codes = g.integers(0, 16, (150, d)).astype(np.uint8)
    step, low = (KV._bf16_bits(g.standard_normal((150, d // 32)).astype(np.float32)) for _ in range(2))
    rec = np.full((4, 40 * d), 0xA5, np.uint8)
    KV.pack_into(rec, side, codes, step, low, 37)
    got = KV.unpack(rec, side).reshape(256, d)[37:187]
    assert np.array_equal(got, KV.values(codes, step, low))
    # every byte of the block that is written whole has its place, and the others keep theirs
    flat = np.full((4, 40 * d), 0x5A, np.uint8)
    KV.pack_into(flat, side, codes, step, low, 37)
    assert np.array_equal(rec[1], flat[1]) and np.all(rec[3] == 0xA5)


# ---------------------------------------------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------------------------------------------
def _p(**kw):
    base = dict(batch=2, n_q_heads=8, n_kv_heads=2, head_dim=128, seq_len=1024, top_k=4)
    base.update(kw)
    return Params(**base)


def _c(k=A, v=A, table=None, n_pages=0):
    return sas_kv4_cache(k, v, table, n_pages)


def _write(p=None, c=None, T=1, k=A, v=A, cl=A, nl=None):
    return lib.sas_kv4_write((p or _p()).c(), _c() if c is None else c, T, k, v, cl, nl, None)


def _read(p=None, c=None, T=1, k=A, v=A, cl=A, nl=None):
    return lib.sas_kv4_read((p or _p()).c(), _c() if c is None else c, T, k, v, cl, nl, None)


def _means(p=None, c=None, T=1, cl=A, nl=None, km=A):
    return lib.sas_kv4_block_mean_keys((p or _p()).c(), _c() if c is None else c, T, cl, nl, km, None)


def _split(p=None, c=None, q=A, cl=A, s=A, idx=A, lse=A, n=1, o=A, lp=A):
    return lib.sas_decode_kv4((p or _p()).c(), q, _c() if c is None else c, cl, s, idx, lse, n, o, lp, None)


def _fused(p=None, c=None, q=A, cl=A, s=A, idx=None, lse=None, o=A, lo=None):
    return lib.sas_decode_fused_kv4((p or _p()).c(), q, _c() if c is None else c, cl, s, idx, lse, o, lo, None)


CALLS = [_write, _read, _means, _split, _fused]


@pytest.mark.parametrize("call", CALLS)
def test_bad_params_and_caches_are_refused(call):
    assert call(p=_p(head_dim=96)) == UNSUPPORTED
    assert call(p=_p(seq_len=1000)) == INVALID
    assert call(p=_p(batch=0)) == INVALID
    assert call(c=_c(k=None)) == INVALID
    assert call(c=_c(k=A + 8)) == INVALID
    assert call(c=_c(v=A + 8)) == INVALID
    assert call(c=_c(table=A, n_pages=0)) == INVALID
    assert call(c=_c(table=A, n_pages=-3)) == INVALID
    assert call(c=_c(table=A + 4, n_pages=10)) == INVALID
    assert call(c=_c(table=A, n_pages=2 ** 25)) == INVALID  # n_pages * Hkv records past the index range
    assert call(cl=None) == INVALID
    assert call(cl=A + 4) == INVALID


@pytest.mark.parametrize("call", [_write, _read, _split, _fused])
def test_the_v_records_are_needed(call):
    assert call(c=_c(v=None)) == INVALID


@pytest.mark.parametrize("call", [_write, _read, _means])
def test_token_counts_are_checked(call):
    for T in (0, -1, 1025):
        assert call(T=T) == INVALID
    assert call(nl=A + 4) == INVALID


def test_write_read_and_means_pointers():
    assert _write(k=None) == INVALID and _write(v=None) == INVALID and _write(k=A + 2) == INVALID
    assert _read(k=None, v=None) == INVALID and _read(k=A + 2) == INVALID and _read(v=A + 2) == INVALID
    assert _means(km=None) == INVALID and _means(km=A + 2) == INVALID
    assert lib.sas_kv4_write(_p().c(), None, 1, A, A, A, None, None) == INVALID
    assert lib.sas_kv4_write(None, _c(), 1, A, A, A, None, None) == INVALID


def test_decode_arguments():
    assert _split(p=_p(n_q_heads=18)) == UNSUPPORTED  # G = 9
    assert _fused(p=_p(n_q_heads=18)) == UNSUPPORTED
    assert _fused(p=_p(top_k=256)) == UNSUPPORTED
    assert _fused(p=_p(seq_len=64 * 2049)) == UNSUPPORTED
    assert _split(n=0) == INVALID and _split(n=6) == INVALID
    assert _split(p=_p(top_k=200), n=3) == UNSUPPORTED  # 67 blocks in a split
    for bad in (dict(q=None), dict(idx=None), dict(o=None), dict(lp=None), dict(s=None), dict(lse=None), dict(q=A + 2)):
        assert _split(**bad) == INVALID, bad
    for bad in (dict(q=None), dict(s=None), dict(o=None), dict(idx=A + 4), dict(lse=A + 4), dict(lo=A + 4)):
        assert _fused(**bad) == INVALID, bad


def test_struct_mirrors_the_header():
    assert [f for f, _ in sas_kv4_cache._fields_] == ["k", "v", "block_table", "n_pages"]
    assert ctypes.sizeof(sas_kv4_cache) == 32
    assert sas.kv4_record_bytes(128) == 5120 == KV.record_bytes(128)


def test_the_binding_refuses_cpu_tensors_and_half_paged_caches():
    p = _p()
    k = torch.zeros((2, 2, 16, 5120), dtype=torch.uint8)
    with pytest.raises(ValueError):
        sas.Kv4Cache(p, k, k.clone())
    with pytest.raises(ValueError):
        sas.empty_kv4_cache(p, n_pages=4, device="cpu")
    with pytest.raises(ValueError):
        sas.empty_kv4_cache(p, block_table=torch.zeros((2, 16), dtype=torch.int32), device="cpu")

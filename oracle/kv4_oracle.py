"""fp64 CPU oracle of the 4-bit KV cache: its quantisation and its byte format.

TEST INFRASTRUCTURE, like ``sas_oracle``: plain NumPy that shares no code with
the library. The attention over the cache is ``sas_oracle.decode`` on the
values that ``unpack`` returns.

A group is 32 channels of one token. m = min, s = bf16((max − min) / 15) with
the difference and the quotient in fp32, 0 below 2^-126, and
code = floor((x − m) / s + 1/2), exactly: the number of half-way points
(k + 1/2) s that x − m reaches. A group whose range is not a finite fp32
number is kept as s = 0, m = NaN. A minimum of zero is kept as +0.
"""
from __future__ import annotations

import numpy as np

GROUP, TILE, BLOCK = 32, 16, 64


def _bf16_bits(x) -> np.ndarray:
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), r)


def _bf16_value(bits) -> np.ndarray:
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def quantise(x):
    """x [..., d] of bf16 values -> (codes uint8 [..., d], step and minimum as bf16 bits [..., d/32])."""
    g = np.asarray(x, np.float64).reshape(*np.shape(x)[:-1], -1, GROUP)
    with np.errstate(all="ignore"):
        low, high = g.min(-1), g.max(-1)  # NaN if any is
        span = high.astype(np.float32) - low.astype(np.float32)
        bad = ~np.isfinite(span)
        step = _bf16_value(_bf16_bits(span / np.float32(15)))
        step = np.where(bad | (step < 2.0 ** -126), 0.0, step)
        # x − m as an unevaluated sum d + e; a half-way point has 13 bits, so d decides unless it is one
        m = low[..., None]
        d = g - m
        e = np.where(np.abs(g) >= np.abs(m), (g - d) - m, g - (d + m))
        q = np.zeros(g.shape)
        for k in range(15):
            half = (k + 0.5) * step[..., None]
            q += (d > half) | ((d == half) & (e >= 0))
    q = np.where(step[..., None] > 0, q, 0.0)
    assert q.min() >= 0 and q.max() <= 15
    low = np.where(bad, np.nan, low + 0.0)  # a minimum of -0 is kept as +0
    return q.astype(np.uint8).reshape(np.shape(x)), _bf16_bits(step), _bf16_bits(low)


def values(codes, step, low) -> np.ndarray:
    """What codes, steps and minima (bf16 bits) stand for, fp64 [..., d]."""
    s, m = _bf16_value(step)[..., None], _bf16_value(low)[..., None]
    c = np.asarray(codes, np.float64).reshape(*np.shape(step), GROUP)
    return (s * c + m).reshape(np.shape(codes))


def record_bytes(d: int) -> int:
    return 40 * d


def _places(d: int, side: str):
    """For (token of a record, channel): code byte and shift; for (token, group): byte of its step and minimum."""
    ng = d // GROUP
    tok, ch = np.meshgrid(np.arange(BLOCK), np.arange(d), indexing="ij")
    tile, r, j, p = tok // TILE, tok % TILE, ch // GROUP, ch % GROUP
    if side == "k":
        word, nib = (r * 4 + p // 8) * ng + j, p % 8
    else:
        u, t, half = r // 8, (r % 8) // 2, r % 2
        word, nib = ((u * 8 + p // 4) * 4 + t) * ng + j, 4 * half + p % 4
    code = tile * 10 * d + 4 * word + nib // 2
    tok, j = np.meshgrid(np.arange(BLOCK), np.arange(ng), indexing="ij")
    tile, r = tok // TILE, tok % TILE
    by_token = r * ng + j
    order = by_token if side == "k" else ((r % 8) // 2 * ng + j) * 4 + 2 * (r // 8) + r % 2
    base = tile * 10 * d + 8 * d
    return code, 4 * (nib % 2), base + 2 * order, base + 2 * TILE * ng + 2 * by_token


def _raw(records, side: str):
    """Codes [..., 64, d], steps and minima (bf16 bits) [..., 64, d/32] of records [..., 40 d]."""
    records = np.asarray(records)
    code_at, shift, step_at, low_at = _places(records.shape[-1] // 40, side)
    step, low = (records[..., at].astype(np.uint16) | (records[..., at + 1].astype(np.uint16) << 8)
                 for at in (step_at, low_at))
    return (records[..., code_at] >> shift.astype(np.uint8)) & 15, step, low


def pack(codes, step, low, side: str) -> np.ndarray:
    """Records [..., 40 d] of whole blocks: codes [..., 64, d], steps and minima (bf16 bits) [..., 64, d/32]."""
    d = codes.shape[-1]
    code_at, shift, step_at, low_at = _places(d, side)
    rec = np.zeros((*codes.shape[:-2], 40 * d), np.uint8)
    for sh in (0, 4):  # the two nibbles of a byte
        rec[..., code_at[shift == sh]] |= codes[..., shift == sh] << sh
    for bits, at in ((step, step_at), (low, low_at)):
        rec[..., at], rec[..., at + 1] = (bits & 255).astype(np.uint8), (bits >> 8).astype(np.uint8)
    return rec


def pack_into(records, side: str, codes, step, low, first: int) -> None:
    """Writes n tokens (codes [n, d], steps and minima [n, d/32]) at positions first.. of records [NB, 40 d], in place."""
    old = _raw(records, side)
    flat = [x.reshape(-1, x.shape[-1]).copy() for x in old]
    for x, new in zip(flat, (codes, step, low)):
        x[first:first + len(new)] = new
    records[:] = pack(*(x.reshape(o.shape) for x, o in zip(flat, old)), side)


def unpack(records, side: str) -> np.ndarray:
    """Values of records [..., 40 d], fp64 [..., 64, d]."""
    return values(*_raw(records, side))

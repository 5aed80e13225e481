"""Cases of the 4-bit KV cache: writing and reading it, its block means, and the sparse decode over it.

The cache keeps K and V in 4 bits. Every token's d channels are cut into groups of 32. A group holds its minimum m
and a step s, both bf16, and sixteen levels: value = s * code + m, with s = bf16((max - min) / 15) and
code = floor((x - m) / s + 1/2) in 0..15. A step below 2^-126 is 0, and then so is every code. A group whose range is
not finite has s = 0 and m = NaN, so that all of it reads as NaN.

One record of 40 d bytes holds 64 tokens of one KV head, of K or of V, as four tiles of 16 tokens. With NG = d / 32
groups, a tile has 8 d bytes of codes and then its steps and minima. Words are 32 bits, little endian, and nibble 0
is the lowest:
  K codes  word [token 0..15][t 0..3][group j]                  nibble p is channel 32 j + 8 t + p
  K steps  bf16 [token][group], minima bf16 [token][group]
  V codes  word [u 0..1][g 0..7][t 0..3][group j]               low half: token 8 u + 2 t, high half: the next token;
                                                                nibble p of a half is channel 32 j + 4 g + p
  V steps  bf16 [t][group][i 0..3] of token 8 (i / 2) + 2 t + i % 2, minima bf16 [token][group]
Records lie densely, [B, Hkv, NKB, 40 d], or in pages, [n_pages, Hkv, 40 d], with the page of block m of sequence b
at block_table[b, m].

A decode step takes one query token for each sequence, at position L - 1. The K history blocks with the highest
scores (ties to the lower block) and the current block, up to L - 1, are attended to. Under the log-softmax gate
log g_m = s_m - LSE(s) is added to the logits of history block m.
"""
import math

import torch

own = False

BLOCK, TILE, GROUP = 64, 16, 32
GATE_LOG_SOFTMAX, GATE_NONE = 0, 1


# ---------------------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------------------
def listed():
    c = []
    # one step's new token of 16 sequences, into pages: the smallest write there is
    c.append(dict(name="write one token B16", op="write", B=16, Hkv=8, d=128, Lmax=32768, T=1, paged=True, ragged=False))
    # a whole prompt goes into an empty cache
    c.append(dict(name="write prompt 32K", op="write", B=1, Hkv=8, d=128, Lmax=32768, T=32768, paged=False, ragged=False))
    # chunks of a prompt, each sequence's of its own length, at odd positions
    c.append(dict(name="write ragged chunk d64", op="write", B=5, Hkv=2, d=64, Lmax=4096, T=517, paged=True, ragged=True))
    # a long cache read back whole, for a dense pass over it
    c.append(dict(name="read 64K", op="read", B=1, Hkv=8, d=128, Lmax=65536, T=65536, paged=False, ragged=False))
    # the last tokens of a few sequences
    c.append(dict(name="read ragged d64", op="read", B=3, Hkv=3, d=64, Lmax=2048, T=1000, paged=True, ragged=True))
    # the selector's block means after a long prompt
    c.append(dict(name="means 64K", op="means", B=1, Hkv=8, d=128, Lmax=65536, T=65536, paged=False, ragged=False))
    # the selector's means after one step: few sequences have just filled a block
    c.append(dict(name="means one token B16", op="means", B=16, Hkv=8, d=128, Lmax=8192, T=1, paged=True, ragged=True))
    # the serving step of this repository's decode benchmark
    c.append(dict(name="step B16 32K K16", op="fused", B=16, Hkv=8, G=4, d=128, Lmax=32768, K=16, paged=True, ragged=False, gate=GATE_NONE))
    # one sequence, 40 query heads on 8 KV heads, the gate kept
    c.append(dict(name="step B1 8K K64 gated", op="fused", B=1, Hkv=8, G=5, d=128, Lmax=8192, K=64, paged=False, ragged=False, gate=GATE_LOG_SOFTMAX))
    # short ragged sequences, small heads
    c.append(dict(name="step B7 1K K4 d64", op="fused", B=7, Hkv=2, G=4, d=64, Lmax=1024, K=4, paged=True, ragged=True, gate=GATE_NONE))
    # the separate calls at a large budget: select, split attention, merge
    c.append(dict(name="split B8 64K K64 gated", op="split", B=8, Hkv=8, G=4, d=128, Lmax=65536, K=64, paged=True, ragged=True, gate=GATE_LOG_SOFTMAX))
    # every block of 128K tokens: attention over the whole cache
    c.append(dict(name="split B1 128K all blocks", op="split", B=1, Hkv=8, G=4, d=128, Lmax=131072, K=2048, paged=False, ragged=False, gate=GATE_NONE))
    return c


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "means", "fused", "fused", "split"])
    c = dict(op=op, B=_log_int(rng, 1, 16), Hkv=rng.choice([1, 2, 3, 4, 8]), d=rng.choice([64, 128, 128]), paged=rng.random() < 0.5, ragged=rng.random() < 0.6)
    if op in ("write", "read", "means"):
        c["T"] = _log_int(rng, 2 * BLOCK if op == "means" else 1, 32768 // c["B"])  # means: one block at least is done
        c["Lmax"] = BLOCK * -(-(c["T"] + rng.randrange(0, 200)) // BLOCK)
        return c
    c["G"] = rng.randrange(1, 9)
    c["gate"] = rng.choice([GATE_NONE, GATE_LOG_SOFTMAX])
    blocks = _log_int(rng, 2, 2048 // c["B"])
    c["Lmax"] = BLOCK * blocks
    c["K"] = _log_int(rng, 1, min(blocks + 4, 255 if op == "fused" else 2048))
    return c


def _spread(c, b, lo, hi, salt):
    """A whole number of [lo, hi] for sequence b, by the case alone."""
    return lo + ((b + 1) * 2654435761 + salt * 40503 + c["Lmax"]) % 1000003 % (hi - lo + 1)


def _lens(c):
    """(cache_len, new_len) of every sequence. Without "T": decode, one new token."""
    B, top = c["B"], c["Lmax"]
    if "T" not in c:
        return ([_spread(c, b, 1, top, 1) for b in range(B)] if c["ragged"] else [top] * B), [1] * B
    if c["op"] == "means" and c["T"] == 1 and c["ragged"]:  # every fourth sequence has just filled a block
        return [BLOCK * _spread(c, b, 1, top // BLOCK, 2) - (1 if b % 4 else 0) for b in range(B)], [1] * B
    new = [_spread(c, b, (c["T"] + 1) // 2, c["T"], 3) for b in range(B)] if c["ragged"] else [c["T"]] * B
    return [_spread(c, b, n, top, 4) if c["ragged"] else top for b, n in enumerate(new)], new


def _n_split(c):
    """Splits that give the card a few CTAs per multiprocessor, each of at most 64 blocks."""
    blocks = c["K"] + 1
    want = max(1, 592 // (c["B"] * c["Hkv"]))
    return max(-(-blocks // 64), min(blocks, want, 64))


# ---------------------------------------------------------------------------------------------------------------
# What a program has in hand
# ---------------------------------------------------------------------------------------------------------------
def _records(shape, d, order, gen):
    """A filled cache: random codes, with steps and minima as groups of normal values have them."""
    ng = d // GROUP
    lead = list(shape) + [BLOCK // TILE]
    codes = torch.randint(0, 256, lead + [8 * d], dtype=torch.uint8, device="cuda", generator=gen)
    step = (torch.rand(lead + [TILE * ng], device="cuda", generator=gen) * 0.2 + 0.18).to(torch.bfloat16)
    middle = 7.5 + 1.5 * torch.randn(lead + [TILE * ng], device="cuda", generator=gen)
    if order == "v":  # minima are [token][group], steps [t][group][i]
        by_token = step.view(lead + [4, ng, 2, 2]).movedim(-2, -4).movedim(-1, -2).reshape(lead + [TILE * ng])
    else:
        by_token = step
    low = (-by_token.float() * middle).to(torch.bfloat16)
    return torch.cat([codes, step.view(torch.uint8), low.view(torch.uint8)], dim=-1).view(list(shape) + [40 * d])


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B, Hkv, d, nkb = c["B"], c["Hkv"], c["d"], c["Lmax"] // BLOCK
    lens, new = _lens(c)
    st = dict(case=c)
    st["cache_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["new_len"] = torch.tensor(new, dtype=torch.int32, device="cuda")
    if c["paged"]:
        pages = B * nkb
        st["table"] = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32).view(B, nkb)
        shape = (pages, Hkv)
    else:
        st["table"] = None
        shape = (B, Hkv, nkb)
    if c["op"] == "write":  # an empty cache
        st["kr"] = torch.zeros(list(shape) + [40 * d], dtype=torch.uint8, device="cuda")
        st["vr"] = torch.zeros(list(shape) + [40 * d], dtype=torch.uint8, device="cuda")
    else:
        st["kr"] = _records(shape, d, "k", gen)
        st["vr"] = _records(shape, d, "v", gen)
    if c["op"] in ("write", "read"):
        bf = dict(dtype=torch.bfloat16, device="cuda")
        st["k_out"], st["v_out"] = torch.zeros((B, Hkv, c["T"], d), **bf), torch.zeros((B, Hkv, c["T"], d), **bf)
    if c["op"] == "write":  # keys have a few strong channels and an offset, values have neither
        loud = 1.0 + 3.0 * (torch.arange(d, device="cuda") % 21 == 5)
        k = torch.randn((B, Hkv, c["T"], d), device="cuda", generator=gen) * loud + 0.5 * torch.randn((1, Hkv, 1, d), device="cuda", generator=gen)
        st["k"] = k.to(torch.bfloat16)
        st["v"] = torch.randn((B, Hkv, c["T"], d), device="cuda", generator=gen).to(torch.bfloat16)
    if c["op"] == "means":
        st["kmean"] = torch.zeros((B, Hkv, nkb, d), dtype=torch.bfloat16, device="cuda")
    if c["op"] in ("fused", "split"):
        Hq, K = Hkv * c["G"], c["K"]
        f32 = dict(dtype=torch.float32, device="cuda")
        st["q"] = torch.randn((B, Hq, d), device="cuda", generator=gen).to(torch.bfloat16)
        st["s"] = math.sqrt(2.0) * torch.randn((B, Hkv, nkb), device="cuda", generator=gen)
        st["out"] = dict(o=torch.empty((B, Hq, d), dtype=torch.bfloat16, device="cuda"), lse_o=torch.empty((B, Hq), **f32),
                         idx=torch.empty((B, Hkv, K), dtype=torch.int32, device="cuda"), lse_s=torch.empty((B, Hkv), **f32))
        if c["op"] == "split":
            n = _n_split(c)
            st["out"].update(o_part=torch.empty((B, Hq, n, d), **f32), lse_part=torch.empty((B, Hq, n), **f32))
    return st


# ---------------------------------------------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------------------------------------------
def _round_trip(x):
    """What the cache holds of x, as the values it stands for."""
    g = x.view(*x.shape[:-1], -1, GROUP).double()
    low, high = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    span = (high - low).float()
    step = (span.double() / 15.0).float().to(torch.bfloat16).double()
    step = torch.where(step < 2.0 ** -126, torch.zeros_like(step), step)
    bad = ~torch.isfinite(span)
    step, low = step.masked_fill(bad, 0.0), low.masked_fill(bad, math.nan)
    code = torch.where(step > 0, torch.floor((g - low) / step + 0.5).clamp(0, 15), torch.zeros_like(g))
    return (step * code + low).view(x.shape).to(torch.bfloat16)


def _nibbles(b):
    return torch.stack([b & 15, b >> 4], dim=-1).float()


def _k_values(r, d):
    """Records [..., 40 d] of K to fp32 [..., 64, d]."""
    ng, lead = d // GROUP, list(r.shape[:-1])
    r = r.view(lead + [4, 10 * d])
    n = _nibbles(r[..., : 8 * d]).view(lead + [BLOCK, 4, ng, 8]).movedim(-2, -3)  # [token][group][t][nibble]
    par = r[..., 8 * d :].contiguous().view(torch.bfloat16).float().view(lead + [4, 2, TILE, ng])
    step, low = (par[..., i, :, :].reshape(lead + [BLOCK, ng, 1, 1]) for i in (0, 1))
    return (n * step + low).reshape(lead + [BLOCK, d])


def _v_values(r, d):
    """Records [..., 40 d] of V to fp32 [..., 64, d]."""
    ng, lead = d // GROUP, list(r.shape[:-1])
    k = len(lead)
    r = r.view(lead + [4, 10 * d])
    n = _nibbles(r[..., : 8 * d]).view(lead + [4, 2, 8, 4, ng, 2, 4])  # [tile][u][g][t][group][parity][nibble]
    n = n.permute(list(range(k)) + [k + i for i in (0, 1, 3, 5, 4, 2, 6)]).reshape(lead + [BLOCK, ng, GROUP])
    par = r[..., 8 * d :].contiguous().view(torch.bfloat16).float().view(lead + [4, 2, TILE * ng])
    step = par[..., 0, :].view(lead + [4, 4, ng, 2, 2])  # [tile][t][group][u][parity]
    step = step.permute(list(range(k)) + [k + i for i in (0, 3, 1, 4, 2)]).reshape(lead + [BLOCK, ng, 1])
    low = par[..., 1, :].reshape(lead + [BLOCK, ng, 1])
    return (n * step + low).reshape(lead + [BLOCK, d])


def _gather(st, recs, blocks):
    """Records of logical blocks [B, Hkv, n] as [B, Hkv, n, 40 d]."""
    B, Hkv, _ = blocks.shape
    b = torch.arange(B, device="cuda").view(B, 1, 1)
    h = torch.arange(Hkv, device="cuda").view(1, Hkv, 1)
    if st["table"] is None:
        return recs[b, h, blocks]
    return recs[st["table"].long()[b, blocks], h]


def _window(st):
    """The blocks that hold the new tokens, and each token's place among them: [B, Hkv, n], [B, T], whether it is one."""
    c = st["case"]
    L, n = st["cache_len"].long(), st["new_len"].long()
    first = torch.div(L - n, BLOCK, rounding_mode="floor")
    span = min(c["Lmax"] // BLOCK, (c["T"] + BLOCK - 2) // BLOCK + 1)
    blocks = (first.view(-1, 1) + torch.arange(span, device="cuda")).clamp(max=c["Lmax"] // BLOCK - 1)
    i = torch.arange(c["T"], device="cuda")
    place = (L - n - first * BLOCK).view(-1, 1) + i
    return blocks.view(c["B"], 1, span).expand(-1, c["Hkv"], -1), place.clamp(max=span * BLOCK - 1), i < n.view(-1, 1)


def _read(st, which, values):
    c = st["case"]
    blocks, place, live = _window(st)
    x = values(_gather(st, st[which], blocks), c["d"]).flatten(2, 3)
    x = torch.gather(x, 2, place.view(c["B"], 1, -1, 1).expand(-1, c["Hkv"], -1, c["d"]))
    return x.to(torch.bfloat16) * live.view(c["B"], 1, -1, 1)


def _means(st):
    """Means of the blocks that the new tokens completed, into the selector's buffer."""
    c = st["case"]
    L, n = st["cache_len"].long(), st["new_len"].long()
    blocks, _, _ = _window(st)
    m = blocks[:, 0]
    done = (BLOCK * (m + 1) <= L.view(-1, 1)) & (BLOCK * (m + 1) > (L - n).view(-1, 1))
    mean = (_k_values(_gather(st, st["kr"], blocks), c["d"]).sum(-2) / BLOCK).to(torch.bfloat16)
    b, k = done.nonzero(as_tuple=True)
    st["kmean"][b, :, m[b, k]] = mean[b, :, k]
    return st["kmean"]


def _select(st):
    """(idx, LSE of the history's scores)."""
    c, s = st["case"], st["s"]
    cur = torch.div(st["cache_len"].long() - 1, BLOCK, rounding_mode="floor").view(-1, 1, 1)
    nkb, K = s.shape[-1], c["K"]
    m = torch.arange(nkb, device="cuda")
    hist = s.masked_fill(m >= cur, -math.inf)
    order = torch.sort(hist, dim=-1, descending=True, stable=True).indices[..., :K]
    order = order.masked_fill(torch.arange(order.shape[-1], device="cuda") >= cur, nkb)
    idx = torch.full((c["B"], c["Hkv"], K), -1, device="cuda")
    idx[..., : order.shape[-1]] = torch.sort(order, dim=-1).values
    idx = idx.masked_fill(idx >= nkb, -1)
    top = hist.amax(-1, keepdim=True)
    top = top.masked_fill(top == -math.inf, 0.0)
    return idx, torch.log(torch.exp(hist - top).sum(-1)) + top[..., 0]


def _step(st):
    c = st["case"]
    B, Hkv, G, d, K = c["B"], c["Hkv"], c["G"], c["d"], c["K"]
    idx, lse_s = _select(st)
    L = st["cache_len"].long().view(-1, 1, 1)
    cur = torch.div(L - 1, BLOCK, rounding_mode="floor")
    blocks = torch.cat([cur.expand(B, Hkv, 1), idx], dim=-1)
    at = blocks.clamp(min=0)
    k = _k_values(_gather(st, st["kr"], at), d).flatten(2, 3)
    logit = (st["q"].float().view(B, Hkv, G, d) / math.sqrt(d)) @ k.transpose(-1, -2)
    del k
    pos = at.unsqueeze(-1) * BLOCK + torch.arange(BLOCK, device="cuda")
    live = ((blocks >= 0).unsqueeze(-1) & (pos < L.unsqueeze(-1))).flatten(2, 3)
    if c["gate"] == GATE_LOG_SOFTMAX:
        gate = torch.gather(st["s"], -1, at) - lse_s.unsqueeze(-1)
        gate[..., 0] = 0.0
        logit = logit + gate.unsqueeze(-1).expand(-1, -1, -1, BLOCK).flatten(2, 3).unsqueeze(2)
    logit = logit.masked_fill(~live.unsqueeze(2), -math.inf)
    top = logit.amax(-1, keepdim=True)
    p = torch.exp(logit - top)
    total = p.sum(-1, keepdim=True)
    o = (p @ _v_values(_gather(st, st["vr"], at), d).flatten(2, 3)) / total
    return dict(o=o.to(torch.bfloat16).view(B, Hkv * G, d), lse_o=(torch.log(total) + top).view(B, Hkv * G), idx=idx.to(torch.int32), lse_s=lse_s)


# ---------------------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------------------
def run(state):
    st, c = state, state["case"]
    if own:
        import learned_block_sparse_warp_b200 as sas
        if "p" not in st:  # what a serving program makes once
            gate = dict(n_q_heads=c["Hkv"] * c["G"], top_k=c["K"], gate_mode=c["gate"]) if "G" in c else dict(n_q_heads=c["Hkv"], top_k=1)
            st["p"] = sas.Params(batch=c["B"], n_kv_heads=c["Hkv"], head_dim=c["d"], seq_len=c["Lmax"], **gate)
            st["cache"] = sas.Kv4Cache(st["p"], st["kr"], st["vr"], st["table"])
        p, cache, L, n = st["p"], st["cache"], st["cache_len"], st["new_len"]
        if c["op"] == "write":
            sas.sas_kv4_write(p, cache, st["k"], st["v"], L, n)
        if c["op"] in ("write", "read"):
            sas.sas_kv4_read(p, cache, st["k_out"], st["v_out"], L, n)
            return dict(k=st["k_out"], v=st["v_out"])
        if c["op"] == "means":
            sas.sas_kv4_block_mean_keys(p, cache, c["T"], L, st["kmean"], n)
            return st["kmean"]
        if c["op"] == "fused":
            sas.decode_step_fused_kv4(p, st["q"], cache, L, st["s"], st["out"])
        else:
            sas.decode_step_kv4(p, st["q"], cache, L, st["s"], st["out"]["o_part"].shape[2], st["out"])
        return {k: st["out"][k] for k in ("o", "lse_o", "idx", "lse_s")}
    if c["op"] == "write":
        live = (torch.arange(c["T"], device="cuda") < st["new_len"].view(-1, 1)).view(c["B"], 1, -1, 1)
        return dict(k=_round_trip(st["k"]) * live, v=_round_trip(st["v"]) * live)
    if c["op"] == "read":
        return dict(k=_read(st, "kr", _k_values), v=_read(st, "vr", _v_values))
    return _means(st) if c["op"] == "means" else _step(st)


def work(case):
    c = case
    lens, new = _lens(c)
    Hkv, d, B = c["Hkv"], c["d"], c["B"]
    held = d // 2 + d // 8  # bytes of one token in a record
    if c["op"] == "write":  # values in, records and the values they stand for out
        n = 2 * Hkv * sum(new)
        return dict(bytes=n * (2 * d + held + 2 * d) + 8 * B, flops=n * d * 6)
    if c["op"] == "read":
        n = 2 * Hkv * sum(new)
        return dict(bytes=n * (held + 2 * d) + 8 * B, flops=n * d * 2)
    if c["op"] == "means":
        done = Hkv * sum(L // BLOCK - (L - n) // BLOCK for L, n in zip(lens, new))
        return dict(bytes=done * (BLOCK * held + 2 * d) + 8 * B, flops=done * BLOCK * d * 3)
    cur = [(L - 1) // BLOCK for L in lens]
    tokens = [L - BLOCK * m + BLOCK * min(c["K"], m) for L, m in zip(lens, cur)]
    rows, Hq = B * Hkv, Hkv * c["G"]
    side = 4 * Hkv * sum(cur) + rows * (4 * c["K"] + 4) + B * Hq * (2 * d + 2 * d + 4)
    return dict(bytes=2 * held * Hkv * sum(tokens) + side, flops=4 * d * Hq * sum(tokens))


# ---------------------------------------------------------------------------------------------------------------
# The definition in 64 bits, sequence by sequence and head by head
# ---------------------------------------------------------------------------------------------------------------
def _table_of(d, which):
    """For each (token of a tile, channel): the byte, and the shift, of its code; and the place of its step and minimum."""
    ng = d // GROUP
    tok = torch.arange(TILE).view(-1, 1).expand(TILE, d)
    ch = torch.arange(d).view(1, -1).expand(TILE, d)
    j, r = ch // GROUP, ch % GROUP
    if which == "kr":
        word = (tok * 4 + r // 8) * ng + j
        nib = r % 8
        step = tok * ng + j
    else:
        u, t, e = tok // 8, tok % 8 // 2, tok % 2
        word = ((u * 8 + r // 4) * 4 + t) * ng + j
        nib = 4 * e + r % 4
        step = (t * ng + j) * 4 + 2 * u + e
    out = [word * 4 + nib // 2, 4 * (nib % 2), 8 * d // 2 + step, 8 * d // 2 + TILE * ng + tok * ng + j]
    return [x.cuda() for x in out]


def _tokens64(st, which, b, h, blocks, table):
    """Tokens of the logical blocks of one sequence's KV head, fp64 [64 n, d]."""
    d = st["case"]["d"]
    r = st[which][st["table"][b, blocks].long(), h] if st["table"] is not None else st[which][b, h, blocks]
    r = r.reshape(-1, 10 * d)
    byte, shift, step, low = table
    code = ((r[:, byte].int() >> shift.int()) & 15).double()
    half = r.view(torch.int16).view(torch.bfloat16)
    return (code * half[:, step].double() + half[:, low].double()).reshape(-1, d)


def exact(case, seed):
    c, st = case, prepare(case, seed)
    lens, new = _lens(c)
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    f64 = dict(dtype=torch.float64, device="cuda")
    if c["op"] in ("write", "read"):
        out = dict(k=torch.zeros((B, Hkv, c["T"], d), **f64), v=torch.zeros((B, Hkv, c["T"], d), **f64))
        for name in out:
            table = _table_of(d, name + "r")
            for b in range(B):
                if c["op"] == "write":
                    x = st[name][b, :, : new[b]].double().unflatten(-1, (-1, GROUP))
                    low, high = x.min(-1, keepdim=True)[0], x.max(-1, keepdim=True)[0]
                    step = ((high - low) / 15).to(torch.bfloat16).double()
                    code = torch.floor((2 * (x - low) + step) / (2 * step))
                    code = torch.minimum(code, torch.full_like(code, 15.0))
                    out[name][b, :, : new[b]] = (low + code * step).flatten(-2)
                    continue
                at = lens[b] - new[b]
                blocks = torch.arange(at // BLOCK, -(-lens[b] // BLOCK), device="cuda")
                for h in range(Hkv):
                    x = _tokens64(st, name + "r", b, h, blocks, table)
                    out[name][b, h, : new[b]] = x[at % BLOCK : at % BLOCK + new[b]]
        return out
    if c["op"] == "means":
        out, table = torch.zeros((B, Hkv, c["Lmax"] // BLOCK, d), **f64), _table_of(d, "kr")
        for b in range(B):
            lo, hi = (lens[b] - new[b]) // BLOCK, lens[b] // BLOCK
            for h in range(Hkv if hi > lo else 0):
                out[b, h, lo:hi] = _tokens64(st, "kr", b, h, torch.arange(lo, hi, device="cuda"), table).view(-1, BLOCK, d).mean(1)
        return out
    G, K, Hq = c["G"], c["K"], Hkv * c["G"]
    o, lse_o = torch.zeros((B, Hq, d), **f64), torch.zeros((B, Hq), **f64)
    idx, lse_s = torch.full((B, Hkv, K), -1, dtype=torch.int32, device="cuda"), torch.zeros((B, Hkv), **f64)
    kt, vt = _table_of(d, "kr"), _table_of(d, "vr")
    for b in range(B):
        cur = (lens[b] - 1) // BLOCK
        for h in range(Hkv):
            s = st["s"][b, h, :cur].double()
            m = torch.arange(cur, device="cuda")
            ahead = (s.view(1, -1) > s.view(-1, 1)) | ((s.view(1, -1) == s.view(-1, 1)) & (m.view(1, -1) < m.view(-1, 1)))
            pick = m[ahead.sum(1) < K]
            idx[b, h, : len(pick)] = pick.int()
            lse_s[b, h] = torch.logsumexp(s, 0) if cur else -math.inf
            blocks = torch.cat([pick, torch.tensor([cur], device="cuda")])
            bias = torch.zeros(len(blocks) * BLOCK, **f64)
            if c["gate"] == GATE_LOG_SOFTMAX and cur:
                bias[: len(pick) * BLOCK] = (s[pick] - lse_s[b, h]).repeat_interleave(BLOCK)
            n = len(pick) * BLOCK + lens[b] - cur * BLOCK
            q = st["q"][b, h * G : (h + 1) * G].double()
            z = q @ _tokens64(st, "kr", b, h, blocks, kt)[:n].T / math.sqrt(d) + bias[:n]
            lse_o[b, h * G : (h + 1) * G] = torch.logsumexp(z, -1)
            o[b, h * G : (h + 1) * G] = torch.softmax(z, -1) @ _tokens64(st, "vr", b, h, blocks, vt)[:n]
    return dict(o=o, lse_o=lse_o, idx=idx, lse_s=lse_s)

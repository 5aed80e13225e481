"""What the 4-bit cache's steps refuse, on the CPU: nothing may have been launched by then, for a step writes the cache, the
means and the scores before its attention. The library is replaced by a recorder, and the codes are the C entry's own."""
import types

import pytest
import torch

import learned_block_sparse_warp_b200 as sas
from tests.test_kv4_handle_host import Fake

INVALID, UNSUPPORTED = 1, 2
A = 0x7F0000000000


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append((name, args)) or 0


def _step(n_split=2, scored=True, at={}, **kw):
    """Arguments of a step whose tensors fit, at fake addresses; `at` moves some of them."""
    shape = dict(batch=2, n_q_heads=8, n_kv_heads=2, head_dim=128, seq_len=1024, top_k=4)
    shape.update(kw)
    p = sas.Params(gate_mode=sas.SAS_GATE_NONE, **shape)
    B, Hq, Hkv, d, NB, K = p.batch, p.n_q_heads, p.n_kv_heads, p.head_dim, p.n_blocks, p.top_k
    t = {}

    def tensor(name, shape, dtype):
        t[name] = Fake(A + 0x1000 * len(t) + at.get(name, 0), shape, dtype)
        return t[name]

    cache = sas.Kv4Cache(p, tensor("k", (B, Hkv, NB, 40 * d), torch.uint8), tensor("v", (B, Hkv, NB, 40 * d), torch.uint8))
    out = dict(idx=tensor("idx", (B, Hkv, K), torch.int32), lse_s=tensor("lse_s", (B, Hkv), torch.float32),
               o_part=tensor("o_part", (B, Hq, n_split, d), torch.float32),
               lse_part=tensor("lse_part", (B, Hq, n_split), torch.float32),
               o=tensor("o", (B, Hq, d), torch.bfloat16), lse_o=tensor("lse_o", (B, Hq), torch.float32))
    q, cl, s = tensor("q", (B, Hq, d), torch.bfloat16), tensor("cache_len", (B,), torch.int32), tensor("s", (B, Hkv, NB), torch.float32)
    km = tensor("kmean", (B, Hkv, NB, d), torch.bfloat16)
    new = [tensor(x, (B, Hkv, 1, d), torch.bfloat16) for x in ("k_new", "v_new")]
    if scored:
        return sas.decode_step_scored_kv4, (p, q, *new, cache, km, cl, s, n_split, out)
    return sas.decode_step_kv4, (p, q, cache, cl, s, n_split, out)


@pytest.fixture
def rec(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(sas, "_device", lambda: 0)
    monkeypatch.setattr(sas, "lib", r)
    monkeypatch.setattr(sas, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(sas, "sas_status_string", lambda code: str(code))
    return r


def test_a_good_step_makes_its_calls_in_order(rec):
    f, args = _step()
    f(*args)
    assert [n for n, _ in rec.calls] == ["sas_kv4_write", "sas_kv4_block_mean_keys", "sas_decode_select_scored",
                                         "sas_decode_kv4", "sas_decode_combine"]
    rec.calls.clear()
    f, args = _step(scored=False)
    f(*args)
    assert [n for n, _ in rec.calls] == ["sas_topk_select", "sas_decode_kv4", "sas_decode_combine"]


REFUSED = [(dict(n_q_heads=18), UNSUPPORTED),                  # G = 9
           (dict(n_split=0), INVALID), (dict(n_split=6), INVALID),
           (dict(n_split=3, top_k=200), UNSUPPORTED)]          # 67 blocks in a split


@pytest.mark.parametrize("scored", [True, False])
@pytest.mark.parametrize("kw,code", REFUSED + [(dict(at={x: 8}), INVALID) for x in
                                               ("q", "cache_len", "s", "idx", "lse_s", "o_part", "lse_part", "o", "lse_o")])
def test_a_refused_step_has_launched_nothing(rec, kw, code, scored):
    f, args = _step(scored=scored, **kw)
    with pytest.raises(sas.SasError) as e:
        f(*args)
    assert e.value.code == code and rec.calls == []


@pytest.mark.parametrize("kw,code", [(dict(at={x: 8}), INVALID) for x in ("kmean", "k_new", "v_new")]
                         + [(dict(batch=1, n_kv_heads=1, n_q_heads=1, seq_len=64 * (8 * 53248 + 2)), UNSUPPORTED)])
def test_a_refused_scored_step_has_launched_nothing(rec, kw, code):
    f, args = _step(**kw)
    with pytest.raises(sas.SasError) as e:
        f(*args)
    assert e.value.code == code and rec.calls == []


@pytest.mark.parametrize("kw,code", REFUSED)
def test_the_codes_are_the_c_entrys(kw, code):
    kw = dict(kw)
    n_split = kw.pop("n_split", 2)
    p = sas.Params(**dict(dict(batch=2, n_q_heads=8, n_kv_heads=2, head_dim=128, seq_len=1024, top_k=4), **kw))
    c = sas.sas_kv4_cache(A, A, None, 0)
    assert sas.lib.sas_decode_kv4(p.c(), A, c, A, A, A, A, n_split, A, A, None) == code


def test_rows_of_scores_past_a_clusters_memory():
    p = sas.Params(batch=1, n_q_heads=1, n_kv_heads=1, head_dim=128, seq_len=64 * (8 * 53248 + 2), top_k=4)
    assert sas.lib.sas_decode_select_scored(p.c(), A, A, A, A, A, A, None) == UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(k_new=1), dict(v_new=1), dict(kmean=1), dict(k_new=1, v_new=1), dict(kmean=1, k_new=1),
                                dict(kmean=1, k_new=1, v_new=1, fused=True)])
def test_a_captured_step_is_one_of_the_three(kw):
    cache = types.SimpleNamespace(k=None, v=None, block_table=None)
    with pytest.raises(ValueError, match="scored step"):
        sas.DecodeGraph.kv4(None, None, cache, None, None, 1, {}, **kw)

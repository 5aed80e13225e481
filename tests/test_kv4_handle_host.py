"""The 4-bit cache's handle on the CPU, over stand-ins for CUDA tensors: the pointers that its calls hand to the library are
those of the tensors that it shows."""
import pytest
import torch

import learned_block_sparse_warp_b200 as sas


class Fake:
    """What the binding looks at in a tensor."""

    def __init__(self, at, shape, dtype=torch.uint8, dev=0):
        self.at, self.shape, self.dtype, self.dev = at, torch.Size(shape), dtype, dev
        self.is_cuda, self.device = True, f"cuda:{dev}"

    def get_device(self):
        return self.dev

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.at


@pytest.fixture(autouse=True)
def device(monkeypatch):
    monkeypatch.setattr(sas, "_device", lambda: 0)


P = sas.Params(batch=2, n_q_heads=4, n_kv_heads=2, head_dim=64, seq_len=256, top_k=2)


def _table(at, **kw):
    return Fake(at, (2, 4), torch.int32, **kw)


def _paged():
    return sas.Kv4Cache(P, Fake(0x1000, (9, 2, 2560)), Fake(0x2000, (9, 2, 2560)), _table(0x3000))


def _seen(cache):
    c = cache.of(P)[0]._obj
    return c.k, c.v, c.block_table, c.n_pages


def test_a_new_block_table_is_used():
    cache = _paged()
    old = cache.of(P)[0]
    assert _seen(cache) == (0x1000, 0x2000, 0x3000, 9)
    new = _table(0x4000)
    cache.block_table = new
    assert cache.block_table is new and _seen(cache) == (0x1000, 0x2000, 0x4000, 9)
    assert old._obj.block_table == 0x3000  # a call that is under way keeps its own


@pytest.mark.parametrize("bad", [None, Fake(0x4000, (2, 5), torch.int32), Fake(0x4000, (2, 4), torch.int64),
                                 _table(0x4000, dev=1)])
def test_a_wrong_block_table_is_refused(bad):
    cache = _paged()
    table = cache.block_table
    with pytest.raises(ValueError):
        cache.block_table = bad
    assert cache.block_table is table and _seen(cache) == (0x1000, 0x2000, 0x3000, 9)


def test_a_dense_cache_stays_dense():
    cache = sas.Kv4Cache(P, Fake(0x1000, (2, 2, 4, 2560)), Fake(0x2000, (2, 2, 4, 2560)))
    with pytest.raises(ValueError):
        cache.block_table = _table(0x4000)
    cache.block_table = None
    assert _seen(cache) == (0x1000, 0x2000, None, 0)


@pytest.mark.parametrize("name", ["k", "v", "dims", "device"])
def test_the_rest_is_read_only(name):
    cache = _paged()
    with pytest.raises(AttributeError):
        setattr(cache, name, getattr(cache, name))


def test_memory_that_moved_is_followed():
    cache = _paged()
    cache.v.at, cache.block_table.at = 0x5000, 0x6000
    assert _seen(cache) == (0x1000, 0x5000, 0x6000, 9)
    cache.k.at, cache.k.shape = 0x7000, torch.Size((8, 2, 2560))  # resized to another number of pages than v has
    with pytest.raises(ValueError):
        cache.of(P)


def test_missing_tensors():
    with pytest.raises(ValueError):
        sas.Kv4Cache(P, None, None)
    with pytest.raises(ValueError):
        sas.Kv4Cache(P, Fake(0x1000, (2, 2, 4, 2560)), None)

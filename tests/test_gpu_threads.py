"""Calls of the library from several host threads at once, on streams of their own: the same kernels with other sizes of
shared memory. Every call has to be accepted, and gives the bits that it gives alone.

The threads call the C entry points with their arguments made beforehand, so that most of their time is spent inside the
library, where the calls overlap.
"""
import threading

import numpy as np
import pytest
import torch

import oracle.sas_oracle as O
from tests.parity_util import bf16_dev, f32_dev
from tests.test_gpu_kv4 import _filled, _i32, _outputs, _params, _qs

pytestmark = pytest.mark.gpu


def _together(jobs, rounds, copies):
    """Runs each job (call(stream handle) -> status, outputs, what to keep) in `copies` threads, and compares its outputs with
    what it gives alone. Copies of a job write the same bits to the same place."""
    import learned_block_sparse_warp_b200 as sas
    alone = []
    for call, outs, _ in jobs:
        assert call(None) == 0
        torch.cuda.synchronize()
        alone.append([t.clone() for t in outs])
        for t in outs:
            t.zero_()
    start, refused = threading.Barrier(len(jobs) * copies), []
    device = torch.cuda.current_device()

    def work(call, stream):
        torch.cuda.set_device(device)
        handle = stream.cuda_stream
        start.wait()
        refused.append(sum(call(handle) != 0 for _ in range(rounds)))

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(call, torch.cuda.Stream())) for call, _, _ in jobs for _ in range(copies)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert sum(refused) == 0, f"{sum(refused)} of {rounds * len(threads)} calls refused"
    assert sas.sas_get_device_error() == 0
    for want, (_, outs, _) in zip(alone, jobs):
        assert all(torch.equal(a, b) for a, b in zip(want, outs))


@pytest.mark.parametrize("form", ["fused", "split"])
def test_kv4_decode_from_several_threads(form):
    import learned_block_sparse_warp_b200 as sas
    jobs = []
    for Hq, Hkv, n_split in ((8, 1, 1), (2, 2, 1)):  # 8 query heads to a KV head and 1: partials of other sizes
        p = _params(1, Hq, Hkv, 128, 1024, 16)
        st = _filled(p, False, seed=Hq, lens=[1000])
        q, s = _qs(p, seed=Hq)
        qd, sd, cl, out = bf16_dev(q), f32_dev(s), _i32([1000]), _outputs(p, n_split)
        sas.decode_step_kv4(p, qd, st.cache, cl, sd, n_split, out)  # the picks, for the split form
        pc, c = p.c(), sas.sas_kv4_cache(st.dev["k"].data_ptr(), st.dev["v"].data_ptr(), None, 0)
        at = {x: t.data_ptr() for x, t in out.items()}
        head = (pc, qd.data_ptr(), c, cl.data_ptr(), sd.data_ptr(), at["idx"], at["lse_s"])
        if form == "fused":
            def call(stream, args=head + (at["o"], at["lse_o"])):
                return sas.lib.sas_decode_fused_kv4(*args, stream)
            outs = [out[x] for x in ("o", "lse_o")]
        else:
            def call(stream, args=head + (n_split, at["o_part"], at["lse_part"])):
                return sas.lib.sas_decode_kv4(*args, stream)
            outs = [out[x] for x in ("o_part", "lse_part")]
        jobs.append((call, outs, (st, qd, sd, cl, out)))
    _together(jobs, 4000, 4)


def test_scored_select_from_several_threads():
    import learned_block_sparse_warp_b200 as sas
    jobs = []
    for NB, K in ((8, 4), (1024, 16)):
        g = torch.Generator(device="cuda").manual_seed(NB)
        p = _params(1, 1, 1, 128, 64 * NB, K, O.GATE_NONE)
        q = torch.randn((1, 1, 128), device="cuda", generator=g).bfloat16()
        km = torch.randn((1, 1, NB, 128), device="cuda", generator=g).bfloat16()
        cl = _i32([64 * NB - 7])
        s = torch.zeros((1, 1, NB), device="cuda")
        idx = torch.empty((1, 1, K), dtype=torch.int32, device="cuda")
        lse = torch.empty((1, 1), device="cuda")

        def call(stream, args=(p.c(), *(t.data_ptr() for t in (q, km, cl, s, idx, lse)))):
            return sas.lib.sas_decode_select_scored(*args, stream)
        jobs.append((call, [idx, lse], (q, km, cl, s)))
    _together(jobs, 4000, 4)
    assert all(np.isfinite(outs[1].cpu().numpy()).all() for _, outs, _ in jobs)

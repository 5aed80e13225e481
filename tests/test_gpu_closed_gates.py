"""GPU parity on histories whose scores are all -inf, under the softmax gates: every gate is closed, inside and outside
the softmax. Tolerances are those of the same paths with open gates (parity_util)."""
import numpy as np
import pytest
import torch

import oracle.sas_oracle as O
from synth import workloads as W
from tests.parity_util import TOL_L, TOL_O, TOL_REL, assert_idx_equal, bf16_dev, f32_dev, host, max_abs, rel_fro
from tests.test_gpu_decode import _case

pytestmark = pytest.mark.gpu

GATES = [O.GATE_LOG_SOFTMAX, O.GATE_SOFTMAX_OUTSIDE]


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("d", [64, 128])
def test_decode_of_a_masked_history(d, gate):
    import learned_block_sparse_warp_b200 as sas
    B, Hq, Hkv, Lmax, K = 3, 16, 4, 2048, 8
    q, kc, vc, s = _case(B, Hq, Hkv, d, Lmax, seed=7 + d)
    s[0] = -np.inf
    s[1, 2] = -np.inf
    s[2, :, ::2] = -np.inf
    cl = np.array([2048, 777, 65], dtype=np.int32)
    p = sas.Params(batch=B, n_q_heads=Hq, n_kv_heads=Hkv, head_dim=d, seq_len=Lmax, top_k=K, gate_mode=gate)
    args = (bf16_dev(q), bf16_dev(kc), bf16_dev(vc), torch.from_numpy(cl).cuda(), f32_dev(s))
    split, fused = sas.empty_decode_outputs(p, 3), sas.empty_decode_outputs(p, 1)
    sas.decode_step(p, *args, 3, split)
    sas.decode_step_fused(p, *args, fused)
    torch.cuda.synchronize()
    assert sas.sas_get_device_error() == 0
    ref = O.decode(q, kc, vc, cl, s.astype(np.float64), K, gate_mode=gate, n_split=1)
    for out in (split, fused):
        assert_idx_equal(out["idx"].cpu().numpy(), ref["idx"])
        assert np.array_equal(np.isneginf(host(out["lse_s"])), np.isneginf(ref["lse_s"]))
        assert max_abs(host(out["o"]), ref["o"]) < TOL_O
        assert max_abs(host(out["lse_o"]), ref["lse"]) < TOL_L


@pytest.mark.parametrize("ws_min", [False, True])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("d", [64, 128])
def test_training_step_with_masked_histories(d, gate, ws_min):
    """Rows of -inf scores (of a whole head, and of single query blocks) between open ones: o, L, dq, dk, dv and ds."""
    import learned_block_sparse_warp_b200 as sas
    B, Hq, Hkv, N, K = 1, 8, 2, 768, 4
    w = W.custom("masked", batch=B, n_q_heads=Hq, n_kv_heads=Hkv, head_dim=d, seq_len=N, top_k=K, seed=3)
    x = W.prefill_inputs(w, with_do=True)
    s = np.array(x["s"], np.float32)
    s[0, 0] = -np.inf
    s[0, 1, 5] = -np.inf
    s[0, 1, 9, :6] = -np.inf
    p = sas.Params(batch=B, n_q_heads=Hq, n_kv_heads=Hkv, head_dim=d, seq_len=N, top_k=K, gate_mode=gate)
    out = sas.empty_prefill_outputs(p, backward=True)
    if ws_min:  # the dQ pass that recomputes S and dP
        out["ws"] = torch.empty((sas.sas_bwd_workspace_size_min(p),), dtype=torch.uint8, device="cuda")
    sas.prefill_step(p, bf16_dev(x["q"]), bf16_dev(x["k"]), bf16_dev(x["v"]), f32_dev(s), bf16_dev(x["do"]), out, backward=True)
    torch.cuda.synchronize()
    assert sas.sas_get_device_error() == 0
    s64 = s.astype(np.float64)
    idx, _ = O.prefill_select(s64, K)
    assert_idx_equal(out["idx"].cpu().numpy(), idx)
    o, L = O.forward(x["q"], x["k"], x["v"], s64, idx, gate_mode=gate)
    assert max_abs(host(out["o"]), o) < TOL_O and max_abs(host(out["lse_o"]), L) < TOL_L
    dq, dk, dv, ds, _ = O.backward(x["q"], x["k"], x["v"], s64, idx, x["do"], gate_mode=gate)
    for n, ref in (("dq", dq), ("dk", dk), ("dv", dv), ("ds", ds)):
        assert rel_fro(host(out[n]), ref) < TOL_REL, n
    assert torch.all(out["ds"][0, 0] == 0) and torch.all(out["ds"][0, 1, 5] == 0)

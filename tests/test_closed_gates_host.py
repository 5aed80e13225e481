"""The oracle on a history whose scores are all -inf: every softmax gate is closed, as a score mask that leaves no block
asks for, and the row is the current block's alone."""
import numpy as np
import pytest

import oracle.sas_oracle as O


@pytest.mark.parametrize("gate", [O.GATE_LOG_SOFTMAX, O.GATE_SOFTMAX_OUTSIDE])
def test_closed_gates(gate):
    g = np.random.default_rng(1)
    N, d = 192, 8
    q, k, v, do = (g.standard_normal((1, 2, N, d)) for _ in range(4))
    s = np.full((1, 2, 3, 3), -np.inf)
    s[0, 1] = g.standard_normal((3, 3))
    idx, lse = O.prefill_select(s, 2)
    assert idx[0, 0, 2].tolist() == [0, 1] and np.isneginf(lse[0, 0]).all()
    assert np.all(O.log_gate(s[0, 0, 2, :2], [0, 1], gate) == -np.inf)
    o, L = O.forward(q, k, v, s, idx, gate_mode=gate)
    dq, dk, dv, ds, dl = O.backward(q, k, v, s, idx, do, gate_mode=gate)
    assert all(np.isfinite(x).all() for x in (o, L, dq, dk, dv, ds, dl))
    assert np.all(ds[0, 0] == 0) and np.all(dl[0, 0] == 0) and np.abs(ds[0, 1]).max() > 0
    # a gate that is next to closed gives the same
    near = np.where(np.isneginf(s), -200.0, s)
    o2, L2 = O.forward(q, k, v, near, idx, gate_mode=O.GATE_LOGIT)
    if gate == O.GATE_LOG_SOFTMAX:
        assert np.allclose(o[:, 0], o2[:, 0], atol=1e-12) and np.allclose(L[:, 0], L2[:, 0], atol=1e-12)
        r2 = O.backward(q, k, v, near, idx, do, gate_mode=O.GATE_LOGIT)
        assert all(np.allclose(a[:, 0], b[:, 0], atol=1e-12) for a, b in zip((dq, dk, dv), r2))
    else:  # the plain logits' softmax over all tokens, the current block's values alone
        z = q[0, 0, 130] @ k[0, 0, :131].T / np.sqrt(d)
        p = np.exp(z - O.logsumexp(z))
        assert np.allclose(o[0, 0, 130], p[128:] @ v[0, 0, 128:131], atol=1e-12)
        assert np.isclose(L[0, 0, 130], O.logsumexp(z))

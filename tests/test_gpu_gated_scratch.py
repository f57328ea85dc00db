"""Scratch of the gated recurrence's backward call where nobody wants log_decay's gradient."""

import pytest
import torch

from test_gpu_gated import make, problem
from test_gpu_sequence_workspaces import Guarded
from token_level_head_phi_gb300 import binding as mb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("marks", [False, True])
@pytest.mark.parametrize("b,n,d", [(1, 3000, 200), (40, 300, 520)])
def test_without_the_decays_gradient(b, n, d, marks, monkeypatch):
    needs = []
    real = mb._Call.workspace
    monkeypatch.setattr(mb._Call, "workspace", lambda self, given: (needs.append(self.need), real(self, given))[1])
    p = problem(b, n, d, "bf16", "decay", True, True)
    dout = make((b, n, d), 60, "bf16")
    kept = mb.mhla_gated_forward(**p, keep=True)[2] if marks else None
    call = lambda **k: mb.mhla_gated_backward(p["x"], p["gate"], dout, p["log_decay"], p["input_gate"],  # noqa: E731
                                              p["state"], marks=kept, **k)
    want = call()
    got = call(params=False)
    assert got[3] is None and all(torch.equal(got[i], want[i]) for i in (0, 1, 2, 4))
    formed = 0 if marks else 4 * b * -(-n // mb.GATED_MARK) * d  # bytes of the marks alone
    assert needs[1] == formed < needs[0]
    if formed:
        ws = Guarded(formed)
        again = call(params=False, workspace=ws.view)
        ws.check()
        assert all(torch.equal(again[i], want[i]) for i in (0, 1, 2, 4))
        with pytest.raises(mb.MhlaError) as e:
            call(params=False, workspace=torch.empty(formed - 1, dtype=torch.uint8, device="cuda"))
        assert e.value.status == mb.MHLA_ERR_WORKSPACE
    monkeypatch.setattr(mb._Call, "workspace", lambda self, given: (None, 0))  # the entry's own memory
    assert torch.equal(call(params=False)[0], want[0])

"""The decode example notices a layer call that gave up a wait in any block of any step.  The failure is
a status word written by the test after the call; no kernel waits in vain."""
import os
import sys

import pytest
import torch

from conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu

TIMEOUT_FLAG = 1  # what a kernel whose bounded wait expires leaves in the word


@pytest.fixture
def stack(cuda_device):
    import few_token_decode as F
    return F.FewTokenStack(F.make_layers(2, 3, seed=4))


def _failing(monkeypatch, call):
    """moe_forward_few, after whose call number `call` the status word says that a wait expired."""
    import few_token_decode as F
    run, n = F.B.moe_forward_few, [0]

    def few(cfg, *a, **kw):
        run(cfg, *a, **kw)
        if n[0] == call:
            a[-1].view(torch.int32)[0] = TIMEOUT_FLAG
        n[0] += 1

    monkeypatch.setattr(F.B, "moe_forward_few", few)
    return F.B


@pytest.mark.parametrize("call", range(4))
def test_a_failure_in_any_block_of_any_step_is_kept(stack, monkeypatch, call):
    B = _failing(monkeypatch, call)
    for _ in range(3):
        stack.step()
    with pytest.raises(B.MoEError) as e:
        stack.check()
    assert e.value.status == B.MOE_ERR_TIMEOUT and f"block {call % 2}" in str(e.value)


def test_no_failure(stack):
    stack.capture()
    for _ in range(3):
        stack.replay()
    stack.check()
    assert (stack.status == 0).all()

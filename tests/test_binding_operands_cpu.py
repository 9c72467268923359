"""The binding refuses operands whose types or sizes are not the configuration's before any address
reaches the library (no GPU needed: a stand-in library notes its calls, CPU tensors stand for device
ones)."""
import pytest
import torch

from mixture_experts_ffn_gemm_gb300 import binding as B

F32, BF16 = torch.float32, torch.bfloat16


class OnDevice(torch.Tensor):
    """A CPU tensor that says that it is on the GPU."""
    is_cuda = True


def dev(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)


@pytest.fixture
def calls(monkeypatch):
    """Calls that reached the library."""
    made = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: made.append((name, a)) or B.MOE_OK

    monkeypatch.setattr(B, "load_library", lambda: Library())
    return made


T, D = 3, 16


def _join(kind="none", res=F32, **given):
    cfg = B.make_join_config(T, D, BF16, res, kind)
    op = dict(resid=dev(T, D, dtype=res), branch=dev(T, D), post_w=dev(D),
              gate={"none": None, "channel": dev(D), "token": dev(T), "element": dev(T, D)}[kind],
              pre_w=dev(D), resid_out=dev(T, D, dtype=res), normed=dev(T, D))
    op.update(given)
    B.moe_block_join(cfg, *op.values(), stream=0)


@pytest.mark.parametrize("gate", ["none", "channel", "token", "element"])
@pytest.mark.parametrize("res", [F32, BF16])
def test_join_takes_what_the_configuration_says(calls, gate, res):
    _join(gate, res)
    _join(gate, res, post_w=None, pre_w=None, normed=None)
    _join(gate, res, post_w=dev(1, D), pre_w=dev(D, 1))  # d consecutive elements
    assert len(calls) == 3


@pytest.mark.parametrize("name,t", [
    ("resid", dev(T, D)), ("resid_out", dev(T, D)), ("branch", dev(T, D, dtype=F32)),
    ("normed", dev(T, D, dtype=F32)), ("branch", dev(T, D, dtype=torch.float16)),
    ("post_w", dev(D, dtype=F32)), ("pre_w", dev(D, dtype=F32)), ("post_w", dev(D - 1)),
    ("pre_w", dev(D + 1)), ("pre_w", dev(1)), ("resid", dev(T - 1, D, dtype=F32))])
def test_join_refuses_types_and_lengths(calls, name, t):
    with pytest.raises(ValueError, match=name):
        _join(**{name: t})
    assert not calls


@pytest.mark.parametrize("kind,gate", [
    ("channel", dev(T)), ("channel", dev(D, dtype=F32)), ("token", dev(T - 1)), ("token", dev(D)),
    ("token", dev(T, dtype=F32)), ("element", dev(D)), ("element", dev(T, D, dtype=F32)),
    ("element", dev(T - 1, D))])
def test_join_refuses_gates(calls, kind, gate):
    with pytest.raises(ValueError, match="gate"):
        _join(kind, gate=gate)
    assert not calls

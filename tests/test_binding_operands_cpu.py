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


FP8, INT4 = torch.float8_e4m3fn, torch.uint8
D2, E, I, L = 256, 6, 128, 64


def _weights(kind, rows, cols, *lead):
    if kind == INT4:
        return dev(*lead, rows, cols // 2, dtype=INT4), dev(*lead, cols // 32, rows)
    if kind == FP8:
        return dev(*lead, rows, cols, dtype=FP8), dev(*lead, rows // 128, cols // 128, dtype=F32)
    return dev(*lead, rows, cols, dtype=kind), None


def _few_operands(kind, shared=1, latent=0):
    """(configuration, operands of exactly its size by name)"""
    act = F32 if kind == F32 else BF16
    cfg = B.make_config(T=T, d=D2, E=E, k=2, I=I, n_shared=shared, d_latent=latent, act_dtype=act,
                        w_dtype=kind, quant_block=32 if kind == INT4 else 128)
    de = latent or D2
    op = dict(x=dev(T, D2, dtype=act), W_r=dev(E, D2, dtype=F32), b=dev(E, dtype=F32))
    op["W13"], op["W13_scale"] = _weights(kind, 2 * I, de, E)
    op["W2"], op["W2_scale"] = _weights(kind, de, I, E)
    if shared:
        op["Ws13"], op["Ws13_scale"] = _weights(kind, 2 * I, D2)
        op["Ws2"], op["Ws2_scale"] = _weights(kind, D2, I)
    if latent:
        op["W_down"], op["W_up"] = dev(latent, D2, dtype=act), dev(D2, latent, dtype=act)
    op["out"] = dev(T, D2, dtype=act)
    return cfg, {n: op.get(n) for n in B._FEW_OPERANDS}


def _few(cfg, op):
    B.moe_forward_few(cfg, *op.values(), dev(256, dtype=torch.uint8), stream=0)


FORMS = [(kind, shared, 0) for kind in (F32, BF16, FP8, INT4) for shared in (0, 1)]
FORMS += [(kind, shared, L) for kind in (F32, BF16) for shared in (0, 1)]


@pytest.mark.parametrize("kind,shared,latent", FORMS)
def test_few_takes_its_sizes_and_refuses_shorter_ones(calls, kind, shared, latent):
    cfg, op = _few_operands(kind, shared, latent)
    _few(cfg, op)
    assert len(calls) == 1
    for name, t in op.items():
        if t is None:
            continue
        with pytest.raises(ValueError, match=name):
            _few(cfg, {**op, name: dev(t.numel() - 1, dtype=t.dtype)})
    assert len(calls) == 1


def test_few_leaves_what_it_does_not_read(calls):
    cfg, op = _few_operands(BF16, shared=0)
    for name in ("Ws13", "Ws2", "W13_scale", "Ws2_scale", "W_down", "W_up"):
        _few(cfg, {**op, name: dev(1)})
    assert len(calls) == 6


def test_few_sizes_follow_the_configuration(calls):
    cfg, op = _few_operands(BF16)
    cfg.T = T + 1
    with pytest.raises(ValueError, match="x"):
        _few(cfg, op)
    cfg.T = T - 1
    _few(cfg, op)
    cfg.E = E + 1
    with pytest.raises(ValueError, match="W_r"):
        _few(cfg, op)
    assert len(calls) == 1

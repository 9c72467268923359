"""GPU tests of the products grouped by expert (moe_grouped_product) against their formulas in 64 bits.

Tolerance.  An output is an fp32 sum of n products of bf16 values (each product is exact in fp32), rounded
once: half a step, 2^-8 |v| for bf16 and 2^-24 |v| for fp32.  The tensor cores add 16 products to the sum
at a time, aligned to the largest and cut no coarser than 2^-22 of it; n / 16 + 2 such steps (the last
block's zeros and an accumulated sum among them) err by at most (n / 16 + 2) 2^-22 sum |a b|."""
import pytest
import torch

from mixture_experts_ffn_gemm_gb300 import binding as B

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
STEP = {F32: 2.0 ** -24, BF16: 2.0 ** -8}
KINDS = ["forward", "grad_x", "grad_w"]
RAGGED = [0, 1, 127, 128, 129, 0, 300, 16, 33, 0]


def _rows(g, R, width, pad):
    return torch.randn(R, width + pad, generator=g, device="cuda").to(BF16)[:, :width]


def _offsets(counts, first=0):
    o = [first]
    for c in counts:
        o.append(o[-1] + c)
    return o


def _make(kind, counts, N, K, pad=0, behind=0, seed=0):
    """Operands of a call; `behind` rows of the buffers belong to no expert."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    offs = _offsets(counts)
    R, E = offs[-1] + behind, len(counts)
    x = _rows(g, R, K, pad) if kind != "grad_x" else None
    dy = _rows(g, R, N, pad) if kind != "forward" else None
    w = torch.randn(E, N, K, generator=g, device="cuda").to(BF16) if kind != "grad_w" else None
    a, b = {"forward": (x, w), "grad_x": (dy, w), "grad_w": (dy, x)}[kind]
    return offs, R, a, b


def _reference(kind, offs, a, b, N, K):
    """(value, sum of the products' magnitudes, longest sum) of each expert's part"""
    parts = []
    for e in range(len(offs) - 1):
        lo, hi = offs[e], offs[e + 1]
        p = a[lo:hi].double()
        q = (b[lo:hi] if kind == "grad_w" else b[e]).double()
        if kind == "forward":
            parts.append((p @ q.t(), p.abs() @ q.abs().t(), K))
        elif kind == "grad_x":
            parts.append((p @ q, p.abs() @ q.abs(), N))
        else:
            parts.append((p.t() @ q, p.abs().t() @ q.abs(), hi - lo))
    return parts


def _out(kind, R, E, N, K, dtype, pad=0, fill=7.0):
    if kind == "grad_w":
        return torch.full((E, N, K), fill, dtype=dtype, device="cuda")
    width = N if kind == "forward" else K
    return torch.full((R, width + pad), fill, dtype=dtype, device="cuda")[:, :width]


def _config(kind, R, E, N, K, dtype, pad=0, accumulate=False):
    return B.make_product_config(R, E, N, K, kind, dtype, accumulate, K + pad, N + pad)


def _call(kind, offs, R, a, b, N, K, dtype, pad=0, accumulate=False, fill=7.0):
    E = len(offs) - 1
    cfg = _config(kind, R, E, N, K, dtype, pad, accumulate)
    ws = B.alloc_product_workspace(cfg)
    out = _out(kind, R, E, N, K, dtype, pad, fill)
    B.moe_grouped_product(cfg, torch.tensor(offs, dtype=torch.int32, device="cuda"), a, b, out, ws)
    assert B.moe_device_status(ws) == B.MOE_OK
    return out


def _check(kind, out, offs, parts, added=0.0):
    for e, (v, mag, n) in enumerate(parts):
        got = out[e] if kind == "grad_w" else out[offs[e]:offs[e + 1]]
        v, mag = v + added, mag + abs(added)
        tol = STEP[out.dtype] * v.abs() + (n / 16 + 2) * 2.0 ** -22 * mag
        assert ((got.double() - v).abs() <= tol).all(), f"expert {e}"


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("N,K", [(128, 256), (8, 8), (264, 72), (736, 1000), (200, 520), (16, 64)])
def test_ragged_groups(cuda_device, kind, N, K, dtype):
    offs, R, a, b = _make(kind, RAGGED, N, K)
    out = _call(kind, offs, R, a, b, N, K, dtype)
    _check(kind, out, offs, _reference(kind, offs, a, b, N, K))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("counts", [[1], [64], [65], [1000], [0, 0, 5], [256] * 3, [3] * 40, [1024, 1500],
                                    [0, 300, 1, 1000, 64, 777, 0, 513], [129, 128], [255, 257, 1]])
def test_group_sizes(cuda_device, kind, counts):
    N, K = 384, 320
    offs, R, a, b = _make(kind, counts, N, K, seed=1)
    out = _call(kind, offs, R, a, b, N, K, BF16)
    _check(kind, out, offs, _reference(kind, offs, a, b, N, K))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("pad", [8, 64])
def test_rows_inside_wider_buffers(cuda_device, kind, pad):
    N, K = 136, 264
    offs, R, a, b = _make(kind, RAGGED, N, K, pad, seed=2)
    out = _call(kind, offs, R, a, b, N, K, BF16, pad)
    _check(kind, out, offs, _reference(kind, offs, a, b, N, K))
    if kind != "grad_w":  # what lies between the rows stays
        whole = out.as_strided((R, out.shape[1] + pad), (out.shape[1] + pad, 1))
        assert (whole[:, out.shape[1]:] == 7.0).all()


@pytest.mark.parametrize("counts", [[37, 50, 0, 21], [337, 150, 0, 421]])
@pytest.mark.parametrize("kind", KINDS)
def test_rows_of_no_expert_and_values_of_others_do_not_reach_a_result(cuda_device, kind, counts):
    """Rows in front of, between and behind: expert 1's operands and the rows behind the last expert hold
    NaN and infinities; every other expert's results are what they are without."""
    N, K = 72, 200
    offs, R, a, b = _make(kind, counts, N, K, behind=70, seed=3)
    parts = _reference(kind, offs, a, b, N, K)
    a, b = a.clone(), b.clone()
    bad = torch.tensor([float("nan"), float("inf"), -float("inf"), 1e38], device="cuda", dtype=BF16)
    for t in (a, b):
        if t.dim() == 2:
            t[offs[1]:offs[2]] = bad.repeat(t.shape[1] // 4)
            t[offs[-1]:] = bad.repeat(t.shape[1] // 4)
        else:
            t[1] = float("nan")
    out = _call(kind, offs, R, a, b, N, K, F32)
    for e in (0, 2, 3):
        v, mag, n = parts[e]
        got = out[e] if kind == "grad_w" else out[offs[e]:offs[e + 1]]
        assert ((got.double() - v).abs() <= STEP[F32] * v.abs() + (n / 16 + 2) * 2.0 ** -22 * mag).all()
    if kind != "grad_w":
        assert (out[offs[-1]:] == 7.0).all()  # rows of no expert are left
        assert not torch.isfinite(out[offs[1]:offs[2]]).any()
    else:
        assert not torch.isfinite(out[1]).any()
        assert (out[2] == 0).all()


@pytest.mark.parametrize("kind", KINDS)
def test_long_fp32_sums_do_not_drift(cuda_device, kind):
    """16,384 positive terms.  The tensor cores cut a step's sum by at most 2^-23 of it, and always downwards;
    an fp32 output's sum is cut at most 32 times (512 terms; the weight gradient's 64 times, 1024 terms) before
    it is added to the others in fp32 (at most 32 roundings of 2^-24)."""
    long, N, K = 16384, 24, 40
    if kind == "grad_w":
        counts = [long, 100]
    elif kind == "forward":
        counts, K = [70, 3], long
    else:
        counts, N = [70, 3], long
    offs, R, a, b = _make(kind, counts, N, K, seed=10)
    a, b = a.abs(), b.abs()
    cuts = 64 if kind == "grad_w" else 32
    out = _call(kind, offs, R, a, b, N, K, F32)
    for e, (v, _, n) in enumerate(_reference(kind, offs, a, b, N, K)):
        got = out[e] if kind == "grad_w" else out[offs[e]:offs[e + 1]]
        assert ((got.double() - v).abs() <= (cuts * 2.0 ** -23 + 33 * 2.0 ** -24) * v).all()


def test_accumulated_weight_gradient(cuda_device):
    N, K = 136, 264
    offs, R, a, b = _make("grad_w", RAGGED, N, K, seed=4)
    out = _call("grad_w", offs, R, a, b, N, K, F32, accumulate=True, fill=2.5)
    _check("grad_w", out, offs, _reference("grad_w", offs, a, b, N, K), added=2.5)


def test_no_rows(cuda_device):
    offs = torch.zeros(4, dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    x, dy = (torch.empty(0, n, dtype=BF16, device="cuda") for n in (64, 16))
    w = torch.ones(3, 16, 64, dtype=BF16, device="cuda")
    B.moe_grouped_product(B.make_product_config(0, 3, 16, 64), offs, x, w, dy, ws)
    for accumulate, want in ((True, 3.0), (False, 0.0)):
        dw = torch.full((3, 16, 64), 3.0, device="cuda")
        cfg = B.make_product_config(0, 3, 16, 64, "grad_w", F32, accumulate)
        B.moe_grouped_product(cfg, offs, dy, x, dw, ws)
        assert (dw == want).all()
    # rows that no expert takes: a gradient of zeros as well
    x, dy = (torch.ones(50, n, dtype=BF16, device="cuda") for n in (64, 16))
    dw = torch.full((3, 16, 64), 3.0, device="cuda")
    B.moe_grouped_product(B.make_product_config(50, 3, 16, 64, "grad_w", F32), offs, dy, x, dw, ws)
    assert (dw == 0).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bad", [[0, 40, 30, 90], [0, 40, 60, 9999], [-5, 40, 60, 90],
                                 [0, -(2 ** 31), 2 ** 31 - 1, 90]])
def test_bad_offsets_stay_inside_the_buffers(cuda_device, kind, bad):
    N, K, R = 64, 128, 90
    _, _, a, b = _make(kind, [30, 30, 30], N, K, seed=5)
    cfg = _config(kind, R, 3, N, K, F32)
    ws = B.alloc_product_workspace(cfg)
    out = _out(kind, R, 3, N, K, F32)
    B.moe_grouped_product(cfg, torch.tensor(bad, dtype=torch.int32, device="cuda"), a, b, out, ws)
    assert B.moe_device_status(ws) == B.MOE_ERR_DEVICE_CHECK
    assert B.moe_device_status(ws) == B.MOE_ERR_DEVICE_CHECK  # it stays until it is reset
    B.moe_reset_device_status(ws)
    assert B.moe_device_status(ws) == B.MOE_OK


@pytest.mark.parametrize("counts", [RAGGED, [0, 300, 1, 1000, 64, 777, 0, 513]])
@pytest.mark.parametrize("kind", KINDS)
def test_equal_calls_give_equal_bits_in_a_graph_and_on_another_stream(cuda_device, kind, counts):
    N, K = 264, 520
    offs, R, a, b = _make(kind, counts, N, K, seed=6)
    first = _call(kind, offs, R, a, b, N, K, BF16)
    E = len(offs) - 1
    cfg = _config(kind, R, E, N, K, BF16)
    ws = B.alloc_product_workspace(cfg)
    o = torch.tensor(offs, dtype=torch.int32, device="cuda")
    second, third = (_out(kind, R, E, N, K, BF16) for _ in range(2))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    B.moe_grouped_product(cfg, o, a, b, second, ws, stream=s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.moe_grouped_product(cfg, o, a, b, third, ws)
    for _ in range(2):
        third.fill_(0)
        graph.replay()
    torch.cuda.synchronize()
    for e in range(E):
        rows = slice(e, e + 1) if kind == "grad_w" else slice(offs[e], offs[e + 1])
        assert torch.equal(first[rows], second[rows]) and torch.equal(first[rows], third[rows])


def test_gradients_of_a_loss_by_differences(cuda_device):
    """L = sum c * y^2 / 2 for y = x W_e^T: dy = c y; dx and dW against central differences of L in 64 bits
    along random directions (L is a polynomial of degree two along a line: the difference is exact)."""
    N, K, counts = 40, 56, [9, 0, 30, 17]
    offs, R, x, w = _make("forward", counts, N, K, seed=7)
    c = torch.rand(R, N, device="cuda", generator=torch.Generator(device="cuda").manual_seed(8))
    y = _call("forward", offs, R, x, w, N, K, F32)
    dy = (c * y).to(BF16)
    dx = _call("grad_x", offs, R, dy, w, N, K, F32)
    dw = _call("grad_w", offs, R, dy, x, N, K, F32)

    def loss(xd, wd):
        total = 0.0
        for e in range(len(counts)):
            s = slice(offs[e], offs[e + 1])
            total = total + (c[s].double() * (xd[s] @ wd[e].t()) ** 2).sum() / 2
        return total

    g = torch.Generator(device="cuda").manual_seed(9)
    xd, wd = x.double(), w.double()
    for grad, which in ((dx, 0), (dw, 1)):
        base = (xd, wd)[which]
        for _ in range(4):
            v = torch.randn(base.shape, generator=g, device="cuda", dtype=torch.float64)
            h = 1e-3
            p, m = ((xd + s * h * v, wd) if which == 0 else (xd, wd + s * h * v) for s in (1, -1))
            want = (loss(*p) - loss(*m)) / (2 * h)
            got = (grad.double() * v).sum()
            # dy is rounded to bf16: half a step of each of its values reaches the gradients
            ay = (2.0 ** -8) * dy.double().abs()
            slack = 0.0
            for e in range(len(counts)):
                s = slice(offs[e], offs[e + 1])
                other = wd[e].abs() if which == 0 else xd[s].abs()
                part = ay[s] @ other if which == 0 else ay[s].t() @ other
                slack = slack + (part * (v[s] if which == 0 else v[e]).abs()).sum()
            assert (got - want).abs() <= slack + 1e-5 * (grad.double() * v).abs().sum()


def test_plain_and_pitched_calls_take_the_quick_check_and_others_are_refused(cuda_device, monkeypatch):
    """The module beside the library takes every accepted operand; what it leaves is refused with a reason."""
    N, K, pad = 64, 128, 8
    offs, R, a, b = _make("forward", [5, 9], N, K, pad, seed=11)
    want = _call("forward", offs, R, a, b, N, K, F32, pad)
    slow = B._addresses
    monkeypatch.setattr(B, "_addresses", None)
    assert torch.equal(_call("forward", offs, R, a, b, N, K, F32, pad)[:, :], want)
    assert torch.equal(_call("forward", offs, R, a.contiguous(), b, N, K, F32), want)
    monkeypatch.setattr(B, "_addresses", slow)
    o = torch.tensor(offs, dtype=torch.int32, device="cuda")
    out = _out("forward", R, 2, N, K, F32)
    cfg = _config("forward", R, 2, N, K, F32)
    ws = B.alloc_product_workspace(cfg)
    good = dict(offsets=o, a=a.contiguous(), b=b, out=out)
    for name, bad in (("offsets", o[:2]), ("offsets", o.long()), ("a", a), ("a", a.float()), ("b", b[:1]),
                      ("b", b.cpu()), ("out", out.to(BF16)), ("out", out.t())):
        with pytest.raises(ValueError, match=name):
            B.moe_grouped_product(cfg, *{**good, name: bad}.values(), ws)
    with pytest.raises(ValueError, match="ws"):
        B.moe_grouped_product(cfg, *good.values(), ws.cpu())
    with pytest.raises(B.MoEError):
        B.moe_grouped_product(cfg, *good.values(), ws[:128])
    B.moe_grouped_product(cfg, *good.values(), ws)
    assert torch.equal(out, want)

"""GPU tests of the block join (moe_block_join) against its formula in 64 bits.

Tolerances.  Outputs are rounded once: half a step, 2^-8 |v| for bf16 and 2^-24 |v| for fp32.  Before
it everything is fp32: r' is a sum of two products of at most six rounded factors, 8 x 2^-24 of
|a r| + |b g v|, the norm's sum of d <= 2^15 squares (no cancellation) stays within 2^-24 sqrt(d) =
2^-16 relative, halved by the root, times 2; the sigmoid's exponential is good to 2^-21.  normed
carries r's error through its factor."""
import pytest
import torch

from mixture_experts_ffn_gemm_gb300 import binding as B

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
STEP = {F32: 2.0 ** -24, BF16: 2.0 ** -8}
EPS = 1e-6


def _rows(g, T, d, pad, dtype, std=1.0, offset=0):
    buf = torch.randn(T * (d + pad) + offset, generator=g, device="cuda") * std
    return buf.to(dtype)[offset:].view(T, d + pad)[:, :d]


def _make(T, d, act, res, gate, sigmoid, post, pre, pad=0, offset=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(resid=_rows(g, T, d, pad, res, 2.0, offset), branch=_rows(g, T, d, pad, act, 0.7, offset))
    st["post_w"] = (torch.rand(d, generator=g, device="cuda") + 0.5).to(act) if post else None
    st["pre_w"] = (torch.rand(d, generator=g, device="cuda") + 0.5).to(act) if pre else None
    st["gate"] = {"none": lambda: None, "element": lambda: _rows(g, T, d, pad, act, 1.0, offset),
                  "channel": lambda: torch.randn(d, generator=g, device="cuda").to(act),
                  "token": lambda: torch.randn(T, generator=g, device="cuda").to(act)}[gate]()
    st["resid_out"] = _rows(g, T, d, pad, res, 1.0, offset)
    st["normed"] = _rows(g, T, d, pad, act, 1.0, offset) if pre else None
    cfg = B.make_join_config(T, d, act, res, gate, sigmoid, 0.9, 0.31, EPS, d + pad, d + pad,
                             d + pad, d + pad, d + pad)
    return cfg, st


def _reference(st, gate, sigmoid):
    """(r', n, magnitude of the terms of r')"""
    v = st["branch"].double()
    d = v.shape[1]
    if st["post_w"] is not None:
        v = v / torch.sqrt(v.pow(2).sum(1, keepdim=True) / d + EPS) * st["post_w"].double()
    if st["gate"] is not None:
        g = st["gate"].double()
        g = torch.sigmoid(g) if sigmoid else g
        v = v * (g[:, None] if gate == "token" else g)
    a, b = torch.tensor([0.9, 0.31], dtype=torch.float32).double().tolist()
    r = a * st["resid"].double()
    mag = r.abs() + (b * v).abs()
    r = r + b * v
    n = None
    if st["pre_w"] is not None:
        f = st["pre_w"].double() / torch.sqrt(r.pow(2).sum(1, keepdim=True) / d + EPS)
        n = (r * f, f.abs())
    return r, n, mag


def _check(cfg, st, ref):
    r, n, mag = ref
    between = (8 * 2.0 ** -24 + 2.0 ** -16 + 2.0 ** -21) * mag
    err = (st["resid_out"].double() - r).abs()
    assert (err <= STEP[st["resid_out"].dtype] * r.abs() + between).all()
    if n is not None:
        err = (st["normed"].double() - n[0]).abs()
        assert (err <= (STEP[st["normed"].dtype] + 2.0 ** -15) * n[0].abs() + between * n[1]).all()


def _run(cfg, st, stream=None):
    B.moe_block_join(cfg, st["resid"], st["branch"], st["post_w"], st["gate"], st["pre_w"],
                     st["resid_out"], st["normed"], stream=stream)


TYPES = [(F32, F32), (BF16, BF16), (BF16, F32)]


@pytest.mark.parametrize("gate", ["none", "channel", "token", "element"])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("act,res", TYPES)
def test_forms(cuda_device, act, res, gate, sigmoid, post, pre):
    cfg, st = _make(37, 520, act, res, gate, sigmoid, post, pre, pad=8, seed=1)
    ref = _reference(st, gate, sigmoid)
    _run(cfg, st)
    _check(cfg, st, ref)


@pytest.mark.parametrize("act,res", TYPES)
@pytest.mark.parametrize("T,d,pad,offset", [
    (1, 1, 0, 0), (1, 7, 0, 0), (3, 8, 0, 0), (5, 33, 1, 0), (2, 255, 0, 0), (700, 64, 0, 0),
    (1, 7168, 0, 0), (2, 7168, 0, 1), (2, 7168, 3, 0), (1500, 7168, 0, 0), (3, 8192, 0, 0),
    (2, 8200, 0, 0), (2, 16384, 8, 8), (3, 16392, 0, 0), (2, 32767, 0, 0), (2, 32768, 0, 0),
    (1217, 1001, 0, 0), (3000, 2056, 8, 0), (40000, 24, 0, 0)])
def test_sizes_pitches_and_alignment(cuda_device, act, res, T, d, pad, offset):
    cfg, st = _make(T, d, act, res, "element", False, True, True, pad, offset, seed=2)
    keep = [t.clone() for t in (st["resid"], st["branch"], st["gate"])]
    ref = _reference(st, "element", False)
    _run(cfg, st)
    _check(cfg, st, ref)
    assert all(torch.equal(a, b) for a, b in zip(keep, (st["resid"], st["branch"], st["gate"])))


@pytest.mark.parametrize("d,pad", [(1000, 0), (1001, 7), (7168, 0), (20000, 0)])
def test_in_place_and_between_rows(cuda_device, d, pad):
    """resid_out = resid and normed = branch; what lies between the rows stays."""
    cfg, st = _make(50, d, BF16, BF16, "channel", True, True, True, pad, seed=3)
    ref = _reference(st, "channel", True)
    bufs = []
    for src in ("resid", "branch"):
        buf = torch.full((50, d + pad), 7.0, dtype=BF16, device="cuda")
        buf[:, :d] = st[src]
        st[src] = buf[:, :d]
        bufs.append(buf)
    st["resid_out"], st["normed"] = st["resid"], st["branch"]
    _run(cfg, st)
    _check(cfg, st, ref)
    assert all((b[:, d:] == 7.0).all() for b in bufs)


def test_rows_are_independent(cuda_device):
    """NaN, infinities and zeros in some rows leave the others' bits; a zero row norms to zero."""
    cfg, st = _make(9, 1024, BF16, BF16, "token", False, True, True, seed=4)
    _run(cfg, st)
    clean = st["resid_out"].clone(), st["normed"].clone()
    st["branch"][2] = float("nan")
    st["resid"][5] = float("inf")
    st["branch"][7] = 0.0
    st["resid"][7] = 0.0
    _run(cfg, st)
    keep = torch.tensor([0, 1, 3, 4, 6, 8], device="cuda")
    assert torch.equal(st["resid_out"][keep], clean[0][keep])
    assert torch.equal(st["normed"][keep], clean[1][keep])
    assert st["resid_out"][2].isnan().all() and (st["normed"][7] == 0).all()
    assert (st["resid_out"][5] == float("inf")).all()


def test_offsets_past_32_bits(cuda_device):
    """The last rows of 2^31 + elements."""
    T, d = 300000, 7200
    cfg, st = _make(1, d, BF16, BF16, "none", False, True, True, seed=5)
    big = torch.zeros(T, d, dtype=BF16, device="cuda")
    big[-1] = st["resid"][0]
    br = torch.zeros(T, d, dtype=BF16, device="cuda")
    br[-1] = st["branch"][0]
    ref = _reference(st, "none", False)
    cfg = B.make_join_config(T, d, resid_scale=0.9, branch_scale=0.31, rms_eps=EPS)
    B.moe_block_join(cfg, big, br, st["post_w"], None, st["pre_w"], big, br)
    st["resid_out"], st["normed"] = big[-1:], br[-1:]
    _check(cfg, st, ref)
    assert (big[:-1] == 0).all()


def test_streams_graph_and_equal_bits(cuda_device):
    cfg, st = _make(333, 2048, BF16, F32, "element", True, True, True, seed=6)
    ref = _reference(st, "element", True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    _run(cfg, st, stream=side)
    side.synchronize()
    _check(cfg, st, ref)
    first = st["normed"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _run(cfg, st)
    st["normed"].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(st["normed"], first)


def test_zero_rows(cuda_device):
    cfg = B.make_join_config(0, 64)
    e = torch.empty(0, 64, dtype=BF16, device="cuda")
    B.moe_block_join(cfg, e, e, None, None, None, e, None)

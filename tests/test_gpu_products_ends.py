"""GPU tests of the products grouped by expert and the microscaled operators at the ends that their documents
allow: factors whose product leaves fp32, weight gradients over millions of rows, rows behind the last expert; and waits that
run out.

Tolerances as in test_gpu_micro.py: half a step of the output's type, 2^-22 sum |a w| for each MMA step of the
sum, two roundings of 2^-24 for the factors; below the smallest normal number half a step is 2^-150 in fp32
(two roundings: 2^-149) and 2^-134 in bf16."""
import pytest
import torch

from mixture_experts_ffn_gemm_gb300 import binding as B
import test_gpu_grouped as grouped
from test_gpu_micro import E4M3, LUT, _operand, gpu, offsets_of, pack, quantize64, scale_index, unpack

pytestmark = pytest.mark.gpu

F32, BF16, U8, I32 = torch.float32, torch.bfloat16, torch.uint8, torch.int32
STEP = {F32: 2.0 ** -24, BF16: 2.0 ** -8}
TINY = {F32: 2.0 ** -149, BF16: 2.0 ** -134 + 2.0 ** -149}
MOST = {F32: 2.0 ** 128 * (1 - 2.0 ** -25), BF16: 2.0 ** 128 * (1 - 2.0 ** -9)}  # rounds to infinity from here on


def _nv_operand(g, offs, K, low, high, zero_rows=()):
    """Codes of positive numbers with scale bytes of low..high, zeros in some rows; values in float64."""
    R = offs[-1]
    code = torch.randint(0, 8, (R, K), generator=g)
    byte = torch.randint(low, high + 1, (R, K // 16), generator=g)
    for r in zero_rows:
        code[r] = 0
    val = (LUT[code].view(R, -1, 16) * torch.tensor(E4M3, dtype=torch.float64)[byte][..., None]).view(R, K)
    scales = torch.full(((R // 128 + len(offs) - 1) * ((K + 63) // 64) * 512,), 255, dtype=U8)
    scales[scale_index(offs, K, "nv").view(-1)] = byte.to(U8).view(-1)
    return pack(code).cuda(), scales.cuda(), val.cuda()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("low,high", [(110, 126), (1, 30)])
@pytest.mark.parametrize("ga,gw", [(4.1e-22, 3.7e-23), (1e-23, 1e-23), (1e22, 1e22), (2.0 ** 100, 2.0 ** -100),
                                   (2.0 ** -100, 2.0 ** 100), (1e30, 1e-30), (2.0 ** -100, 1.0), (3e-24, 1e18)])
def test_factors_whose_product_leaves_fp32(cuda_device, ga, gw, low, high, dtype):
    """Each factor lies in its range, the result in fp32 or not: the value of the formula in either case, and
    zero for rows of zeros."""
    K, N, counts = 1024, 136, [5, 0, 140]
    offs, E = offsets_of(counts), len(counts)
    g = torch.Generator().manual_seed(1)
    a, sa, va = _nv_operand(g, offs, K, low, high, zero_rows=(2, 77))
    w, sw, vw = _nv_operand(g, [e * N for e in range(E + 1)], K, low, high)
    fa = torch.tensor([ga], device="cuda")
    fw = torch.tensor([gw, 1.0, gw * 0.75], device="cuda")
    cfg = B.make_micro_product_config(offs[-1], E, N, K, "nv", dtype)
    ws = B.alloc_micro_product_workspace(cfg)
    out = torch.full((offs[-1], N), 7.0, dtype=dtype, device="cuda")
    B.moe_micro_product(cfg, gpu(offs), a, sa, fa, w, sw, fw, out, ws)
    assert B.moe_device_status(ws) == B.MOE_OK
    for e in range(E):
        s = slice(offs[e], offs[e + 1])
        f = float(fa.double()) * float(fw[e].double())
        v = f * (va[s] @ vw[e * N:(e + 1) * N].t())  # all terms are positive: the sum of magnitudes too
        tol = (STEP[dtype] + (K / 64 + 3) * 2.0 ** -22) * v + TINY[dtype]
        got = out[s].double()
        assert (got[v == 0] == 0).all()
        over, within = v - tol >= MOST[dtype], v + tol < MOST[dtype]
        assert torch.isinf(got[over]).all()
        assert ((got - v).abs() <= tol)[within].all(), f"expert {e}"


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("ga,gw", [(1e22, 1e22), (2.0 ** 100, 2.0 ** 100), (2.0 ** 100, 2.0 ** -100),
                                   (2.0 ** -100, 2.0 ** 100), (1e-23, 1e-23)])
def test_swiglu_with_factors_whose_product_leaves_fp32(cuda_device, ga, gw, dtype):
    """Rows of zeros stay zeros; where the factors' product is a plain number, so is every output."""
    K, N, counts = 256, 128, [5, 0, 140]
    offs, E = offsets_of(counts), len(counts)
    g = torch.Generator().manual_seed(2)
    a, sa, va = _nv_operand(g, offs, K, 30, 60, zero_rows=(2, 77))
    w, sw, vw = _nv_operand(g, [e * 2 * N for e in range(E + 1)], K, 30, 60)
    fa, fw = torch.tensor([ga], device="cuda"), torch.full((E,), gw, device="cuda")
    cfg = B.make_micro_product_config(offs[-1], E, N, K, "nv", dtype, swiglu=True)
    ws = B.alloc_micro_product_workspace(cfg)
    out = torch.full((offs[-1], N), 7.0, dtype=dtype, device="cuda")
    B.moe_micro_product(cfg, gpu(offs), a, sa, fa, w, sw, fw, out, ws)
    assert B.moe_device_status(ws) == B.MOE_OK
    assert (out[[2, 77]] == 0).all()
    if ga * gw == 1.0:
        for e in range(E):
            s = slice(offs[e], offs[e + 1])
            y = va[s] @ vw[e * 2 * N:(e + 1) * 2 * N].t()
            gate, up = y[:, :N], y[:, N:]
            v = gate * torch.sigmoid(gate) * up
            # 1.1 |u| of the gate's error (sigma is at least 1/2 here), |silu| of the other half's, the exponential's
            tol = (STEP[dtype] + 3.3 * (K / 64 + 3) * 2.0 ** -22 + 2.0 ** -20) * v
            assert ((out[s].double() - v).abs() <= tol).all(), f"expert {e}"
    elif ga * gw < 1.0:
        assert (out == 0).all()  # of the order of 1e-80


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows", [1 << 21, (1 << 23) - 5])
def test_weight_gradients_of_long_groups_do_not_drift(cuda_device, rows, dtype):
    """Positive terms.  A step cuts the sum by at most 2^-23 of it, always downwards, and a bf16 output's sum is
    cut at most 1024 times (an fp32 one's 64 times) before it is added to the others in fp32: 2^-13 (2^-17) of the
    sum.  rows / 16384 (rows / 1024) such additions round by 2^-24 of it each."""
    N, K, counts = 24, 40, [rows, 100, 0, 37]
    offs, R, a, b = grouped._make("grad_w", counts, N, K, seed=20)
    a.abs_(), b.abs_()
    out = grouped._call("grad_w", offs, R, a, b, N, K, dtype)
    steps = 1024 if dtype is BF16 else 64
    for e in range(len(counts)):
        v = torch.zeros(N, K, dtype=torch.float64, device="cuda")
        for lo in range(offs[e], offs[e + 1], 1 << 20):
            s = slice(lo, min(lo + (1 << 20), offs[e + 1]))
            v += a[s].double().t() @ b[s].double()
        tol = STEP[dtype] + steps * 2.0 ** -23 + (counts[e] / (16 * steps) + 2) * 2.0 ** -24
        assert ((out[e].double() - v).abs() <= tol * v).all(), f"expert {e}"


@pytest.mark.parametrize("counts", [[0, 1, 127, 128, 129, 0, 300, 16, 33, 0], [16384, 16385, 0, 16383, 32768 + 17, 5],
                                    [70000, 3, 64, 0, 60000]])
@pytest.mark.parametrize("N,K", [(264, 72), (200, 520), (8, 8), (736, 1000)])
def test_weight_gradients_of_calls_with_many_rows(cuda_device, counts, N, K):
    """Ragged groups in a call of more than 2^17 rows, most of them of no expert in the first case."""
    behind = (1 << 17) + 8 - sum(counts) if sum(counts) <= 1 << 17 else 0
    offs, R, a, b = grouped._make("grad_w", counts, N, K, behind=behind, seed=21)
    assert R > 1 << 17
    a[offs[-1]:], b[offs[-1]:] = float("nan"), float("inf")
    out = grouped._call("grad_w", offs, R, a, b, N, K, BF16)
    grouped._check("grad_w", out, offs, grouped._reference("grad_w", offs, a, b, N, K))
    again = grouped._call("grad_w", offs, R, a, b, N, K, BF16)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("counts,behind", [([3, 0, 140], 200), ([1], 1), ([0, 0], 5), ([128, 128], 7), ([2, 700], 3000)])
def test_rows_behind_the_last_expert_are_not_quantised(cuda_device, fmt, dtype, counts, behind):
    """A padded buffer without destinations: the groups' rows as ever; the others' codes and scales stay, and the
    status too."""
    K, offs = 320, offsets_of(counts)
    R, E = offs[-1], len(counts)
    x = torch.randn(R + behind, K, generator=torch.Generator().manual_seed(30)).to(dtype)
    x[R:] = float("nan")
    cfg = B.make_micro_config(R + behind, K, fmt, groups=E, dtype=dtype)
    codes, scales = B.alloc_micro(cfg)
    codes.fill_(0xEE)
    scales.fill_(0xEE)
    ws = B.alloc_micro_workspace(cfg)
    B.moe_micro_quantize(cfg, x.cuda(), None, gpu(offs), None, codes, scales, ws)
    assert B.moe_device_status(ws) == B.MOE_OK
    code, byte = quantize64(x[:R], fmt)
    assert torch.equal(unpack(codes)[:R], code) and (codes[R:] == 0xEE).all()
    got = scales.cpu()
    idx = scale_index(offs, K, fmt)
    assert torch.equal(got[idx.view(-1)].long(), byte.view(-1))
    # columns behind K in a row's last tile (of 64 channels with nv, which K fills, of 128 with mx) are free;
    # everything else is as it was
    written = torch.zeros_like(got, dtype=torch.bool)
    tile = 64 if fmt == "nv" else 128
    whole = scale_index(offs, (K + tile - 1) // tile * tile, fmt)
    written[whole.view(-1)] = True
    assert (got[~written] == 0xEE).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_a_padded_chain_of_products_raises_nothing(cuda_device, fmt):
    """Product, quantisation, product, back in a buffer with room for more rows than the experts have: the status
    stays clear, rows behind keep what they held, and the others are what they are without the room."""
    counts, N, K = [70, 0, 33], 128, 192
    offs, E = offsets_of(counts), len(counts)
    w1, w2 = (torch.randn(E, N, k, generator=torch.Generator().manual_seed(31)).to(BF16).cuda() for k in (K, N))
    x = torch.randn(offs[-1], K, generator=torch.Generator().manual_seed(32)).to(BF16).cuda()
    results = []
    for room in (0, 77):
        R = offs[-1] + room
        xp = torch.full((R, K), float("nan"), dtype=BF16, device="cuda")
        xp[:offs[-1]] = x
        h, y, back = (torch.full((R, N), 7.0, dtype=t, device="cuda") for t in (BF16, F32, F32))
        cfg = B.make_micro_config(R, N, fmt, groups=E)
        cw = B.make_micro_config(E * N, N, fmt, groups=E)
        ws = B.alloc_micro_workspace(cfg)
        hq, wq = B.alloc_micro(cfg), B.alloc_micro(cw)
        B.moe_micro_quantize(cw, w2.view(E * N, N), None, None, None, *wq, ws)
        B.moe_grouped_product(B.make_product_config(R, E, N, K), gpu(offs), xp, w1, h, ws)
        B.moe_micro_quantize(cfg, h, None, gpu(offs), None, *hq, ws)
        B.moe_micro_product(B.make_micro_product_config(R, E, N, N, fmt, F32), gpu(offs), *hq, None, *wq, None, y, ws)
        B.moe_micro_dequantize(B.make_micro_config(R, N, fmt, groups=E, dtype=F32), *hq, gpu(offs), None, back, ws)
        assert B.moe_device_status(ws) == B.MOE_OK
        assert all((t[offs[-1]:] == 7.0).all() for t in (h, y, back))
        results.append([t[:offs[-1]].clone() for t in (h, y, back)])
    for a, b in zip(*results):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", grouped.KINDS)
def test_an_expired_wait_is_reported_and_the_next_call_is_right(cuda_device, kind, dtype):
    """The failure path without a GPU fault: the test flag withholds copies, the waits for them (20 ms) run out,
    the kernel returns with MOE_ERR_TIMEOUT in the status and the context stays usable."""
    N, K, counts = 264, 520, [0, 1, 127, 128, 129, 0, 300, 16, 33, 0]
    offs, R, a, b = grouped._make(kind, counts, N, K, seed=40)
    cfg = grouped._config(kind, R, len(counts), N, K, dtype)
    cfg.flags |= B.MOE_PRODUCT_TEST_STALL
    ws = B.alloc_product_workspace(cfg)
    out = grouped._out(kind, R, len(counts), N, K, dtype)
    B.moe_grouped_product(cfg, gpu(offs), a, b, out, ws)
    assert B.moe_device_status(ws) == B.MOE_ERR_TIMEOUT
    out = grouped._call(kind, offs, R, a, b, N, K, dtype)
    grouped._check(kind, out, offs, grouped._reference(kind, offs, a, b, N, K))


@pytest.mark.parametrize("width,rows,dtype", [(8192, 393216, BF16), (8192, 393216, F32), (16384, 129024, BF16)])
def test_a_run_longer_than_the_waits_limit_passes(cuda_device, width, rows, dtype):
    """A group whose blocks are all whole, several times the limit long (10 ms under this flag), and behind it
    one whose last block is cleared: the warp that clears it waits from the start, and no wait runs out."""
    counts = [rows, 7]
    offs, R = offsets_of(counts), sum(counts)
    g = torch.Generator(device="cuda").manual_seed(41)
    a, b = (torch.empty(R, width, dtype=BF16, device="cuda").normal_(generator=g) for _ in range(2))
    cfg = grouped._config("grad_w", R, 2, width, width, dtype)
    cfg.flags |= B.MOE_PRODUCT_TEST_SHORT_WAITS
    ws = B.alloc_product_workspace(cfg)
    out = torch.empty(2, width, width, dtype=dtype, device="cuda")
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    B.moe_grouped_product(cfg, gpu(offs), a, b, out, ws)
    end.record()
    assert B.moe_device_status(ws) == B.MOE_OK
    assert start.elapsed_time(end) > 20.0  # else it shows nothing
    for e, n in enumerate(counts):
        v, mag = (torch.zeros(64, 64, dtype=torch.float64, device="cuda") for _ in range(2))
        for lo in range(offs[e], offs[e + 1], 1 << 16):
            p, q = (t[lo:min(lo + (1 << 16), offs[e + 1]), -64:].double() for t in (a, b))
            v += p.t() @ q
            mag += p.abs().t() @ q.abs()
        tol = STEP[dtype] * v.abs() + (n / 16 + 2) * 2.0 ** -22 * mag
        assert ((out[e, -64:, -64:].double() - v).abs() <= tol).all()


def test_calls_without_the_quick_check_give_the_same(cuda_device, monkeypatch):
    """Where the module of the quick check could not be built, the binding checks and calls by itself."""
    N, K, counts, pad = 72, 192, [5, 0, 140], 8
    offs, E = offsets_of(counts), len(counts)
    offs, R, a, b = grouped._make("forward", counts, N, K, pad, seed=50)

    def run():
        y = grouped._call("forward", offs, R, a, b, N, K, F32, pad)
        cfg = B.make_micro_config(R, K, "nv", groups=E, ld=K + pad)
        cw = B.make_micro_config(E * N, K, "nv", groups=E)
        q, w, ws = B.alloc_micro(cfg), B.alloc_micro(cw), B.alloc_micro_workspace(cfg)
        f = torch.tensor([0.01], device="cuda")
        out, back = (torch.zeros(R, n, device="cuda") for n in (N, K))
        B.moe_micro_quantize(cfg, a, None, gpu(offs), f, *q, ws)
        B.moe_micro_quantize(cw, b.view(E * N, K), None, None, f, *w, ws)
        B.moe_micro_product(B.make_micro_product_config(R, E, N, K, "nv", F32), gpu(offs), *q, f, *w, f.expand(E)
                            .contiguous(), out, ws)
        B.moe_micro_dequantize(B.make_micro_config(R, K, "nv", groups=E, dtype=F32), *q, gpu(offs), f, back, ws)
        assert B.moe_device_status(ws) == B.MOE_OK
        return y, *q, out, back

    want = run()
    monkeypatch.setattr(B, "_operands_module", lambda: None)
    for one, other in zip(want, run()):
        assert torch.equal(one, other)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [0.02, 1.0, 1e4, 1e12])
def test_swiglu_of_large_gates_of_either_sign(cuda_device, scale, dtype):
    """Gates from a hundredth to far beyond the exponential's range, both signs: SiLU is the gate, or zero."""
    K, N, counts = 256, 128, [5, 0, 140]
    offs, E = offsets_of(counts), len(counts)
    g = torch.Generator().manual_seed(60)
    a, sa, va = _operand(g, offs, K, "nv")
    w, sw, vw = _operand(g, [e * 2 * N for e in range(E + 1)], K, "nv")
    fa, fw = torch.tensor([scale], device="cuda"), torch.full((E,), 2.0 ** -10, device="cuda")
    cfg = B.make_micro_product_config(offs[-1], E, N, K, "nv", dtype, swiglu=True)
    ws = B.alloc_micro_product_workspace(cfg)
    out = torch.full((offs[-1], N), 7.0, dtype=dtype, device="cuda")
    B.moe_micro_product(cfg, gpu(offs), a, sa, fa, w, sw, fw, out, ws)
    assert B.moe_device_status(ws) == B.MOE_OK
    f = float(fa.double()) * 2.0 ** -10
    for e in range(E):
        s = slice(offs[e], offs[e + 1])
        we = vw[e * 2 * N:(e + 1) * 2 * N]
        y = f * (va[s] @ we.t())
        err = ((K / 64 + 3) * 2.0 ** -22) * f * (va[s].abs() @ we.abs().t())
        gate, up, eg, eu = y[:, :N], y[:, N:], err[:, :N], err[:, N:]
        act = gate * torch.sigmoid(gate)
        # SiLU moves by at most 1.1 times its argument's error, and hardly where it is zero (x exp(x) of the end
        # nearer to it).  The approximate division is zero where 1 + exp(-x) passes 2^126: there |SiLU| is below
        # 89 * 2^-126, which is 1.05e-36
        slope = torch.where(gate < -20, (1 - gate) * torch.exp(gate + eg), torch.full_like(gate, 1.1))
        tol = slope * eg * (up.abs() + eu) + act.abs() * eu + (STEP[dtype] + 2.0 ** -20) * (act * up).abs() + 1.1e-36 * up.abs()
        assert ((out[s].double() - act * up).abs() <= tol + TINY[dtype]).all(), f"expert {e}"

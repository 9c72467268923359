"""GPU tests of microscaled 4-bit floating point: quantisation bit for bit against its definition in 64 bits
(where every quotient is decided exactly), the product against its formula, and a whole layer.

Tolerance of the product.  Codes and scales are exact numbers, so an output is a sum of K / 64 tensor-core
steps of exact block sums, each step aligned to the largest term and cut no coarser than 2^-22 of it:
(K / 64 + 2) 2^-22 sum |a w|, then factors (two roundings of 2^-24) and half a step of the output's type,
2^-8 |v| for bf16 and 2^-24 |v| for fp32.  SwiGLU h = g sigma(g) u from such g and u: the derivative of
SiLU is at most 1.1, its value at most |g|; its exponential is good to 2^-21 (bf16) and 2^-22 (fp32)."""
import math
import os
import subprocess
import sys

import pytest
import torch

from conftest import ROOT
from mixture_experts_ffn_gemm_gb300 import binding as B

pytestmark = pytest.mark.gpu

F32, BF16, U8 = torch.float32, torch.bfloat16, torch.uint8
STEP = {F32: 2.0 ** -24, BF16: 2.0 ** -8}
BLOCK = {"mx": 32, "nv": 16}
MAGS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
LUT = torch.tensor(MAGS + [-m for m in MAGS], dtype=torch.float64)
E4M3 = [float(v) for v in torch.arange(127, dtype=U8).view(torch.float8_e4m3fn).double()]


def _nearest_code(y):
    """Codes of magnitudes: nearest of MAGS, ties to the even code (float64 holds each midpoint)."""
    mid = [(MAGS[i] + MAGS[i + 1]) / 2 for i in range(7)]
    code = torch.zeros_like(y, dtype=torch.int64)
    for i, m in enumerate(mid):
        code += (y > m) | ((y == m) & (i % 2 == 1))
    return code


def quantize64(x, fmt, g=1.0):
    """(codes [R][K] 0..15, scale bytes [R][K / B]).  The quotients are decided in float64: x has at most 24
    bits and a scale times a midpoint at most 31, so unequal ones differ by more than float64's step."""
    R, K = x.shape
    v = x.double().cpu().view(R, K // BLOCK[fmt], BLOCK[fmt])
    amax = v.abs().amax(-1)
    finite = torch.isfinite(v).all(-1)
    amax = torch.where(finite, amax, torch.ones_like(amax))
    if fmt == "mx":
        _, e = torch.frexp(amax)
        byte = torch.where(amax > 0, (e - 1 + 127 - 2).clamp(min=0), torch.full_like(e, 127))
        S = torch.ldexp(torch.ones_like(amax), byte - 127)
        nan_byte = 255
    else:
        table = torch.tensor(E4M3, dtype=torch.float64)
        want = (amax / (6.0 * g)).clamp(max=448.0)
        hi = torch.searchsorted(table, want.contiguous()).clamp(max=126)
        lo = (hi - 1).clamp(min=0)
        up, down = table[hi] * (6.0 * g) - amax, amax - table[lo] * (6.0 * g)
        byte = torch.where((up < down) | ((up == down) & (hi % 2 == 0)) | (want == table[hi]), hi, lo)
        S = table[byte] * g
        nan_byte = 127
    y = torch.where(S[..., None] > 0, v.abs() / S[..., None].clamp(min=1e-300), torch.zeros_like(v))
    code = _nearest_code(y) + 8 * torch.signbit(v).long()
    code = torch.where(finite[..., None], code, torch.zeros_like(code))
    byte = torch.where(finite, byte.long(), torch.full_like(byte.long(), nan_byte))
    return code.view(R, K), byte


def scale_index(offs, K, fmt):
    """Byte index of each (row, scale column) by the documented layout; rows of all groups in order."""
    cols = K // BLOCK[fmt]
    kt = (cols + 3) // 4
    idx = torch.full((offs[-1], cols), -1, dtype=torch.int64)
    c = torch.arange(cols)
    for e in range(len(offs) - 1):
        r = torch.arange(offs[e + 1] - offs[e])
        first = offs[e] // 128 + e
        idx[offs[e]:offs[e + 1]] = (((first + r // 128) * kt)[:, None] + (c // 4)[None]) * 512 + (
            r % 32 * 16 + r % 128 // 32 * 4)[:, None] + (c % 4)[None]
    return idx


def unpack(codes):
    c = codes.cpu()
    return torch.stack([c & 15, c >> 4], 2).view(c.shape[0], -1).long()


def pack(code):
    c = code.view(code.shape[0], -1, 2)
    return (c[:, :, 0] | (c[:, :, 1] << 4)).to(U8)


def offsets_of(counts):
    o = [0]
    for c in counts:
        o.append(o[-1] + c)
    return o


def gpu(offs):
    return torch.tensor(offs, dtype=torch.int32, device="cuda")


def _inputs(R, K, dtype, seed=0):
    """Normal values, blocks of zeros, tiny and huge ones, exact midpoints between codes."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, K, generator=g) * torch.exp2(torch.randint(-6, 6, (R, 1), generator=g).float())
    x[:, ::37] *= 16
    if R > 2:
        x[1, :64] = 0
        x[2, :64] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -5.0,
                                  0.0, -0.0, 7.0, 7.5] * 4)
    if R > 4:
        x[3] *= 1e-38
        x[4] *= 1e35
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("fmt,g", [("mx", None), ("nv", None), ("nv", 0.0371), ("nv", 2.0 ** -5),
                                   ("nv", 1e-20)])
@pytest.mark.parametrize("R,K,pad", [(1, 64, 0), (7, 192, 8), (300, 320, 0), (33, 2112, 64), (5, 7168, 0)])
def test_quantize_is_exact(cuda_device, fmt, g, dtype, R, K, pad):
    x = _inputs(R, K, dtype, seed=R)
    buf = torch.zeros(R, K + pad, dtype=dtype, device="cuda")
    buf[:, :K] = x.cuda()
    cfg = B.make_micro_config(R, K, fmt, dtype=dtype, ld=K + pad)
    codes, scales = B.alloc_micro(cfg)
    ws = B.alloc_micro_workspace(cfg)
    f = None if g is None else torch.tensor([g], device="cuda")
    B.moe_micro_quantize(cfg, buf[:, :K], None, None, f, codes, scales, ws)
    assert B.moe_device_status(ws) == B.MOE_OK
    code, byte = quantize64(x, fmt, 1.0 if f is None else float(f.double()))
    assert torch.equal(scales.cpu().long()[scale_index([0, R], K, fmt)], byte)
    assert torch.equal(unpack(codes), code)


@pytest.mark.parametrize("g", [1.0, 0.75, 0.0371, 1.7e-3])
def test_quotients_next_to_a_border_stay_on_their_side(cuda_device, g):
    """fp32 values at, just below and just above every midpoint between two codes, and block maxima at,
    below and above midpoints between two scales."""
    f = torch.tensor([g], dtype=F32)
    gd = float(f.double())
    rows = []
    for s in E4M3[8:127:5]:
        for m in [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]:
            base = torch.tensor(m * s * gd, dtype=torch.float64).to(F32)
            r = torch.zeros(16, dtype=F32)
            r[0] = torch.tensor(6.0 * s * gd, dtype=torch.float64).to(F32)
            r[1], r[2], r[3] = base, torch.nextafter(base, f * 0), torch.nextafter(base, f * 1e9)
            r[4:7] = -r[1:4]
            rows.append(r)
    for i in range(1, 126):  # maxima around the midpoints of neighbouring scales
        mid = torch.tensor((E4M3[i] + E4M3[i + 1]) / 2 * 6.0 * gd, dtype=torch.float64).to(F32)
        for top in (mid, torch.nextafter(mid, f * 0), torch.nextafter(mid, f * 1e9)):
            r = torch.linspace(-1, 1, 16) * top * 0.7
            r[5] = top
            rows.append(r)
    while len(rows) % 4:
        rows.append(torch.zeros(16))
    x = torch.stack(rows).view(-1, 64)
    cfg = B.make_micro_config(x.shape[0], 64, "nv", dtype=F32)
    codes, scales = B.alloc_micro(cfg)
    ws = B.alloc_micro_workspace(cfg)
    B.moe_micro_quantize(cfg, x.cuda(), None, None, f.cuda(), codes, scales, ws)
    code, byte = quantize64(x, "nv", gd)
    assert torch.equal(scales.cpu().long()[scale_index([0, x.shape[0]], 64, "nv")], byte)
    assert torch.equal(unpack(codes), code)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_blocks_with_nan_or_infinity_read_as_nan(cuda_device, fmt, dtype):
    K, bs = 256, BLOCK[fmt]
    x = torch.ones(4, K, dtype=dtype)
    x[0, 5], x[1, 70], x[2, 255] = float("nan"), float("inf"), -float("inf")
    cfg = B.make_micro_config(4, K, fmt, dtype=dtype)
    codes, scales = B.alloc_micro(cfg)
    ws = B.alloc_micro_workspace(cfg)
    B.moe_micro_quantize(cfg, x.cuda(), None, None, None, codes, scales, ws)
    code, byte = quantize64(x, fmt)
    assert torch.equal(scales.cpu().long()[scale_index([0, 4], K, fmt)], byte)
    assert torch.equal(unpack(codes), code)
    out = torch.empty(4, K, dtype=dtype, device="cuda")
    B.moe_micro_dequantize(cfg, codes, scales, None, None, out, ws)
    bad = (~torch.isfinite(x)).view(4, -1, bs).any(-1, keepdim=True).expand(4, K // bs, bs).reshape(4, K)
    assert torch.equal(torch.isnan(out.cpu()), bad)


def test_factor_outside_its_range(cuda_device):
    for g in (0.0, -1.0, float("nan"), float("inf"), 1e-35):
        cfg = B.make_micro_config(3, 64, "nv")
        codes, scales = B.alloc_micro(cfg)
        ws = B.alloc_micro_workspace(cfg)
        B.moe_micro_quantize(cfg, torch.ones(3, 64, dtype=BF16, device="cuda"), None, None,
                             torch.tensor([g], device="cuda"), codes, scales, ws)
        assert B.moe_device_status(ws) == B.MOE_ERR_DEVICE_CHECK
        assert (scales.cpu()[scale_index([0, 3], 64, "nv")] == 127).all() and (codes == 0).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("counts,k", [([0, 5, 130, 0, 1, 124], 4), ([2], 1), ([1] * 40, 8), ([64, 0, 200], 3)])
def test_rows_to_their_experts_and_back(cuda_device, fmt, counts, k):
    """Each token to k rows of the experts' order; rows that no token names, and those behind the last
    expert, keep their bytes; destinations outside are skipped."""
    K, offs = 192, offsets_of(counts)
    R, behind = offs[-1], 9
    T = R // k
    g = torch.Generator().manual_seed(3)
    dest = torch.randperm(R, generator=g)[:T * k].view(T, k)
    dest[0, 0] = -1
    named = dest[dest >= 0]
    x = _inputs(T, K, BF16, seed=5)
    cfg = B.make_micro_config(R + behind, K, fmt, groups=len(counts), src_rows=T, copies=k)
    codes, scales = B.alloc_micro(cfg)
    codes.fill_(0xEE)
    scales.fill_(0xEE)
    ws = B.alloc_micro_workspace(cfg)
    B.moe_micro_quantize(cfg, x.cuda(), dest.to(torch.int32).cuda(), gpu(offs), None, codes, scales, ws)
    assert B.moe_device_status(ws) == B.MOE_ERR_DEVICE_CHECK  # the -1
    code, byte = quantize64(x, fmt)
    src = torch.full((R,), -1, dtype=torch.int64)
    src[dest.clamp(min=0).view(-1)] = torch.arange(T * k) // k
    if dest[0, 0] < 0 and not (named == 0).any():
        src[0] = -1
    idx = scale_index(offs, K, fmt)
    want = torch.full_like(scales.cpu(), 0xEE)
    want[idx[src >= 0].view(-1)] = byte[src[src >= 0]].to(U8).view(-1)
    # the last scale tile's columns behind K are not part of the format
    used = torch.zeros_like(want, dtype=torch.bool)
    used[idx.view(-1)] = True
    assert torch.equal(scales.cpu()[used], want[used])
    assert torch.equal(unpack(codes)[:R][src >= 0], code[src[src >= 0]])
    assert (codes.cpu()[:R][src < 0] == 0xEE).all() and (codes.cpu()[R:] == 0xEE).all()
    for dtype in (BF16, F32):
        back = B.make_micro_config(R + behind, K, fmt, groups=len(counts), dtype=dtype, ld=K + 8)
        out = torch.full((R + behind, K + 8), 7.0, dtype=dtype, device="cuda")
        B.moe_reset_device_status(ws)
        B.moe_micro_dequantize(back, codes, scales, gpu(offs), None, out[:, :K], ws)
        assert B.moe_device_status(ws) == B.MOE_OK
        S = torch.ldexp(torch.ones(byte.shape, dtype=torch.float64), byte - 127) if fmt == "mx" else \
            torch.tensor(E4M3 + [math.nan], dtype=torch.float64)[byte]
        val = (LUT[code].view(T, -1, BLOCK[fmt]) * S[..., None]).view(T, K)
        assert torch.equal(out.cpu().double()[:R, :K][src >= 0], val[src[src >= 0]].to(dtype).double())
        assert (out[:, K:] == 7.0).all() and (out[R:] == 7.0).all()


def _operand(g, offs, K, fmt):
    """Random codes and scales in the documented layout, and the values [rows][K] in float64."""
    R = offs[-1]
    code = torch.randint(0, 16, (R, K), generator=g)
    if fmt == "mx":
        byte = torch.randint(120, 131, (R, K // 32), generator=g)
        S = torch.ldexp(torch.ones(byte.shape, dtype=torch.float64), byte - 127)
    else:
        byte = torch.randint(30, 90, (R, K // 16), generator=g)
        S = torch.tensor(E4M3, dtype=torch.float64)[byte]
    val = (LUT[code].view(R, -1, BLOCK[fmt]) * S[..., None]).view(R, K)
    per = 64 if fmt == "nv" else 128
    size = (R // 128 + len(offs) - 1) * ((K + per - 1) // per) * 512
    # bytes outside the format: NaN in either format
    scales = torch.full((size,), 255, dtype=U8)
    scales[scale_index(offs, K, fmt).view(-1)] = byte.to(U8).view(-1)
    return pack(code).cuda(), scales.cuda(), val.cuda()


RAGGED = [0, 1, 127, 128, 129, 0, 300, 16, 33, 0]


def _product(counts, N, K, fmt, swiglu, dtype, pad=0, seed=0, factors=True):
    g = torch.Generator().manual_seed(seed)
    E, offs = len(counts), offsets_of(counts)
    R, per = offs[-1], (2 * N if swiglu else N)
    a, sa, va = _operand(g, offs, K, fmt)
    w, sw, vw = _operand(g, [e * per for e in range(E + 1)], K, fmt)
    fa = fw = None
    if fmt == "nv" and factors:
        fa = torch.tensor([0.37], device="cuda")
        fw = (torch.rand(E, generator=g) + 0.5).cuda() / K
    cfg = B.make_micro_product_config(R, E, N, K, fmt, dtype, swiglu, N + pad)
    ws = B.alloc_micro_product_workspace(cfg)
    out = torch.full((R, N + pad), 7.0, dtype=dtype, device="cuda")
    B.moe_micro_product(cfg, gpu(offs), a, sa, fa, w, sw, fw, out[:, :N], ws)
    assert B.moe_device_status(ws) == B.MOE_OK
    assert (out[:, N:] == 7.0).all()
    for e in range(E):
        s = slice(offs[e], offs[e + 1])
        f = (float(fa.double()) * float(fw[e].double())) if fa is not None else 1.0
        we = vw[e * per:(e + 1) * per]
        y = f * (va[s] @ we.t())
        err = ((K / 64 + 2) * 2.0 ** -22 + 2.0 ** -22) * (f * (va[s].abs() @ we.abs().t()))
        if swiglu:
            gate, up = y[:, :N], y[:, N:]
            eg, eu = err[:, :N], err[:, N:]
            act = gate * torch.sigmoid(gate)
            y = act * up
            err = 1.1 * eg * (up.abs() + eu) + act.abs() * eu + 2.0 ** -20 * y.abs()
        assert ((out[s, :N].double() - y).abs() <= STEP[dtype] * y.abs() + err).all(), f"expert {e}"


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,K", [(128, 64), (256, 256), (8, 192), (264, 320), (736, 2112), (384, 1024)])
def test_product_of_ragged_groups(cuda_device, fmt, dtype, N, K):
    _product(RAGGED, N, K, fmt, False, dtype)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,K", [(128, 64), (256, 448), (384, 1024)])
def test_product_with_swiglu(cuda_device, fmt, dtype, N, K):
    # mx values are about a power of two each: sums of K of them stay in the exponential's range
    _product(RAGGED, N, K, fmt, True, dtype, seed=1)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("counts", [[1], [5], [16], [17], [256, 0, 1000], [3] * 40, [700, 1500]])
def test_product_group_sizes(cuda_device, fmt, swiglu, counts):
    _product(counts, 256, 512, fmt, swiglu, BF16, pad=8, seed=2)


def test_product_refuses_and_survives_bad_offsets(cuda_device):
    g = torch.Generator().manual_seed(1)
    a, sa, _ = _operand(g, [0, 30, 60, 90], 128, "mx")
    w, sw, _ = _operand(g, [0, 64, 128, 192], 128, "mx")
    cfg = B.make_micro_product_config(90, 3, 64, 128, "mx")
    ws = B.alloc_micro_product_workspace(cfg)
    out = torch.empty(90, 64, dtype=BF16, device="cuda")
    for bad in ([0, 40, 30, 90], [0, 40, 60, 9999], [-5, 40, 60, 90], [0, -(2 ** 31), 2 ** 31 - 1, 90]):
        B.moe_micro_product(cfg, gpu(bad), a, sa, None, w, sw, None, out, ws)
        assert B.moe_device_status(ws) == B.MOE_ERR_DEVICE_CHECK
        B.moe_reset_device_status(ws)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_rows_of_no_expert_are_left(cuda_device, fmt):
    g = torch.Generator().manual_seed(1)
    a, sa, _ = _operand(g, [0, 30, 200], 128, fmt)
    w, sw, _ = _operand(g, [0, 64, 128], 128, fmt)
    cfg = B.make_micro_product_config(200, 2, 64, 128, fmt, F32)
    ws = B.alloc_micro_product_workspace(cfg)
    out = torch.full((200, 64), 7.0, device="cuda")
    B.moe_micro_product(cfg, gpu([0, 30, 77]), a, sa, None, w, sw, None, out, ws)
    assert (out[77:] == 7.0).all() and (out[:77] != 7.0).any()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_a_layer_of_microscaled_experts(cuda_device, fmt):
    """Router, permutation, quantisation, product with SwiGLU, quantisation, product, combine: the run
    that a layer with 4-bit experts is, replayed from a CUDA graph, against the same steps in 64 bits.
    h is rounded to bf16 before it is quantised; the reference quantises the h that the run made, so
    that each step is held to its own tolerance."""
    T, d, E, k, I = 96, 512, 12, 4, 256
    P = T * k
    g = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, W_r, b = rnd(T, d).to(BF16), rnd(E, d) * d ** -0.5, rnd(E) * 0.01
    W13, W2 = (rnd(E * 2 * I, d) * d ** -0.5).to(BF16), (rnd(E * d, I) * I ** -0.5).to(BF16)
    cfg = B.make_config(T=T, d=d, E=E, k=k, I=I, n_shared=0)
    ws = B.alloc_workspace(cfg)
    f = lambda t: (t.abs().amax().float() / (6 * 448)).view(1) if fmt == "nv" else None  # noqa: E731
    fx, fh = f(x), torch.tensor([0.002], device="cuda") if fmt == "nv" else None
    f13, f2 = f(W13), f(W2)
    coded = []
    for w, rows, K, fac in ((W13, 2 * I, d, f13), (W2, d, I, f2)):
        c = B.make_micro_config(E * rows, K, fmt, groups=E)
        buf = B.alloc_micro(c)
        B.moe_micro_quantize(c, w, None, None, fac, *buf, ws)
        coded.append(buf)
    each = lambda v: None if v is None else v.expand(E).contiguous()  # noqa: E731
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    idx, wgt = i32((T, k)), torch.zeros(T, k, device="cuda")
    counts, offsets, src, dst = i32(E + 1), i32(E + 2), i32(P), i32(P)
    qx = B.make_micro_config(P, d, fmt, groups=E, src_rows=T, copies=k)
    qh = B.make_micro_config(P, I, fmt, groups=E)
    p13 = B.make_micro_product_config(P, E, I, d, fmt, BF16, swiglu=True)
    p2 = B.make_micro_product_config(P, E, d, I, fmt, F32)
    xb, hb = B.alloc_micro(qx), B.alloc_micro(qh)
    h = torch.zeros(P, I, dtype=BF16, device="cuda")
    y, out = torch.zeros(P, d, device="cuda"), torch.zeros(T, d, dtype=BF16, device="cuda")

    def layer():
        B.moe_router(cfg, x, W_r, b, None, idx, wgt, ws)
        B.moe_permute(cfg, idx, counts, offsets, src, dst, ws)
        B.moe_micro_quantize(qx, x, dst, offsets, fx, *xb, ws)
        B.moe_micro_product(p13, offsets, *xb, fx, *coded[0], each13, h, ws)
        B.moe_micro_quantize(qh, h, None, offsets, fh, *hb, ws)
        B.moe_micro_product(p2, offsets, *hb, fh, *coded[1], each2, y, ws)
        B.moe_combine(cfg, y, dst, wgt, None, out, ws)

    each13, each2 = each(f13), each(f2)
    layer()
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert B.moe_device_status(ws) == B.MOE_OK
    assert torch.equal(first, out)

    def values(t, fac):
        gd = 1.0 if fac is None else float(fac.double())
        code, byte = quantize64(t, fmt, gd)
        S = torch.ldexp(torch.ones(byte.shape, dtype=torch.float64), byte - 127) if fmt == "mx" else \
            torch.tensor(E4M3, dtype=torch.float64)[byte] * gd
        return (LUT[code].view(t.shape[0], -1, BLOCK[fmt]) * S[..., None]).view(t.shape).cuda()

    v13, v2 = values(W13, f13).view(E, 2 * I, d), values(W2, f2).view(E, d, I)
    vx, vh = values(x, fx)[(src // k).long()], values(h, fh)
    offs = offsets.cpu().tolist()
    want = torch.zeros(P, d, dtype=torch.float64, device="cuda")
    for e in range(E):
        s = slice(offs[e], offs[e + 1])
        a13 = vx[s] @ v13[e].t()
        gate, up = a13[:, :I], a13[:, I:]
        he = gate * torch.sigmoid(gate) * up
        mag = vx[s].abs() @ v13[e].abs().t()
        err = (d / 64 + 3) * 2.0 ** -22 * mag
        tol = 2.0 ** -8 * he.abs() + 1.1 * err[:, :I] * (up.abs() + err[:, I:]) + \
            (gate * torch.sigmoid(gate)).abs() * err[:, I:] + 2.0 ** -20 * he.abs()
        assert ((h[s].double() - he).abs() <= tol).all()
        want[s] = vh[s] @ v2[e].t()
        mag2 = vh[s].abs() @ v2[e].abs().t()
        assert ((y[s].double() - want[s]).abs() <= (I / 64 + 3) * 2.0 ** -22 * mag2
                + 2.0 ** -24 * want[s].abs()).all()
    terms = wgt.double()[:, :, None] * y.double()[dst.view(T, k).long()]
    total = terms.sum(1)
    # k products and k sums in fp32, then half a step
    assert ((out.double() - total).abs() <= 2.0 ** -8 * total.abs() + 2 * k * 2.0 ** -24 * terms.abs().sum(1)).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("swiglu", [False, True])
def test_nan_rows_and_weights_stay_their_own(cuda_device, fmt, swiglu):
    """A NaN channel makes its row's outputs NaN and no other row's; a NaN weight block its expert's column."""
    K, N, counts = 256, 128, [40, 70, 9]
    offs, E = offsets_of(counts), len(counts)
    g = torch.Generator().manual_seed(4)
    per = 2 * N if swiglu else N
    x = torch.randn(offs[-1], K, generator=g).to(BF16)
    w = (torch.randn(E * per, K, generator=g) / 16).to(BF16)

    def run(x, w):
        cx = B.make_micro_config(offs[-1], K, fmt, groups=E)
        cw = B.make_micro_config(E * per, K, fmt, groups=E)
        bx, bw = B.alloc_micro(cx), B.alloc_micro(cw)
        ws = B.alloc_micro_workspace(cx)
        B.moe_micro_quantize(cx, x.cuda(), None, gpu(offs), None, *bx, ws)
        B.moe_micro_quantize(cw, w.cuda(), None, None, None, *bw, ws)
        out = torch.zeros(offs[-1], N, device="cuda")
        cfg = B.make_micro_product_config(offs[-1], E, N, K, fmt, F32, swiglu)
        B.moe_micro_product(cfg, gpu(offs), *bx, None, *bw, None, out, ws)
        assert B.moe_device_status(ws) == B.MOE_OK
        return out.cpu()

    clean = run(x, w)
    assert torch.isfinite(clean).all()
    x2, w2 = x.clone(), w.clone()
    x2[50, 77] = float("nan")
    x2[0, 3] = float("inf")
    w2[2 * per + 5, 200] = float("nan")
    got = run(x2, w2)
    bad = torch.zeros_like(clean, dtype=torch.bool)
    bad[50], bad[0] = True, True
    bad[offs[2]:, 5] = True
    assert torch.equal(torch.isnan(got), bad)
    assert torch.equal(got[~bad], clean[~bad])


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_two_streams_at_once(cuda_device, fmt):
    """Two products and quantisations under way together, each on its own workspace, give what they give
    alone."""
    counts = [300, 0, 17, 450]
    offs, E, N, K = offsets_of(counts), len(counts), 512, 1024
    g = torch.Generator().manual_seed(6)
    w, sw, _ = _operand(g, [e * N for e in range(E + 1)], K, fmt)
    xs = [torch.randn(offs[-1], K, generator=g).to(BF16).cuda() for _ in range(2)]
    cx = B.make_micro_config(offs[-1], K, fmt, groups=E)
    cfg = B.make_micro_product_config(offs[-1], E, N, K, fmt)
    o = gpu(offs)

    def go(x, stream, buf, ws, out):
        B.moe_micro_quantize(cx, x, None, o, None, *buf, ws, stream=stream)
        B.moe_micro_product(cfg, o, *buf, None, w, sw, None, out, ws, stream=stream)

    state = [(B.alloc_micro(cx), B.alloc_micro_workspace(cx), torch.zeros(offs[-1], N, dtype=BF16, device="cuda"))
             for _ in range(4)]
    for i in range(2):
        go(xs[i], None, *state[i])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for i in range(2):
            go(xs[i], streams[i], *state[2 + i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(state[i][2], state[2 + i][2])
        assert B.moe_device_status(state[2 + i][1]) == B.MOE_OK


def test_the_first_call_of_a_process_may_be_captured(cuda_device):
    """Kernels are loaded and their attributes set by the first call: one under capture, replayed after."""
    code = """
import torch
from mixture_experts_ffn_gemm_gb300 import binding as B
torch.cuda.init()
o = torch.tensor([0, 3, 40], dtype=torch.int32, device="cuda")
x = torch.ones(40, 128, dtype=torch.bfloat16, device="cuda")
w = torch.ones(2, 64, 128, dtype=torch.bfloat16, device="cuda")
y = torch.zeros(40, 64, dtype=torch.bfloat16, device="cuda")
cq, cw = B.make_micro_config(40, 128, groups=2), B.make_micro_config(128, 128, groups=2)
bq, bw = B.alloc_micro(cq), B.alloc_micro(cw)
z = torch.zeros(40, 64, device="cuda")
ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    B.moe_grouped_product(B.make_product_config(40, 2, 64, 128), o, x, w, y, ws)
    B.moe_micro_quantize(cw, w.view(128, 128), None, None, None, *bw, ws)
    B.moe_micro_quantize(cq, x, None, o, None, *bq, ws)
    B.moe_micro_product(B.make_micro_product_config(40, 2, 64, 128, "mx", torch.float32), o, *bq, None,
                        *bw, None, z, ws)
assert (y == 0).all() and (z == 0).all()
g.replay()
torch.cuda.synchronize()
assert (y == 128).all() and (z == 128).all() and B.moe_device_status(ws) == B.MOE_OK
print("replayed")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, PYTHONPATH=ROOT))
    assert r.returncode == 0 and "replayed" in r.stdout, r.stderr

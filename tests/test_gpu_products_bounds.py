"""GPU tests of what the products grouped by expert and the microscaled operators leave alone: outputs with a margin
on either side of the buffer under offsets out of range, and every byte of the scales that is no written row's.

Offsets out of range: an expert's rows begin at its first bound taken into [0, rows] and end at its second one
taken into what remains.  Tolerances as in test_gpu_grouped.py and test_gpu_micro.py."""
import pytest
import torch

import test_gpu_grouped as grouped
from mixture_experts_ffn_gemm_gb300 import binding as B
from test_gpu_micro import _operand, gpu, offsets_of, quantize64, scale_index, unpack

pytestmark = pytest.mark.gpu

F32, BF16, U8, I32 = torch.float32, torch.bfloat16, torch.uint8, torch.int32
STEP = {F32: 2.0 ** -24, BF16: 2.0 ** -8}
MARGIN, R = 4096, 90
BAD = [[0, 40, 30, 90], [0, 40, 60, 9999], [-5, 40, 60, 90], [0, -(2 ** 31), 2 ** 31 - 1, 90], [91, 95, 80, 20],
       [-7, -3, -1, 0]]


def _ranges(bad):
    out = []
    for a, z in zip(bad, bad[1:]):
        lo = min(max(a, 0), R)
        out.append((lo, min(max(z, lo), R)))
    return out


def _within(numel, dtype):
    """(the whole buffer, its middle)"""
    whole = torch.full((numel + 2 * MARGIN,), 7.0, dtype=dtype, device="cuda")
    return whole, whole[MARGIN:MARGIN + numel]


def _margins_hold(whole):
    assert (whole[:MARGIN] == 7.0).all() and (whole[-MARGIN:] == 7.0).all()


def _rows_hold(out, ranges, values):
    """Rows of one expert have its value, rows of several one of theirs, rows of none what they held.
    values[e]: (value, tolerance) of all R rows by expert e."""
    fits = torch.zeros(R, dtype=torch.bool, device="cuda")
    taken = torch.zeros_like(fits)
    for (lo, hi), (v, tol) in zip(ranges, values):
        fits[lo:hi] |= ((out[lo:hi].double() - v[lo:hi]).abs() <= tol[lo:hi]).all(1)
        taken[lo:hi] = True
    assert (fits == taken).all()
    assert (out[~taken] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", grouped.KINDS)
@pytest.mark.parametrize("bad", BAD)
def test_products_under_offsets_out_of_range(cuda_device, kind, bad, dtype):
    N, K, E = 64, 136, 3
    _, _, a, b = grouped._make(kind, [30, 30, 30], N, K, seed=5)
    cfg = grouped._config(kind, R, E, N, K, dtype)
    ws = B.alloc_product_workspace(cfg)
    shape = {"forward": (R, N), "grad_x": (R, K), "grad_w": (E, N, K)}[kind]
    whole, out = _within(torch.Size(shape).numel(), dtype)
    out = out.view(shape)
    B.moe_grouped_product(cfg, gpu(bad), a, b, out, ws)
    assert B.moe_device_status(ws) == B.MOE_ERR_DEVICE_CHECK
    _margins_hold(whole)
    ranges = _ranges(bad)
    if kind == "grad_w":
        for e, (lo, hi) in enumerate(ranges):
            p, q = a[lo:hi].double(), b[lo:hi].double()
            v, mag = p.t() @ q, p.abs().t() @ q.abs()
            tol = STEP[dtype] * v.abs() + ((hi - lo) / 16 + 2) * 2.0 ** -22 * mag
            assert ((out[e].double() - v).abs() <= tol).all()
        return
    values = []
    for e in range(E):
        w = b[e].double().t() if kind == "forward" else b[e].double()
        v, mag = a.double() @ w, a.double().abs() @ w.abs()
        values.append((v, STEP[dtype] * v.abs() + (w.shape[0] / 16 + 2) * 2.0 ** -22 * mag))
    _rows_hold(out, ranges, values)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("bad", BAD)
def test_microscaled_products_under_offsets_out_of_range(cuda_device, fmt, bad, dtype):
    N, K, E = 64, 192, 3
    ranges = _ranges(bad)
    clean = [r[0] for r in ranges] + [ranges[-1][1]]
    in_order = all(z == a for (_, z), (a, _) in zip(ranges, ranges[1:])) and clean[0] == 0 and clean[-1] == R
    g = torch.Generator().manual_seed(6)
    offs = clean if in_order else [0, 30, 60, R]  # where the scales lie follows the experts' first rows
    a, sa, va = _operand(g, offs, K, fmt)
    w, sw, vw = _operand(g, [e * N for e in range(E + 1)], K, fmt)
    cfg = B.make_micro_product_config(R, E, N, K, fmt, dtype)
    ws = B.alloc_micro_product_workspace(cfg)
    whole, out = _within(R * N, dtype)
    out = out.view(R, N)
    B.moe_micro_product(cfg, gpu(bad), a, sa, None, w, sw, None, out, ws)
    assert B.moe_device_status(ws) == B.MOE_ERR_DEVICE_CHECK
    _margins_hold(whole)
    if in_order:
        values = []
        for e in range(E):
            we = vw[e * N:(e + 1) * N].t()
            v, mag = va @ we, va.abs() @ we.abs()
            values.append((v, STEP[dtype] * v.abs() + (K / 64 + 3) * 2.0 ** -22 * mag))
        _rows_hold(out, ranges, values)
    else:
        taken = torch.zeros(R, dtype=torch.bool)
        for lo, hi in ranges:
            taken[lo:hi] = True
        assert (out[~taken.cuda()] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("bad", BAD)
def test_quantisation_and_back_under_offsets_out_of_range(cuda_device, fmt, bad, dtype):
    """Rows that find no group, or one that ends in front of them, are skipped; nothing outside is written."""
    K, E = 192, 3
    cfg = B.make_micro_config(R, K, fmt, groups=E, dtype=dtype)
    ws = B.alloc_micro_workspace(cfg)
    size = B.moe_micro_scales_size(cfg)
    codes, scales = (torch.full((n + 2 * MARGIN,), 0xEE, dtype=U8, device="cuda") for n in (R * K // 2, size))
    x = torch.randn(R, K, generator=torch.Generator().manual_seed(7)).to(dtype).cuda()
    inner = lambda t: t[MARGIN:-MARGIN]  # noqa: E731
    dest = torch.arange(R, dtype=I32, device="cuda")
    for d in (None, dest):
        B.moe_micro_quantize(cfg, x, d, gpu(bad), None, inner(codes).view(R, K // 2), inner(scales), ws)
    whole, out = _within(R * K, dtype)
    B.moe_micro_dequantize(cfg, inner(codes).view(R, K // 2), inner(scales), gpu(bad), None, out.view(R, K), ws)
    assert B.moe_device_status(ws) in (B.MOE_OK, B.MOE_ERR_DEVICE_CHECK)
    _margins_hold(whole)
    for t in (codes, scales):
        assert (t[:MARGIN] == 0xEE).all() and (t[-MARGIN:] == 0xEE).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("K", [64, 192, 320])
@pytest.mark.parametrize("counts,k", [([0, 5, 130, 0, 1, 124], 4), ([2], 1), ([1] * 40, 8), ([64, 0, 200], 3)])
def test_scales_of_rows_that_no_token_names_are_not_written(cuda_device, fmt, K, counts, k):
    """Of a tile's bytes only the named rows' are written: their columns, and those behind K in their last tile."""
    offs = offsets_of(counts)
    rows, behind = offs[-1], 9
    T = max(1, rows // k - 1)  # at least k rows stay without a token, where there is more than one
    g = torch.Generator().manual_seed(8)
    dest = torch.randperm(rows, generator=g)[:T * k].view(T, k)
    x = torch.randn(T, K, generator=g).to(BF16)
    cfg = B.make_micro_config(rows + behind, K, fmt, groups=len(counts), src_rows=T, copies=k)
    codes, scales = B.alloc_micro(cfg)
    codes.fill_(0xEE)
    scales.fill_(0xEE)
    ws = B.alloc_micro_workspace(cfg)
    B.moe_micro_quantize(cfg, x.cuda(), dest.to(I32).cuda(), gpu(offs), None, codes, scales, ws)
    assert B.moe_device_status(ws) == B.MOE_OK
    code, byte = quantize64(x, fmt)
    src = torch.full((rows,), -1, dtype=torch.int64)
    src[dest.view(-1)] = torch.arange(T * k) // k
    named = src >= 0
    tile = 64 if fmt == "nv" else 128
    want = torch.full_like(scales.cpu(), 0xEE)
    want[scale_index(offs, K, fmt)[named].view(-1)] = byte[src[named]].to(U8).view(-1)
    free = torch.zeros_like(want, dtype=torch.bool)
    padded = scale_index(offs, (K + tile - 1) // tile * tile, fmt)
    free[padded[named][:, byte.shape[1]:].reshape(-1)] = True
    assert torch.equal(scales.cpu()[~free], want[~free])
    assert torch.equal(unpack(codes)[:rows][named], code[src[named]])
    assert (codes.cpu()[:rows][~named] == 0xEE).all() and (codes[rows:] == 0xEE).all()

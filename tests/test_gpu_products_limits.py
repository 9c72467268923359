"""GPU tests of the products grouped by expert and the microscaled operators at the ends of their ranges:
buffers whose offsets pass 32 bits, the widest sums and outputs, the most experts and copies, rows that start
at any multiple of 16 bytes.

Tolerances as in test_gpu_grouped.py and test_gpu_micro.py: half a step of the output's type, and
2^-22 sum |a b| for every MMA step of the sum (16 bf16 products, 64 microscaled ones)."""
import pytest
import torch

from mixture_experts_ffn_gemm_gb300 import binding as B

pytestmark = pytest.mark.gpu

F32, BF16, U8, I32 = torch.float32, torch.bfloat16, torch.uint8, torch.int32
STEP = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


def _randn(*shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda", dtype=F32).to(BF16)


def _close(got, v, mag, steps):
    tol = STEP[got.dtype] * v.abs() + (steps + 2) * 2.0 ** -22 * mag
    assert ((got.double() - v).abs() <= tol).all()


def _product(kind, offs, a, b, out, N, K, **kw):
    cfg = B.make_product_config(rows=kw.pop("rows"), E=len(offs) - 1, N=N, K=K, kind=kind, out_dtype=out.dtype,
                                **kw)
    ws = B.alloc_product_workspace(cfg)
    B.moe_grouped_product(cfg, torch.tensor(offs, dtype=I32, device="cuda"), a, b, out, ws)
    assert B.moe_device_status(ws) == B.MOE_OK


def test_rows_beyond_32_bit_offsets(cuda_device):
    """The rows of the last experts lie past 2^32 elements of x and of dx, and past 2^31 of y."""
    K, N, R = 7168, 16, 620000
    offs = [0, 300000, R - 300, R]
    x = torch.zeros(R, K, dtype=BF16, device="cuda")
    x[-400:] = _randn(400, K)
    w = _randn(3, N, K, seed=1)
    y = torch.empty(R, N, dtype=F32, device="cuda")
    _product("forward", offs, x, w, y, N, K, rows=R)
    tail = slice(R - 400, R)
    e = torch.where(torch.arange(R - 400, R, device="cuda") < offs[2], 1, 2)
    v = torch.stack([x[tail].double() @ w[i].double().t() for i in (1, 2)])
    mag = torch.stack([x[tail].double().abs() @ w[i].double().abs().t() for i in (1, 2)])
    pick = (e - 1).view(1, -1, 1).expand(1, -1, N)
    _close(y[tail], v.gather(0, pick)[0], mag.gather(0, pick)[0], K // 16)
    assert (y[:R - 400] == 0).all()
    dy = torch.zeros(R, N, dtype=BF16, device="cuda")
    dy[tail] = _randn(400, N, seed=2)
    dw = torch.empty(3, N, K, dtype=F32, device="cuda")
    _product("grad_w", offs, dy, x, dw, N, K, rows=R)
    for i, (lo, hi) in enumerate(zip(offs, offs[1:])):
        s = slice(max(lo, R - 400), hi)
        p, q = (dy[s].double(), x[s].double()) if hi > R - 400 else (dy[:1].double(), x[:1].double())
        _close(dw[i], p.t() @ q, p.abs().t() @ q.abs(), (hi - lo) // 16)
    x.fill_(7.0)
    _product("grad_x", offs, dy, w, x, N, K, rows=R)
    v = torch.stack([dy[tail].double() @ w[i].double() for i in (1, 2)])
    mag = torch.stack([dy[tail].double().abs() @ w[i].double().abs() for i in (1, 2)])
    pick = (e - 1).view(1, -1, 1).expand(1, -1, K)
    _close(x[tail], v.gather(0, pick)[0], mag.gather(0, pick)[0], 1)
    assert (x[:1000] == 0).all() and (x[300000:301000] == 0).all()


def test_codes_beyond_32_bit_offsets(cuda_device):
    K, R = 7168, 620000
    x = torch.zeros(R, K, dtype=BF16, device="cuda")
    x[-200:] = _randn(200, K)
    offs = torch.tensor([0, 1000, R - 77, R], dtype=I32, device="cuda")
    cfg = B.make_micro_config(R, K, "nv", groups=3)
    codes, scales = B.alloc_micro(cfg)
    ws = B.alloc_micro_workspace(cfg)
    B.moe_micro_quantize(cfg, x, None, offs, None, codes, scales, ws)
    small = B.make_micro_config(200, K, "nv")
    c2, s2 = B.alloc_micro(small)
    B.moe_micro_quantize(small, x[-200:], None, None, None, c2, s2, ws)
    assert torch.equal(codes[-200:], c2) and (codes[:-200] == 0).all()
    back, want = torch.empty_like(x), torch.empty(200, K, dtype=BF16, device="cuda")
    B.moe_micro_dequantize(cfg, codes, scales, offs, None, back, ws)
    B.moe_micro_dequantize(small, c2, s2, None, None, want, ws)
    assert torch.equal(back[-200:], want) and (back[:-200] == 0).all()
    w = _randn(3 * 8, K, seed=3)
    cw = B.make_micro_config(24, K, "nv", groups=3)
    bw = B.alloc_micro(cw)
    B.moe_micro_quantize(cw, w, None, None, None, *bw, ws)
    y = torch.empty(R, 8, dtype=F32, device="cuda")
    B.moe_micro_product(B.make_micro_product_config(R, 3, 8, K, "nv", F32), offs, codes, scales, None, *bw, None,
                        y, ws)
    assert B.moe_device_status(ws) == B.MOE_OK
    wv = torch.empty(24, K, dtype=F32, device="cuda")
    B.moe_micro_dequantize(B.make_micro_config(24, K, "nv", groups=3, dtype=F32), *bw, None, None, wv, ws)
    for rows, e in ((slice(R - 200, R - 77), 1), (slice(R - 77, R), 2)):
        p, q = back[rows].double(), wv[8 * e:8 * e + 8].double()
        _close(y[rows], p @ q.t(), p.abs() @ q.abs().t(), K // 64)
    assert (y[:R - 200] == 0).all()


def test_wide_pitches(cuda_device):
    """Rows 2^21 elements apart: outputs past 2^32 elements."""
    R, N, K, ld = 2100, 24, 64, 1 << 21
    x, w = _randn(R, K), _randn(2, N, K, seed=1)
    flat = torch.full(((R - 1) * ld + N,), 7.0, dtype=BF16, device="cuda")
    y = flat.as_strided((R, N), (ld, 1))
    _product("forward", [0, 40, R], x, w, y, N, K, rows=R, ld_y=ld)
    for lo, hi, e in ((0, 40, 0), (40, R, 1)):
        p, q = x[lo:hi].double(), w[e].double()
        _close(y[lo:hi], p @ q.t(), p.abs() @ q.abs().t(), K // 16)
    assert (flat[N:ld] == 7.0).all() and (flat[-ld:-N] == 7.0).all()


@pytest.mark.parametrize("N,K", [(8, 131072), (131072, 8), (131072, 64)])
def test_widest_products(cuda_device, N, K):
    offs = [0, 3, 3, 40]
    x, dy, w = _randn(40, K), _randn(40, N, seed=1), _randn(3, N, K, seed=2)
    y, dx = torch.empty(40, N, dtype=BF16, device="cuda"), torch.empty(40, K, dtype=F32, device="cuda")
    dw = torch.empty(3, N, K, dtype=BF16, device="cuda")
    _product("forward", offs, x, w, y, N, K, rows=40)
    _product("grad_x", offs, dy, w, dx, N, K, rows=40)
    _product("grad_w", offs, dy, x, dw, N, K, rows=40)
    for e, (lo, hi) in enumerate(zip(offs, offs[1:])):
        a, b, c = x[lo:hi].double(), dy[lo:hi].double(), w[e].double()
        _close(y[lo:hi], a @ c.t(), a.abs() @ c.abs().t(), K / 16)
        _close(dx[lo:hi], b @ c, b.abs() @ c.abs(), N / 16)
        _close(dw[e], b.t() @ a, b.abs().t() @ a.abs(), 3)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("N,K", [(8, 131072), (131072, 64)])
def test_widest_microscaled_products(cuda_device, fmt, N, K):
    offs = torch.tensor([0, 3, 3, 40], dtype=I32, device="cuda")
    x, w = _randn(40, K), _randn(3 * N, K, seed=2)
    cx, cw = B.make_micro_config(40, K, fmt, groups=3), B.make_micro_config(3 * N, K, fmt, groups=3)
    bx, bw = B.alloc_micro(cx), B.alloc_micro(cw)
    ws = B.alloc_micro_workspace(cx)
    B.moe_micro_quantize(cx, x, None, offs, None, *bx, ws)
    B.moe_micro_quantize(cw, w, None, None, None, *bw, ws)
    y = torch.empty(40, N, dtype=F32, device="cuda")
    B.moe_micro_product(B.make_micro_product_config(40, 3, N, K, fmt, F32), offs, *bx, None, *bw, None, y, ws)
    xv, wv = torch.empty(40, K, dtype=F32, device="cuda"), torch.empty(3 * N, K, dtype=F32, device="cuda")
    B.moe_micro_dequantize(B.make_micro_config(40, K, fmt, groups=3, dtype=F32), *bx, offs, None, xv, ws)
    B.moe_micro_dequantize(B.make_micro_config(3 * N, K, fmt, groups=3, dtype=F32), *bw, None, None, wv, ws)
    assert B.moe_device_status(ws) == B.MOE_OK
    for e, (lo, hi) in enumerate(((0, 3), (3, 3), (3, 40))):
        p, q = xv[lo:hi].double(), wv[e * N:(e + 1) * N].double()
        _close(y[lo:hi], p @ q.t(), p.abs() @ q.abs().t(), K / 64)


def test_most_experts_and_copies(cuda_device):
    """1023 experts, a third of them with rows; 32 copies of each token."""
    E, T, k, K, N = 1023, 30, 32, 64, 40
    R = T * k
    g = torch.Generator().manual_seed(5)
    pick = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)])
    flat = pick.view(-1)
    order = torch.sort(flat, stable=True).indices
    dest = torch.empty(R, dtype=torch.int64)
    dest[order] = torch.arange(R)
    offs = [0] + torch.cumsum(torch.bincount(flat, minlength=E), 0).tolist()
    o = torch.tensor(offs, dtype=I32, device="cuda")
    x, w = _randn(T, K), _randn(E * N, K, seed=6)
    cx = B.make_micro_config(R, K, "mx", groups=E, src_rows=T, copies=k)
    cw = B.make_micro_config(E * N, K, "mx", groups=E)
    bx, bw = B.alloc_micro(cx), B.alloc_micro(cw)
    ws = B.alloc_micro_workspace(cx)
    B.moe_micro_quantize(cx, x, dest.to(I32).cuda(), o, None, *bx, ws)
    B.moe_micro_quantize(cw, w, None, None, None, *bw, ws)
    y = torch.empty(R, N, dtype=F32, device="cuda")
    B.moe_micro_product(B.make_micro_product_config(R, E, N, K, "mx", F32), o, *bx, None, *bw, None, y, ws)
    xv, wv = torch.empty(R, K, dtype=F32, device="cuda"), torch.empty(E * N, K, dtype=F32, device="cuda")
    B.moe_micro_dequantize(B.make_micro_config(R, K, "mx", groups=E, dtype=F32), *bx, o, None, xv, ws)
    B.moe_micro_dequantize(B.make_micro_config(E * N, K, "mx", groups=E, dtype=F32), *bw, None, None, wv, ws)
    assert B.moe_device_status(ws) == B.MOE_OK
    token = (order // k).cuda()
    assert ((xv - x[token].float()).abs() <= 0.25 * x[token].float().abs().view(R, -1, 32).amax(-1)
            .repeat_interleave(32, 1)).all()  # e2m1 with a power-of-two scale: at most 8 cut to 6
    expert = torch.sort(flat, stable=True).values.cuda()
    we = wv.view(E, N, K)[expert].double()
    v = torch.einsum("rk,rnk->rn", xv.double(), we)
    mag = torch.einsum("rk,rnk->rn", xv.double().abs(), we.abs())
    _close(y, v, mag, 1)
    xb = x[token]
    yb = torch.empty(R, N, dtype=F32, device="cuda")
    _product("forward", offs, xb, w.view(E, N, K), yb, N, K, rows=R)
    wb = w.view(E, N, K)[expert].double()
    _close(yb, torch.einsum("rk,rnk->rn", xb.double(), wb),
           torch.einsum("rk,rnk->rn", xb.double().abs(), wb.abs()), K / 16)


@pytest.mark.parametrize("skip", [8, 24])
def test_rows_that_start_at_multiples_of_16_bytes(cuda_device, skip):
    """Slices of wider buffers whose first element and pitch are multiples of 16 bytes, not of 32."""
    R, N, K, pad = 150, 72, 192, 40
    offs = [0, 60, 61, R]
    xw, dyw = _randn(R, K + pad), _randn(R, N + pad, seed=1)
    x, dy, w = xw[:, skip:skip + K], dyw[:, skip:skip + N], _randn(3, N, K, seed=2)
    for kind, a, b, ref in (("forward", x, w, None), ("grad_x", dy, w, None), ("grad_w", dy, x, None)):
        width = N if kind == "forward" else K
        if kind == "grad_w":
            out = torch.empty(3 * N * K + 8, dtype=BF16, device="cuda")[8:].view(3, N, K)
        else:
            out = torch.zeros(R, width + pad, dtype=BF16, device="cuda")[:, skip:skip + width]
        _product(kind, offs, a, b, out, N, K, rows=R, ld_x=K + pad, ld_y=N + pad)
        for e, (lo, hi) in enumerate(zip(offs, offs[1:])):
            p = a[lo:hi].double()
            q = (b[lo:hi] if kind == "grad_w" else b[e]).double()
            got = out[e] if kind == "grad_w" else out[lo:hi]
            if kind == "forward":
                _close(got, p @ q.t(), p.abs() @ q.abs().t(), K / 16)
            elif kind == "grad_x":
                _close(got, p @ q, p.abs() @ q.abs(), N / 16)
            else:
                _close(got, p.t() @ q, p.abs().t() @ q.abs(), (hi - lo) / 16)
    plain = B.make_micro_config(R, K, "nv")
    odd = B.make_micro_config(R, K, "nv", ld=K + pad)
    ws = B.alloc_micro_workspace(plain)
    one, two = B.alloc_micro(plain), B.alloc_micro(plain)
    B.moe_micro_quantize(plain, x.contiguous(), None, None, None, *one, ws)
    B.moe_micro_quantize(odd, x, None, None, None, *two, ws)
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    v1 = torch.empty(R, K, dtype=BF16, device="cuda")
    v2 = torch.full((R, K + pad), 7.0, dtype=BF16, device="cuda")
    B.moe_micro_dequantize(plain, *one, None, None, v1, ws)
    B.moe_micro_dequantize(odd, *one, None, None, v2[:, skip:skip + K], ws)
    assert torch.equal(v1, v2[:, skip:skip + K])
    assert (v2[:, :skip] == 7.0).all() and (v2[:, skip + K:] == 7.0).all()


def test_tensors_that_are_no_plain_memory_are_refused(cuda_device):
    """Tensors that throw when asked for their sizes, strides or address: an error, not the process's end."""
    N, K, ld = 64, 128, 136
    offs = torch.tensor([0, 5, 14], dtype=I32, device="cuda")
    b = _randn(2, N, K)
    out = torch.empty(14, N, dtype=F32, device="cuda")
    ragged = torch.nested.nested_tensor([_randn(K), _randn(K - 8)] * 7)
    sparse = _randn(14, K).to_sparse()
    fixed = B.make_product_config(rows=14, E=2, N=N, K=K, out_dtype=F32)
    wide = B.make_product_config(rows=14, E=2, N=N, K=K, out_dtype=F32, ld_x=ld)
    ws = B.alloc_product_workspace(fixed)
    for cfg in (fixed, wide):
        for bad in (ragged, sparse):
            with pytest.raises((ValueError, RuntimeError)):
                B.moe_grouped_product(cfg, offs, bad, b, out, ws)
    with pytest.raises((ValueError, RuntimeError)):
        B.moe_grouped_product(fixed, offs, _randn(14, K), b, out, torch.zeros(256, dtype=U8, device="cuda").to_sparse())
    assert B.moe_device_status(ws) == B.MOE_OK


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_a_chain_in_which_each_kernel_reads_what_the_one_before_wrote(cuda_device, fmt):
    """Quantise, multiply, quantise the product in the same buffers, and so on, back to back and captured: the
    same bits as with a synchronisation behind each call.  Offsets, factors and destinations change too."""
    R, K, steps = 300, 512, 24
    w = _randn(2 * K, K, seed=1) * 0.1
    cw = B.make_micro_config(2 * K, K, fmt, groups=2)
    bw = B.alloc_micro(cw)
    cx = B.make_micro_config(R, K, fmt, groups=2)
    bx = B.alloc_micro(cx)
    ws = B.alloc_micro_workspace(cx)
    pc = B.make_micro_product_config(R, 2, K, K, fmt, BF16)
    B.moe_micro_quantize(cw, w, None, None, None, *bw, ws)
    first = _randn(R, K, seed=2)
    x, y = first.clone(), torch.empty_like(first)
    splits = [[0, (37 * i) % (R + 1), R] for i in range(steps)]
    all_offs = torch.tensor(splits, dtype=I32, device="cuda")
    all_dest = torch.stack([torch.randperm(R, generator=torch.Generator().manual_seed(i)) for i in range(steps)])
    all_dest = all_dest.to(I32).cuda()
    all_factor = torch.logspace(-3, 3, steps, base=2.0, device="cuda")
    offs, dest, factor = all_offs[0].clone(), all_dest[0].clone(), all_factor[:1].clone()

    g = factor if fmt == "nv" else None

    def run(sync):
        wait = torch.cuda.synchronize if sync else (lambda: None)
        x.copy_(first)
        for i in range(steps):
            offs.copy_(all_offs[i])
            dest.copy_(all_dest[i])
            factor.copy_(all_factor[i:i + 1])
            wait()
            B.moe_micro_quantize(cx, x, dest, offs, g, *bx, ws)
            wait()
            B.moe_micro_product(pc, offs, *bx, g, *bw, None, y, ws)
            wait()
            B.moe_micro_quantize(cx, y, dest, offs, g, *bx, ws)
            wait()
            B.moe_micro_dequantize(cx, *bx, offs, g, x, ws)
            wait()
            B.moe_micro_quantize(cx, x, dest, offs, g, *bx, ws)
            wait()
            B.moe_micro_product(pc, offs, *bx, g, *bw, None, x, ws)
            wait()
        return x.clone(), y.clone(), bx[0].clone(), bx[1].clone()

    want = run(True)
    assert torch.isfinite(want[0]).all() and (want[0] != 0).any()
    for _ in range(10):
        for a, b in zip(run(False), want):
            assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(False)
    for _ in range(10):
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert B.moe_device_status(ws) == B.MOE_OK

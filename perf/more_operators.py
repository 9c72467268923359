"""Workloads of the microscaled 4-bit operators and of the products grouped by expert: their plain form,
calls and inputs.

quant    Microscaled 4-bit floating point: rows in blocks of B channels, each block a scale S and 4-bit
         codes c of e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), the value c S.
         "mx": B = 32, S = 2^(floor(log2 amax) - 2) (a power of two held as its exponent);
         "nv": B = 16, S = s g with s = e4m3(amax / (6 g)) and a factor g of the whole tensor.
         c = x / S rounded to nearest (ties to the even code), at most 6.  Rows may be gathered: row r
         is source row perm_src[r] / k, and row t goes to the k rows dest[t], the order in which the
         experts take their tokens.  The pass goes to codes and scales and back to the values that
         they stand for.
micro    The experts' product on such operands: row r of expert e gives out[r][n] = sum_k x[r][k]
         W_e[n][k], x quantised from the tokens' rows within the pass, W_e held in 4 bits; with SwiGLU
         out = SiLU(x W1_e) * (x W3_e).
grouped  Products grouped by expert with ragged sizes, bf16 operands, rows [offsets[e], offsets[e+1])
         of expert e:  y = x W_e^T;  its gradients dx = dy W_e and dW_e = dy^T x.

``own`` false: elementary torch operations.  ``own`` true: the library's entry points.
"""
import math

import torch

own = False

DEV = "cuda"


def _quant(name, T, K, fmt, act="bf16", out="bf16", k=1, E=1, pad=0):
    return {"name": name, "op": "quant", "T": T, "K": K, "fmt": fmt, "act": act, "out": out, "k": k,
            "E": E, "pad": pad}


def _micro(name, T, k, E, N, K, fmt, swiglu=False, out="bf16"):
    return {"name": name, "op": "micro", "T": T, "k": k, "E": E, "N": N, "K": K, "fmt": fmt,
            "swiglu": swiglu, "out": out}


def _grouped(name, kind, T, k, E, N, K, out="bf16", pad=0):
    return {"name": name, "op": "grouped", "kind": kind, "T": T, "k": k, "E": E, "N": N, "K": K,
            "out": out, "pad": pad}


def listed():
    return [
        # one token's row, taken by its eight experts: launch latency only
        _quant("quant_mx_t1", 1, 7168, "mx", k=8, E=384),
        # a prompt's rows in the experts' order, finer blocks with a factor of the tensor
        _quant("quant_nv_t4096", 4096, 7168, "nv", k=8, E=384),
        # one token through the second product of its eight experts: eight rows, eight matrices
        _micro("micro_mx_t1", 1, 8, 384, 7168, 2048, "mx", out="f32"),
        # a decode batch through the first product and SwiGLU: every expert's weights once
        _micro("micro_nv_t128_swiglu", 128, 8, 384, 2048, 7168, "nv", swiglu=True),
        # a prompt of 8192 tokens through the first product and SwiGLU
        _micro("micro_mx_t8192_swiglu", 8192, 8, 384, 2048, 7168, "mx", swiglu=True),
        # the same prompt through the second product
        _micro("micro_nv_t8192", 8192, 8, 384, 7168, 2048, "nv"),
        # a small layer of ragged widths
        _micro("micro_mx_ragged", 131, 6, 60, 736, 2112, "mx"),
        # a decode step of sixteen sequences: few rows of many experts, the weights stream once
        _grouped("grouped_fwd_t16", "forward", 16, 8, 384, 2048, 7168),
        # a training batch over 64 experts: the product and its two gradients
        _grouped("grouped_fwd_t8192", "forward", 8192, 8, 64, 4096, 7168),
        _grouped("grouped_gradx_t4096", "grad_x", 4096, 8, 64, 4096, 7168),
        _grouped("grouped_gradw_t4096", "grad_w", 4096, 8, 64, 4096, 7168, out="f32"),
        # a small layer of ragged widths, rows inside wider buffers, some experts without a row
        _grouped("grouped_gradw_ragged", "grad_w", 41, 6, 60, 736, 1000, pad=8),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["quant", "micro", "micro", "grouped", "grouped"])
    k = rng.randint(1, 8)
    E = max(k, log_int(4, 384))
    if op == "quant":
        K = max(1, log_int(64, 7168) // 64) * 64
        return {"op": op, "T": log_int(1, 4096), "K": K, "fmt": rng.choice(["mx", "nv"]),
                "act": rng.choice(["bf16", "bf16", "f32"]), "out": rng.choice(["bf16", "f32"]),
                "k": k, "E": E, "pad": rng.choice([0, 0, 8, 64])}
    T = log_int(1, 8192)
    if op == "micro":
        swiglu = rng.random() < 0.5
        step = 128 if swiglu else 8
        N = max(1, log_int(128, 2048 if swiglu else 7168) // step) * step
        K = max(1, log_int(64, 7168 if swiglu or N <= 4096 else 3584) // 64) * 64
        return {"op": op, "T": T, "k": k, "E": E, "N": N, "K": K,
                "fmt": rng.choice(["mx", "nv"]), "swiglu": swiglu,
                "out": rng.choice(["bf16", "f32"])}
    N = max(1, log_int(64, 4096) // 8) * 8
    K = max(1, log_int(64, 7168) // 8) * 8
    kind = rng.choice(["forward", "grad_x", "grad_w"])
    if kind == "grad_w" or T > 64:  # a training batch
        E = min(E, 64)
    if kind != "forward":
        T = min(T, 4096)
    return {"op": op, "kind": kind, "T": T, "k": min(k, E), "E": E, "N": N, "K": K,
            "out": rng.choice(["bf16", "f32"]), "pad": rng.choice([0, 0, 8, 64])}


# ----------------------------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------------------------
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_BLOCK = {"mx": 32, "nv": 16}


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, std, dtype):
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat = out.view(-1)
    for a in range(0, flat.numel(), 1 << 29):
        flat[a:a + (1 << 29)].normal_(0.0, std, generator=g)
    return out


def _tokens(g, T, K, pad, dtype):
    """Activations: normal, one channel in 64 eight times as large; rows inside rows of K + pad."""
    x = _normal(g, (T, K + pad), 1.0, dtype)
    x[:, ::64] *= 8.0
    return x[:, :K]


def _routing(g, T, k, E):
    """Each token's k experts, some experts more popular: (perm_src int32 [T k], its inverse dest, and
    offsets as a list)."""
    like = torch.randn(E, device=DEV, generator=g) * 0.5
    u = torch.rand(T, E, device=DEV, generator=g).clamp_(1e-7, 1.0 - 1e-7)
    idx = (like - torch.log(-torch.log(u))).topk(k, dim=1).indices.reshape(-1)
    perm = torch.sort(idx, stable=True).indices
    dest = torch.empty_like(perm)
    dest[perm] = torch.arange(T * k, device=DEV)
    counts = torch.bincount(idx, minlength=E).cpu().tolist()
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    return perm.to(torch.int32), dest.to(torch.int32), offsets


def _tiled_scales(s, rows_of_group):
    """Scale bytes [G * rows][C] in the order in which the library keeps them: tiles of 128 rows by 4
    columns, a group's first tile at (its first row) // 128 + its number, a tile's row r, column c at
    (r % 32) * 16 + r // 32 * 4 + c."""
    C = s.shape[1]
    G, kt = s.shape[0] // rows_of_group, (C + 3) // 4
    per = (rows_of_group + 127) // 128
    tiles = torch.zeros(s.shape[0] // 128 + G, kt, 512, dtype=torch.uint8, device=DEV)
    pad = torch.zeros(per * 128, kt * 4, dtype=torch.uint8, device=DEV)
    for e in range(G):
        pad[:rows_of_group, :C] = s[e * rows_of_group:(e + 1) * rows_of_group]
        t = pad.view(per, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).reshape(per, kt, 512)
        first = e * rows_of_group // 128 + e
        tiles[first:first + per] = t
    return tiles.view(-1)


def _prepare_quant(case, seed):
    g = _generator(seed)
    T, K, k, E = (case[n] for n in ("T", "K", "k", "E"))
    st = {"case": case, "x": _tokens(g, T, K, case["pad"], _DT[case["act"]])}
    st["perm"], st["dest"], st["offs"] = _routing(g, T, k, E)
    st["g"] = None
    if case["fmt"] == "nv":  # the factor that brings the tensor's largest block scale to 448
        st["g"] = (st["x"].abs().amax().float() / (6.0 * 448.0)).reshape(1)
    if own:
        from mixture_experts_ffn_gemm_gb300 import binding as B
        st["offsets"] = torch.tensor(st["offs"], dtype=torch.int32, device=DEV)
        st["cfg"] = B.make_micro_config(rows=T * k, K=K, format=case["fmt"], groups=E,
                                        dtype=_DT[case["act"]], ld=K + case["pad"], src_rows=T,
                                        copies=k)
        st["back"] = B.make_micro_config(rows=T * k, K=K, format=case["fmt"], groups=E,
                                         dtype=_DT[case["out"]])
        st["codes"], st["scales"] = B.alloc_micro(st["cfg"], DEV)
        st["ws"] = B.alloc_micro_workspace(st["cfg"], DEV)
        st["out"] = torch.empty(T * k, K, dtype=_DT[case["out"]], device=DEV)
    return st


def _prepare_micro(case, seed):
    g = _generator(seed)
    T, k, E, N, K, fmt = (case[n] for n in ("T", "k", "E", "N", "K", "fmt"))
    st = {"case": case, "x": _tokens(g, T, K, 0, torch.bfloat16)}
    st["perm"], st["dest"], st["offs"] = _routing(g, T, k, E)
    rows = N * (2 if case["swiglu"] else 1)
    st["w"] = torch.empty(E * rows, K // 2, dtype=torch.uint8, device=DEV)
    flat = st["w"].view(-1)
    for a in range(0, flat.numel(), 1 << 29):
        # two codes of a byte, each with a normal weight's histogram: 6 at the blocks' largest
        n = min(1 << 29, flat.numel() - a)
        v = torch.randn(n, 2, device=DEV, generator=g, dtype=torch.bfloat16).mul_(2.4)
        mag = torch.zeros(n, 2, dtype=torch.uint8, device=DEV)
        for t in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
            mag += v.abs() > t
        mag += (v < 0).to(torch.uint8) * 8
        flat[a:a + n] = mag[:, 0] + mag[:, 1] * 16
        del v, mag
    C = K // _BLOCK[fmt]
    st["gx"] = st["gw"] = None
    if fmt == "mx":  # exponents, 127 stands for 1: near K^-0.5 / 2
        mid = 127 - int(round(math.log2(2.0 * K ** 0.5)))
        st["s"] = torch.randint(mid - 1, mid + 2, (E * rows, C), device=DEV, generator=g).to(
            torch.uint8)
    else:  # e4m3 scales of 16 to 448, a factor for each expert
        f = torch.rand(E * rows, C, device=DEV, generator=g) * 432.0 + 16.0
        st["s"] = f.to(torch.float8_e4m3fn).view(torch.uint8)
        st["gw"] = (torch.rand(E, device=DEV, generator=g) + 0.5) * (K ** -0.5 / 600.0)
        st["gx"] = torch.full((1,), 42.0 / (6.0 * 448.0), device=DEV)
    if own:
        from mixture_experts_ffn_gemm_gb300 import binding as B
        st["offsets"] = torch.tensor(st["offs"], dtype=torch.int32, device=DEV)
        st["w_scales"] = _tiled_scales(st["s"], rows)
        st["qcfg"] = B.make_micro_config(rows=T * k, K=K, format=fmt, groups=E, src_rows=T,
                                         copies=k)
        st["codes"], st["scales"] = B.alloc_micro(st["qcfg"], DEV)
        st["cfg"] = B.make_micro_product_config(rows=T * k, E=E, N=N, K=K, format=fmt,
                                                out_dtype=_DT[case["out"]],
                                                swiglu=case["swiglu"])
        st["ws"] = B.alloc_micro_product_workspace(st["cfg"], DEV)
        st["out"] = torch.empty(T * k, N, dtype=_DT[case["out"]], device=DEV)
    return st


def _prepare_grouped(case, seed):
    g = _generator(seed)
    T, k, E, N, K, kind, pad = (case[n] for n in ("T", "k", "E", "N", "K", "kind", "pad"))
    R = T * k
    st = {"case": case}
    _, _, st["offs"] = _routing(g, T, k, E)
    x = dy = w = None
    if kind != "grad_x":
        x = _normal(g, (R, K + pad), 1.0, torch.bfloat16)[:, :K]
    if kind != "forward":
        dy = _normal(g, (R, N + pad), 0.1, torch.bfloat16)[:, :N]
    if kind != "grad_w":
        w = _normal(g, (E, N, K), K ** -0.5, torch.bfloat16)
    st["a"] = x if kind == "forward" else dy
    st["b"] = x if kind == "grad_w" else w
    if own:
        from mixture_experts_ffn_gemm_gb300 import binding as B
        st["offsets"] = torch.tensor(st["offs"], dtype=torch.int32, device=DEV)
        st["cfg"] = B.make_product_config(rows=R, E=E, N=N, K=K, kind=kind,
                                          out_dtype=_DT[case["out"]],
                                          ld_x=K if kind == "grad_x" else K + pad,
                                          ld_y=N if kind == "forward" else N + pad)
        st["ws"] = B.alloc_product_workspace(st["cfg"], DEV)
        shape = {"forward": (R, N), "grad_x": (R, K), "grad_w": (E, N, K)}[kind]
        st["out"] = torch.empty(shape, dtype=_DT[case["out"]], device=DEV)
    return st


def prepare(case, seed):
    return {"quant": _prepare_quant, "micro": _prepare_micro, "grouped": _prepare_grouped}[
        case["op"]](case, seed)


# ----------------------------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------------------------
_MAGS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _plain_values(x, fmt, g):
    """The values that x's codes and scales stand for, fp32 [T][K] (the quantisation in 64 bits: values
    next to a border between two codes, or two scales, stay on their side)."""
    T, K = x.shape
    v = x.double().reshape(T, K // _BLOCK[fmt], _BLOCK[fmt])
    amax = v.abs().amax(dim=2, keepdim=True)
    if fmt == "mx":
        _, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1)
        scale = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), (e - 3).clamp(-127, 127)),
                            torch.ones_like(amax))
    else:
        gd = g.double()
        # e4m3: three bits behind the leading one, from 2^-6 on; at most 448
        q = (amax / (6.0 * gd)).clamp(max=448.0)
        _, e = torch.frexp(q)
        step = torch.ldexp(torch.ones_like(q), (e - 1).clamp(min=-6) - 3)
        scale = torch.round(q / step) * step * gd
    y = v.abs() / torch.where(scale > 0, scale, torch.ones_like(scale))
    y = torch.where(scale > 0, y, torch.zeros_like(y))
    idx = ((y > 0.25).long() + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5)
           + (y > 5.0))
    mag = torch.tensor(_MAGS, device=x.device, dtype=torch.float64)[idx]
    return (torch.where(v < 0, -mag, mag) * scale).reshape(T, K).float()


def _plain_weight(codes, s, fmt, g):
    """4-bit codes [N][K / 2] and scale bytes [N][K / B] as fp32 [N][K]."""
    N, half = codes.shape
    c = torch.stack([codes & 15, codes >> 4], dim=2).view(N, 2 * half).int()
    lut = torch.tensor(_MAGS + tuple(-m for m in _MAGS), device=codes.device)
    v = lut[c].view(N, -1, _BLOCK[fmt])
    if fmt == "mx":
        scale = torch.ldexp(torch.ones(s.shape, device=s.device), s.int() - 127)
    else:
        scale = s.view(torch.float8_e4m3fn).float() * g
    return (v * scale[:, :, None]).view(N, 2 * half)


def _plain_quant(st):
    case = st["case"]
    v = _plain_values(st["x"], case["fmt"], st["g"]).to(_DT[case["out"]])
    return v[(st["perm"] // case["k"]).long()]


def _plain_micro(st):
    case = st["case"]
    N, fmt, offs = case["N"], case["fmt"], st["offs"]
    rows = N * (2 if case["swiglu"] else 1)
    x = _plain_values(st["x"], fmt, st["gx"])
    src = (st["perm"] // case["k"]).long()
    out = torch.empty(src.shape[0], N, dtype=_DT[case["out"]], device=x.device)
    for e in range(case["E"]):
        a, z = offs[e], offs[e + 1]
        if a == z:
            continue
        w = _plain_weight(st["w"][e * rows:(e + 1) * rows], st["s"][e * rows:(e + 1) * rows], fmt,
                          None if st["gw"] is None else st["gw"][e:e + 1])
        y = x[src[a:z]] @ w.t()
        if case["swiglu"]:
            gate, up = y.chunk(2, dim=1)
            y = gate * torch.sigmoid(gate) * up
        out[a:z] = y.to(out.dtype)
    return out


def _plain_grouped(st):
    case = st["case"]
    kind, offs, a, b = case["kind"], st["offs"], st["a"], st["b"]
    dt = _DT[case["out"]]
    parts = []
    for e in range(case["E"]):
        lo, hi = offs[e], offs[e + 1]
        if kind == "grad_w":
            parts.append((a[lo:hi].float().t() @ b[lo:hi].float()).to(dt))
        elif hi > lo:
            w = b[e].float()
            parts.append((a[lo:hi].float() @ (w.t() if kind == "forward" else w)).to(dt))
    return torch.stack(parts) if kind == "grad_w" else torch.cat(parts)


def run(state):
    st = state
    case = st["case"]
    op = case["op"]
    if not own:
        return {"quant": _plain_quant, "micro": _plain_micro, "grouped": _plain_grouped}[op](st)
    from mixture_experts_ffn_gemm_gb300 import binding as B
    if op == "quant":
        B.moe_micro_quantize(st["cfg"], st["x"], st["dest"], st["offsets"], st["g"], st["codes"],
                             st["scales"], st["ws"])
        B.moe_micro_dequantize(st["back"], st["codes"], st["scales"], st["offsets"], st["g"],
                               st["out"], st["ws"])
    elif op == "micro":
        B.moe_micro_quantize(st["qcfg"], st["x"], st["dest"], st["offsets"], st["gx"], st["codes"],
                             st["scales"], st["ws"])
        B.moe_micro_product(st["cfg"], st["offsets"], st["codes"], st["scales"], st["gx"], st["w"],
                            st["w_scales"], st["gw"], st["out"], st["ws"])
    else:
        B.moe_grouped_product(st["cfg"], st["offsets"], st["a"], st["b"], st["out"], st["ws"])
    return st["out"]


# ----------------------------------------------------------------------------------------------
# The definition in 64 bits
# ----------------------------------------------------------------------------------------------
def _exact_values(x, fmt, g):
    """Codes by the nearest of the eight magnitudes, the even code at equal distance."""
    T, K = x.shape
    B = _BLOCK[fmt]
    v = x.to(torch.float64).view(T, K // B, B) if x.is_contiguous() else \
        x.contiguous().to(torch.float64).view(T, K // B, B)
    top = v.abs().amax(-1)
    if fmt == "mx":
        p = torch.floor(torch.log2(top.clamp(min=1e-300)))
        p = torch.where(torch.pow(2.0, p) > top, p - 1, p)
        p = torch.where(torch.pow(2.0, p + 1) <= top, p + 1, p)
        S = torch.where(top > 0, torch.pow(2.0, (p - 2).clamp(-127, 127)), torch.ones_like(top))
    else:
        g = g.to(torch.float64)
        want = top / (6.0 * g)
        # every non-negative e4m3 number, and the nearest one
        codes = torch.arange(127, device=x.device, dtype=torch.uint8)
        grid = codes.view(torch.float8_e4m3fn).to(torch.float64)
        hi = torch.searchsorted(grid, want.contiguous()).clamp(max=126)
        lo = (hi - 1).clamp(min=0)
        dh, dl = (grid[hi] - want).abs(), (want - grid[lo]).abs()
        pick_hi = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
        S = torch.where(pick_hi, grid[hi], grid[lo]) * g
    unit = torch.where(S > 0, S, torch.full_like(S, math.inf))[..., None]
    y = v.abs() / unit
    best = torch.zeros_like(y)
    dist = y.clone()
    for i, m in enumerate(_MAGS[1:], 1):
        d = (y - m).abs()
        take = (d < dist) | ((d == dist) & (i % 2 == 0))
        best = torch.where(take, torch.full_like(best, m), best)
        dist = torch.where(take, d, dist)
    return (torch.sign(v) * best * S[..., None]).view(T, K)


def _exact_weight(codes, s, fmt, g):
    N, half = codes.shape
    lo = torch.remainder(codes, 16).to(torch.int64)
    hi = torch.div(codes, 16, rounding_mode="floor").to(torch.int64)
    table = torch.tensor([m * sgn for sgn in (1.0, -1.0) for m in _MAGS], dtype=torch.float64,
                         device=codes.device)
    w = torch.empty(N, half, 2, dtype=torch.float64, device=codes.device)
    w[:, :, 0] = table[lo]
    w[:, :, 1] = table[hi]
    w = w.view(N, 2 * half)
    if fmt == "mx":
        S = torch.pow(2.0, s.to(torch.float64) - 127.0)
    else:
        S = s.view(torch.float8_e4m3fn).to(torch.float64) * g.to(torch.float64)
    return w * S.repeat_interleave(_BLOCK[fmt], dim=1)


def _exact(case, st):
    op, offs = case["op"], st["offs"]
    if op == "quant":
        src = torch.div(st["perm"], case["k"], rounding_mode="floor").long()
        parts = [_exact_values(st["x"][a:a + 1024], case["fmt"], st["g"])
                 for a in range(0, case["T"], 1024)]
        return torch.cat(parts).index_select(0, src)
    if op == "grouped":
        kind, a, b = case["kind"], st["a"], st["b"]
        if kind == "grad_w":
            out = torch.zeros(case["E"], case["N"], case["K"], dtype=torch.float64, device=DEV)
        else:
            out = torch.zeros(offs[-1], case["N"] if kind == "forward" else case["K"],
                              dtype=torch.float64, device=DEV)
        for e in range(case["E"]):
            s = slice(offs[e], offs[e + 1])
            if offs[e] == offs[e + 1]:
                continue
            if kind == "forward":
                out[s] = torch.einsum("rk,nk->rn", a[s].double(), b[e].double())
            elif kind == "grad_x":
                out[s] = torch.einsum("rn,nk->rk", a[s].double(), b[e].double())
            else:
                out[e] = torch.einsum("rn,rk->nk", a[s].double(), b[s].double())
        return out
    N, fmt = case["N"], case["fmt"]
    per = N * (2 if case["swiglu"] else 1)
    src = torch.div(st["perm"], case["k"], rounding_mode="floor").long()
    x = torch.cat([_exact_values(st["x"][a:a + 1024], fmt, st["gx"])
                   for a in range(0, case["T"], 1024)])
    out = torch.zeros(offs[-1], N, dtype=torch.float64, device=DEV)
    for e in range(case["E"]):
        s = slice(offs[e], offs[e + 1])
        if offs[e] == offs[e + 1]:
            continue
        w = _exact_weight(st["w"][e * per:(e + 1) * per], st["s"][e * per:(e + 1) * per], fmt,
                          None if st["gw"] is None else st["gw"][e])
        rows = x.index_select(0, src[s])
        y = rows @ w[:N].T
        if case["swiglu"]:
            y = y / (1.0 + torch.exp(-y)) * (rows @ w[N:].T)
        out[s] = y
    return out


def exact(case, seed):
    global own
    keep, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = keep
    with torch.no_grad():
        return _exact(case, st)


# ----------------------------------------------------------------------------------------------
# What one pass cannot do without
# ----------------------------------------------------------------------------------------------
def work(case):
    T, k, E, K = case["T"], case["k"], case["E"], case["K"]
    R = T * k
    o = 4 if case["out"] == "f32" else 2
    if case["op"] == "quant":
        a = 4 if case["act"] == "f32" else 2
        coded = R * K // 2 + R * K // _BLOCK[case["fmt"]]
        # x once; codes and scales written and read back; the values written
        return {"bytes": T * K * a + 2 * coded + R * K * o + 4 * R, "flops": 4 * R * K}
    N = case["N"]
    used = E * (1.0 - (1.0 - k / E) ** T)  # the expected number of distinct experts
    if case["op"] == "micro":
        rows = N * (2 if case["swiglu"] else 1)
        per = 0.5 + 1.0 / _BLOCK[case["fmt"]]
        # the tokens' rows once, the selected experts' weights once, the output once
        return {"bytes": int(T * K * 2 + used * rows * K * per + R * N * o),
                "flops": 2 * R * rows * K}
    ins = {"forward": R * K * 2 + used * N * K * 2, "grad_x": R * N * 2 + used * N * K * 2,
           "grad_w": R * (N + K) * 2}[case["kind"]]
    outs = {"forward": R * N, "grad_x": R * K, "grad_w": E * N * K}[case["kind"]]
    return {"bytes": int(ins + outs * o), "flops": 2 * R * N * K}

"""Workloads of the few-token MoE layer and of the block join: their plain form, calls and inputs.

Two operators of a transformer block's FFN half are described here.

few   The whole mixture-of-experts layer for at most 16 tokens (serving: one new token of each of a
      few sequences): logits z = x W_r, s = sigmoid(z), the k largest s + b (ties to the lower
      expert), gates G = gate_scale s / sum of the selected s, SwiGLU experts
      E_i(x) = (SiLU(x W1_i) * (x W3_i)) W2_i, out = sum G_i E_i(x) + E_shared(x).  Latent form: the
      experts act on x W_down, and their sum passes an RMSNorm and W_up before the shared expert is
      added.  Expert weights: fp32, bf16, e4m3 with a scale per 128 x 128 block, or 4-bit integers
      with a bf16 scale per 32 input channels (the product rounded to bf16 is the weight).
join  What stands between two blocks: the branch's post-norm, its gate and scale, the residual sum
      and the norm that the next block starts with:
      r' = resid_scale r + branch_scale g RMSNorm(y) w_post,  n = RMSNorm(r') w_pre.

``own`` false: elementary torch operations.  ``own`` true: the library's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
GATE_SCALE = 2.827
EPS = 1e-6


def _few(name, T, d, E, k, I, shared=True, latent=0, w="bf16"):
    return {"name": name, "op": "few", "T": T, "d": d, "E": E, "k": k, "I": I, "shared": shared,
            "latent": latent, "w": w}


def _join(name, T, d, act="bf16", resid="bf16", post=True, gate="none", sigmoid=False, pre=True,
          pad=0):
    return {"name": name, "op": "join", "T": T, "d": d, "act": act, "resid": resid, "post": post,
            "gate": gate, "sigmoid": sigmoid, "pre": pre, "pad": pad}


def listed():
    return [
        # the smallest layer of the repository's configurations, two tokens: launch latency only
        _few("few_tiny_f32_t2", 2, 256, 16, 4, 128, w="f32"),
        # one token of one sequence through the full-size layer: nine experts' weights
        _few("few_k2_bf16_t1", 1, 7168, 384, 8, 2048),
        # a full group of sixteen sequences: about 110 of the 384 experts
        _few("few_k2_bf16_t16", 16, 7168, 384, 8, 2048),
        # four sequences through the latent layer (narrow experts, two more projections)
        _few("few_latent_bf16_t4", 4, 7168, 384, 8, 2048, latent=3584),
        # four sequences, experts stored as e4m3 with block scales
        _few("few_k2_fp8_t4", 4, 7168, 384, 8, 2048, w="fp8"),
        # one sequence, experts stored as 4-bit groups: a quarter of the bytes, the latency shows
        _few("few_k2_int4_t1", 1, 7168, 384, 8, 2048, w="int4"),
        # a small layer of ragged widths without a shared expert, an odd number of tokens
        _few("few_ragged_bf16_t7", 7, 2080, 60, 6, 736, shared=False),
        # one token between two blocks: launch latency only
        _join("join_t1", 1, 7168),
        # a decode batch, fp32 residual stream, a learned gate per channel
        _join("join_t128_channel", 128, 7168, resid="f32", gate="channel"),
        # a prompt of 16,384 tokens, both norms and a gate per channel
        _join("join_t16384_channel", 16384, 7168, gate="channel"),
        # an output gate per element through a sigmoid, rows inside a wider buffer, no post-norm
        _join("join_t4096_element", 4096, 7168, post=False, gate="element", sigmoid=True, pad=64),
        # odd width in fp32, a gate per token
        _join("join_f32_odd", 1999, 1001, act="f32", resid="f32", gate="token"),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    if rng.random() < 0.55:
        w = rng.choice(["bf16", "bf16", "fp8", "int4", "f32"])
        step = {"bf16": 32, "fp8": 128, "int4": 32, "f32": 16}[w]
        latent = 0
        T = rng.randint(1, 16)
        k = rng.randint(1, 8)
        E = max(k, log_int(4, 384))
        d = max(1, log_int(128, 7168) // step) * step
        I = max(1, log_int(128, 2048) // step) * step
        shared = rng.random() < 0.7
        if w == "bf16" and rng.random() < 0.3:
            latent = max(1, d // 2 // step) * step
        if w == "f32":  # the fp32 layer is for small models
            d, I = min(d, 2048), min(I, 1024)
        return {"op": "few", "T": T, "d": d, "E": E, "k": k, "I": I, "shared": shared,
                "latent": latent, "w": w}
    act = rng.choice(["bf16", "bf16", "f32"])
    d = log_int(64, 7168)
    if rng.random() < 0.7:
        d = max(8, d // 8 * 8)
    T = log_int(1, 16384 if act == "bf16" else 8192)
    gate = rng.choice(["none", "channel", "token", "element"])
    resid = "f32" if act == "f32" or rng.random() < 0.3 else "bf16"
    if gate == "element" or resid == "f32":  # more bytes a row
        T = max(1, T // 2)
    return {"op": "join", "T": T, "d": d, "act": act, "resid": resid,
            "post": rng.random() < 0.7, "gate": gate,
            "sigmoid": gate != "none" and rng.random() < 0.5, "pre": rng.random() < 0.8,
            "pad": rng.choice([0, 0, 1, 8, 64])}


# ----------------------------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------------------------
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


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


def _fp8_weights(g, n, rows, cols, std):
    q = torch.empty(n, rows, cols, dtype=torch.float8_e4m3fn, device=DEV)
    s = torch.empty(n, rows // 128, cols // 128, dtype=torch.float32, device=DEV)
    for i in range(n):
        m = torch.randn(rows // 128, 128, cols // 128, 128, device=DEV, generator=g) * std
        s[i] = m.abs().amax(dim=(1, 3)) / 448.0
        q[i] = (m / s[i][:, None, :, None]).clamp_(-448.0, 448.0).view(rows, cols).to(q.dtype)
    return q, s


def _int4_weights(g, n, rows, cols, std):
    """Codes of a normal distribution quantised with a step of its deviation / 2.2, a bf16 scale for
    each 32 input channels, eight codes to a word (code i in nibble i / 2 + 4 (i % 2))."""
    q = torch.empty(n, rows, cols // 2, dtype=torch.uint8, device=DEV)
    s = torch.empty(n, cols // 32, rows, dtype=torch.bfloat16, device=DEV)
    for i in range(n):
        c = torch.randn(rows, cols // 8, 8, device=DEV, generator=g).mul_(2.2).round_()
        u = c.clamp_(-8, 7).add_(8).to(torch.uint8)
        # byte j of a word: nibbles 2j and 2j + 1, which hold codes (0, 2), (4, 6), (1, 3), (5, 7)
        for j, (lo, hi) in enumerate(((0, 2), (4, 6), (1, 3), (5, 7))):
            q[i].view(rows, cols // 8, 4)[:, :, j] = u[:, :, lo] | (u[:, :, hi] << 4)
        s[i] = (torch.rand(cols // 32, rows, device=DEV, generator=g) * 0.4 + 0.8) * (std / 2.2)
    return q, s


def _prepare_few(case, seed):
    g = _generator(seed)
    T, d, E, k, I, L, w = (case[n] for n in ("T", "d", "E", "k", "I", "latent", "w"))
    de = L or d
    act = torch.float32 if w == "f32" else torch.bfloat16
    st = {"case": case}
    st["x"] = _normal(g, (T, d), 1.0, act)
    st["W_r"] = _normal(g, (E, d), 1.7 * d ** -0.5, torch.float32)
    st["b"] = torch.rand(E, device=DEV, generator=g) * 0.1 - 0.05
    for name in ("W13_scale", "W2_scale", "Ws13", "Ws2", "Ws13_scale", "Ws2_scale", "W_down",
                 "W_up"):
        st[name] = None
    if w in ("f32", "bf16"):
        st["W13"] = _normal(g, (E, 2 * I, de), de ** -0.5, act)
        st["W2"] = _normal(g, (E, de, I), I ** -0.5, act)
        if case["shared"]:
            st["Ws13"] = _normal(g, (2 * I, d), d ** -0.5, act)
            st["Ws2"] = _normal(g, (d, I), I ** -0.5, act)
    else:
        make = _fp8_weights if w == "fp8" else _int4_weights
        st["W13"], st["W13_scale"] = make(g, E, 2 * I, d, d ** -0.5)
        st["W2"], st["W2_scale"] = make(g, E, d, I, I ** -0.5)
        if case["shared"]:
            for name, rows, cols in (("Ws13", 2 * I, d), ("Ws2", d, I)):
                q, s = make(g, 1, rows, cols, cols ** -0.5)
                st[name], st[name + "_scale"] = q[0], s[0]
    if L:
        st["W_down"] = _normal(g, (L, d), d ** -0.5, act)
        st["W_up"] = _normal(g, (d, L), L ** -0.5, act)
    st["out"] = torch.empty(T, d, dtype=act, device=DEV)
    if own:
        from mixture_experts_ffn_gemm_gb300 import binding as B
        wdt = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn,
               "int4": torch.uint8}[w]
        st["cfg"] = B.make_config(T=T, d=d, E=E, k=k, I=I, n_shared=1 if case["shared"] else 0,
                                  d_latent=L, latent_norm=1 if L else 0, act_dtype=act,
                                  w_dtype=wdt, quant_block=32 if w == "int4" else 128,
                                  gate_scale=GATE_SCALE, rms_eps=EPS)
        st["ws"] = B.alloc_few_workspace(st["cfg"], DEV)
    return st


def _rows(g, T, d, pad, std, dtype):
    """T rows of d values inside rows of d + pad, as a slice of a wider buffer is."""
    return _normal(g, (T, d + pad), std, dtype)[:, :d]


def _prepare_join(case, seed):
    g = _generator(seed)
    T, d, pad = case["T"], case["d"], case["pad"]
    act, rdt = _DT[case["act"]], _DT[case["resid"]]
    st = {"case": case, "resid_scale": 1.0, "branch_scale": 0.22}
    st["resid"] = _rows(g, T, d, pad, 2.0, rdt)
    st["branch"] = _rows(g, T, d, pad, 0.7, act)

    def weight():
        return (torch.rand(d, device=DEV, generator=g) * 0.4 + 0.8).to(act)

    st["post_w"] = weight() if case["post"] else None
    st["pre_w"] = weight() if case["pre"] else None
    gate = case["gate"]
    st["gate"] = (None if gate == "none" else _normal(g, (d,), 1.0, act) if gate == "channel" else
                  _normal(g, (T,), 1.0, act) if gate == "token" else _rows(g, T, d, pad, 1.0, act))
    st["resid_out"] = torch.empty(T, d, dtype=rdt, device=DEV)
    st["normed"] = torch.empty(T, d, dtype=act, device=DEV) if case["pre"] else None
    if own:
        from mixture_experts_ffn_gemm_gb300 import binding as B
        st["cfg"] = B.make_join_config(
            T=T, d=d, act_dtype=act, resid_dtype=rdt, gate=gate, gate_sigmoid=case["sigmoid"],
            resid_scale=st["resid_scale"], branch_scale=st["branch_scale"], rms_eps=EPS,
            ld_resid=d + pad, ld_branch=d + pad, ld_gate=d + pad if gate == "element" else 0)
    return st


def prepare(case, seed):
    return _prepare_few(case, seed) if case["op"] == "few" else _prepare_join(case, seed)


# ----------------------------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------------------------
def _unpack_int4(q, s):
    """[R][C/2] packed, [C/32][R] scales -> the bf16 weights as fp32 [R][C]."""
    R, C = q.shape[0], q.shape[1] * 2
    words = q.view(torch.int32)  # [R][C/8]
    codes = torch.stack([(words >> (4 * (i // 2 + 4 * (i % 2)))) & 15 for i in range(8)], dim=2)
    w = (codes.view(R, C // 32, 32) - 8).float() * s.t().float()[:, :, None]
    return w.view(R, C).to(torch.bfloat16).float()


def _weight(q, s, kind, e=None):
    """One weight matrix in fp32; e: a one-element index tensor into stacked weights."""
    if e is not None:
        raw = q.view(torch.uint8) if kind == "fp8" else q
        q = raw.index_select(0, e)[0]
        q = q.view(torch.float8_e4m3fn) if kind == "fp8" else q
        s = None if s is None else s.index_select(0, e)[0]
    if kind == "fp8":
        R, C = q.shape
        blk = q.float().view(R // 128, 128, C // 128, 128) * s[:, None, :, None]
        return blk.view(R, C)
    if kind == "int4":
        return _unpack_int4(q, s)
    return q.float()


def _swiglu(x, w13, w2):
    g, u = (x @ w13.t()).chunk(2, dim=-1)
    return (g * torch.sigmoid(g) * u) @ w2.t()


def _plain_few(st):
    case = st["case"]
    T, k, kind = case["T"], case["k"], case["w"]
    x = st["x"].float()
    # the router in 64 bits: keys next to the border of the selection stay on their side
    s = torch.sigmoid(st["x"].double() @ st["W_r"].double().t())
    order = torch.sort(s + st["b"].double(), dim=1, descending=True, stable=True).indices
    idx = order[:, :k]
    gates = s.gather(1, idx)
    gates = (GATE_SCALE * gates / gates.sum(dim=1, keepdim=True)).float()
    xe = x @ st["W_down"].float().t() if case["latent"] else x
    y = torch.zeros_like(xe)
    for t in range(T):
        for j in range(k):
            e = idx[t, j:j + 1]
            w13 = _weight(st["W13"], st["W13_scale"], kind, e)
            w2 = _weight(st["W2"], st["W2_scale"], kind, e)
            y[t:t + 1] += gates[t, j] * _swiglu(xe[t:t + 1], w13, w2)
    if case["latent"]:
        y = y / torch.sqrt((y * y).mean(dim=1, keepdim=True) + EPS)
        y = y @ st["W_up"].float().t()
    if case["shared"]:
        y = y + _swiglu(x, _weight(st["Ws13"], st["Ws13_scale"], kind),
                        _weight(st["Ws2"], st["Ws2_scale"], kind))
    return y.to(st["x"].dtype)


def _plain_join(st):
    case = st["case"]
    v = st["branch"].float()
    if st["post_w"] is not None:
        v = v / torch.sqrt((v * v).mean(dim=1, keepdim=True) + EPS) * st["post_w"].float()
    if st["gate"] is not None:
        g = st["gate"].float()
        g = torch.sigmoid(g) if case["sigmoid"] else g
        v = v * (g[:, None] if case["gate"] == "token" else g)
    r = st["resid_scale"] * st["resid"].float() + st["branch_scale"] * v
    if st["pre_w"] is None:
        return [r.to(st["resid"].dtype)]
    n = r / torch.sqrt((r * r).mean(dim=1, keepdim=True) + EPS) * st["pre_w"].float()
    return [r.to(st["resid"].dtype), n.to(st["branch"].dtype)]


def run(state):
    st = state
    if st["case"]["op"] == "few":
        if not own:
            return _plain_few(st)
        from mixture_experts_ffn_gemm_gb300 import binding as B
        B.moe_forward_few(st["cfg"], st["x"], st["W_r"], st["b"], st["W13"], st["W2"],
                          st["W13_scale"], st["W2_scale"], st["Ws13"], st["Ws2"],
                          st["Ws13_scale"], st["Ws2_scale"], st["W_down"], st["W_up"], st["out"],
                          st["ws"])
        return st["out"]
    if not own:
        return _plain_join(st)
    from mixture_experts_ffn_gemm_gb300 import binding as B
    B.moe_block_join(st["cfg"], st["resid"], st["branch"], st["post_w"], st["gate"], st["pre_w"],
                     st["resid_out"], st["normed"])
    return [st["resid_out"]] if st["normed"] is None else [st["resid_out"], st["normed"]]


# ----------------------------------------------------------------------------------------------
# The definition in 64 bits
# ----------------------------------------------------------------------------------------------
def _dequant64(q, s, kind):
    if kind == "fp8":
        scale = s.double().repeat_interleave(128, dim=0).repeat_interleave(128, dim=1)
        return q.to(torch.float64) * scale
    if kind == "int4":
        R, half = q.shape
        by = q.view(R, half // 4, 4).to(torch.int64)
        word = by[:, :, 0] + by[:, :, 1] * 256 + by[:, :, 2] * 65536 + by[:, :, 3] * 16777216
        out = torch.empty(R, half // 4, 8, dtype=torch.float64, device=q.device)
        for i in range(8):
            nibble = i // 2 + 4 * (i % 2)
            out[:, :, i] = (torch.div(word, 16 ** nibble, rounding_mode="floor") % 16 - 8).double()
        out = out.view(R, half * 2)
        scale = s.double().t().repeat_interleave(32, dim=1)
        # 4-bit times 8-bit significands: the product is exact in 64 and in 32 bits
        return (out * scale).float().to(torch.bfloat16).double()
    return q.double()


def _exact_few(case, st):
    x = st["x"].double()
    T, k, kind, I = case["T"], case["k"], case["w"], case["I"]

    def mlp(v, w13, w2):
        a = w13 @ v
        gate, up = a[:I], a[I:]
        return w2 @ (gate / (1.0 + torch.exp(-gate)) * up)

    score = 1.0 / (1.0 + torch.exp(-(x @ st["W_r"].double().T)))
    key = (score + st["b"].double()).cpu().tolist()
    score = score.cpu().tolist()
    xe = x @ st["W_down"].double().T if case["latent"] else x
    y = torch.zeros(T, xe.shape[1], dtype=torch.float64, device=DEV)
    users = {}
    for t in range(T):
        chosen = sorted(range(case["E"]), key=lambda e: (-key[t][e], e))[:k]
        total = sum(score[t][e] for e in chosen)
        for e in chosen:
            users.setdefault(e, []).append((t, GATE_SCALE * score[t][e] / total))
    for e, toks in users.items():
        scales = [None if st[n] is None else st[n][e] for n in ("W13_scale", "W2_scale")]
        w13 = _dequant64(st["W13"][e], scales[0], kind)
        w2 = _dequant64(st["W2"][e], scales[1], kind)
        for t, gate in toks:
            y[t] += gate * mlp(xe[t], w13, w2)
    if case["latent"]:
        y = y * torch.rsqrt(y.pow(2).sum(dim=1, keepdim=True) / y.shape[1] + EPS)
        y = y @ st["W_up"].double().T
    if case["shared"]:
        w13 = _dequant64(st["Ws13"], st["Ws13_scale"], kind)
        w2 = _dequant64(st["Ws2"], st["Ws2_scale"], kind)
        for t in range(T):
            y[t] += mlp(x[t], w13, w2)
    return y


def _exact_join(case, st):
    out = []
    T, d = case["T"], case["d"]
    for a in range(0, T, 4096):  # rows in pieces
        z = min(T, a + 4096)
        y = st["branch"][a:z].double()
        if case["post"]:
            y = y * torch.rsqrt(y.pow(2).sum(1) / d + EPS)[:, None] * st["post_w"].double()
        if case["gate"] != "none":
            g = st["gate"].double()
            if case["gate"] == "token":
                g = g[a:z].view(-1, 1)
            elif case["gate"] == "element":
                g = g[a:z]
            y = y * (1.0 / (1.0 + torch.exp(-g)) if case["sigmoid"] else g)
        r = st["resid_scale"] * st["resid"][a:z].double() + st["branch_scale"] * y
        n = None
        if case["pre"]:
            n = r * torch.rsqrt(r.pow(2).sum(1) / d + EPS)[:, None] * st["pre_w"].double()
        out.append((r, n))
    r = torch.cat([p[0] for p in out])
    return [r, torch.cat([p[1] for p in out])] if case["pre"] else [r]


def exact(case, seed):
    global own
    keep, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = keep
    with torch.no_grad():
        return _exact_few(case, st) if case["op"] == "few" else _exact_join(case, st)


# ----------------------------------------------------------------------------------------------
# What one pass cannot do without
# ----------------------------------------------------------------------------------------------
def work(case):
    T, d = case["T"], case["d"]
    if case["op"] == "join":
        a, r = (4 if case["act"] == "f32" else 2), (4 if case["resid"] == "f32" else 2)
        per_row = d * (2 * r + a + (a if case["pre"] else 0))
        vec = d * a * (int(case["post"]) + int(case["pre"]))
        gate = {"none": 0, "channel": d * a, "token": T * a, "element": T * d * a}[case["gate"]]
        flops = T * d * (3 + (4 if case["post"] else 0) + (4 if case["pre"] else 0))
        return {"bytes": T * per_row + vec + gate, "flops": flops}
    E, k, I, L = case["E"], case["k"], case["I"], case["latent"]
    de = L or d
    per = {"f32": 4.0, "bf16": 2.0, "fp8": 1.0 + 4.0 / 16384, "int4": 0.5 + 2.0 / 32}[case["w"]]
    a = 4 if case["w"] == "f32" else 2
    experts = E * (1.0 - (1.0 - k / E) ** T)  # the expected number of distinct experts
    shared = 1 if case["shared"] else 0
    nbytes = (experts * 3 * de * I * per + shared * 3 * d * I * per + E * d * 4 + E * 4
              + 2 * T * d * a + 2 * L * d * a)
    flops = 2.0 * T * (k * 3 * de * I + shared * 3 * d * I + E * d + 2 * L * d)
    return {"bytes": int(nbytes), "flops": int(flops)}

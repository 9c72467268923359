"""GPU tests of the whole layer for a few tokens (moe_forward_few) against a plain implementation of
its equations in 64 bits on the stored weights.

Tolerances.  Output rounding: at most half a step, 2^-8 |v| for bf16, 2^-24 |v| for fp32.  Before
it, relative to the rms of the output row: values held between the products keep 16 bits or more
(relative 2^-17 each, independent, so their sum stays below 5 sigma = 2^-14.5), fp32 sums of K <= 2^14
terms (2^-24 sqrt(K) = 2^-17 when rounded, 2^-24 K / 16 = 2^-14 when every partial sum of 16 terms
is truncated), twice over for the two products: below 2^-12 for bf16, doubled to 2^-11.  fp32: sums
only, 2^-24 sqrt(K) times 4, K <= 2^12: 2^-16.
Tokens whose k-th and (k+1)-th keys lie within 1e-5 are not compared (their choice may differ)."""
from dataclasses import replace

import pytest
import torch

from mixture_experts_ffn_gemm_gb300 import binding as B
from mixture_experts_ffn_gemm_gb300 import synthetic as S

pytestmark = pytest.mark.gpu

BASE = S.WORKLOADS["tiny_fp32"]


def _workload(kind, T, d=256, E=16, k=4, I=128, shared=1, latent=0):
    return replace(BASE, name=f"few_{kind}", act="f32" if kind == "f32" else "bf16",
                   fp8=kind == "fp8", int4=kind == "int4", quant_block=32 if kind == "int4" else 128,
                   T=T, d=d, E=E, k=k, I=I, I_shared=I, n_shared=shared, d_latent=latent,
                   latent_norm=1 if latent else 0)


def _w64(q, s):
    if q.dtype == torch.float8_e4m3fn:
        return q.double() * s.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    if q.dtype == torch.uint8:
        by = q.view(q.shape[0], -1, 4).long()
        word = by[..., 0] | by[..., 1] << 8 | by[..., 2] << 16 | by[..., 3] << 24
        u = torch.stack([word >> 4 * (i // 2 + 4 * (i % 2)) & 15 for i in range(8)], -1)
        w = (u.view(q.shape[0], -1) - 8).double() * s.double().t().repeat_interleave(32, 1)
        return w.to(torch.bfloat16).double()  # the product is exact in 64 bits: one rounding
    return q.double()


def reference(L):
    """(out [T][d] fp64, key margin [T]) of a synthetic layer."""
    w, x = L.w, L.x.double()

    def scale(s, e):
        return None if s is None else s[e]

    def mlp(v, w13, w2):
        g, u = (w13 @ v).chunk(2)
        return w2 @ (g * torch.sigmoid(g) * u)

    sig = torch.sigmoid(x @ L.W_r.double().t())
    key = sig + L.b.double()
    key = torch.where(key.isnan(), torch.full_like(key, -float("inf")), key)
    srt = torch.sort(key, dim=1, descending=True, stable=True)
    idx = srt.indices[:, :w.k]
    margin = (srt.values[:, w.k - 1] - srt.values[:, w.k] if w.k < w.E
              else torch.full((x.shape[0],), 1.0, device=x.device))
    g = sig.gather(1, idx)
    g = w.gate_scale * g / g.sum(1, keepdim=True)
    xe = x @ L.W_down.double().t() if w.d_latent else x
    y = torch.zeros(x.shape[0], w.d_expert, dtype=torch.float64, device=x.device)
    for e in idx.unique().tolist():
        w13, w2 = _w64(L.W13[e], scale(L.W13_scale, e)), _w64(L.W2[e], scale(L.W2_scale, e))
        for t, j in (idx == e).nonzero().tolist():
            y[t] += g[t, j] * mlp(xe[t], w13, w2)
    if w.d_latent:
        if w.latent_norm:
            y = y / torch.sqrt((y * y).mean(1, keepdim=True) + w.rms_eps)
        y = y @ L.W_up.double().t()
    if w.n_shared:
        w13, w2 = _w64(L.Ws13, L.Ws13_scale), _w64(L.Ws2, L.Ws2_scale)
        for t in range(x.shape[0]):
            y[t] += mlp(x[t], w13, w2)
    return y, margin


def few(L, stream=None, ws=None, out=None):
    cfg = B.config_for(L.w, T=L.x.shape[0])
    if ws is None:
        ws = B.alloc_few_workspace(cfg)
    if out is None:
        out = torch.full((L.x.shape[0], L.w.d), float("nan"), dtype=L.x.dtype, device="cuda")
    B.moe_forward_few(cfg, L.x, *B.layer_weights(L), out, ws, stream=stream)
    return out, ws


def compare(out, ref, margin):
    eps, between = (2.0 ** -24, 2.0 ** -16) if out.dtype == torch.float32 else (2.0 ** -8, 2.0 ** -11)
    rms = ref.pow(2).mean(1, keepdim=True).sqrt()
    err = (out.double() - ref).abs()
    bad = (err > eps * ref.abs() + between * rms) | ~out.double().isfinite()
    bad &= (margin >= 1e-5)[:, None]
    assert not bad.any(), (int(bad.sum()), float((err / rms)[bad].max()))
    assert (margin >= 1e-5).any()


def check(w, seed=0):
    L = S.make_layer(w, seed=seed, device="cuda")
    out, ws = few(L)
    assert B.moe_device_status(ws) == B.MOE_OK
    compare(out, *reference(L))
    return L, out


@pytest.mark.parametrize("T", [1, 2, 3, 5, 8, 9, 15, 16])
@pytest.mark.parametrize("kind", ["f32", "bf16", "fp8", "int4"])
def test_every_token_count(cuda_device, kind, T):
    check(_workload(kind, T), seed=T)


SHAPES = [  # widths that do not fill a tile, a chunk of the weight stream or the grid
    ("f32", dict(d=16, E=1, k=1, I=16)), ("f32", dict(d=48, E=5, k=5, I=80)),
    ("bf16", dict(d=32, E=1, k=1, I=32)), ("bf16", dict(d=96, E=7, k=7, I=160)),
    ("bf16", dict(d=1056, E=33, k=3, I=32)), ("bf16", dict(d=32, E=40, k=2, I=1120)),
    ("bf16", dict(d=2080, E=60, k=6, I=736)), ("bf16", dict(d=5152, E=3, k=2, I=2080)),
    ("fp8", dict(d=128, E=2, k=1, I=128)), ("fp8", dict(d=1152, E=9, k=4, I=640)),
    ("fp8", dict(d=2176, E=20, k=5, I=896)),
    ("int4", dict(d=32, E=2, k=2, I=32)), ("int4", dict(d=2080, E=12, k=3, I=736)),
    ("int4", dict(d=96, E=200, k=32, I=160)), ("bf16", dict(d=64, E=1023, k=32, I=64)),
]


@pytest.mark.parametrize("shared", [0, 1])
@pytest.mark.parametrize("kind,shape", SHAPES)
def test_ragged_widths(cuda_device, kind, shape, shared):
    check(_workload(kind, 7, shared=shared, **shape), seed=3)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("shared", [0, 1])
@pytest.mark.parametrize("T,d,latent,I", [(1, 256, 128, 128), (4, 512, 1056 // 2 // 32 * 32, 96),
                                          (16, 992, 480, 224)])
def test_latent(cuda_device, kind, T, d, latent, I, shared):
    check(_workload(kind, T, d=d, latent=latent, I=I, shared=shared), seed=5)


def test_latent_without_norm(cuda_device):
    check(replace(_workload("bf16", 3, latent=128), latent_norm=0), seed=6)


@pytest.mark.parametrize("name,T", [("k2_decode_bf16", 1), ("k2_decode_bf16", 16),
                                    ("k3_latent_bf16", 2), ("k2_fp8", 3), ("k2_int4_decode", 2)])
def test_full_width_fewer_experts(cuda_device, name, T):
    """The layer's full widths over 24 experts."""
    check(replace(S.WORKLOADS[name], T=T, E=24, x_dist="normal", w_init="fan_in"), seed=7)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
def test_all_tokens_on_the_same_experts(cuda_device, kind):
    """Equal tokens: every selected expert has all 16 rows."""
    L = S.make_layer(_workload(kind, 16, E=64, k=2), seed=8, device="cuda")
    L.x[:] = L.x[:1]
    out, _ = few(L)
    compare(out, *reference(L))
    assert (out == out[:1]).all()


def test_ties_and_disabled_experts(cuda_device):
    """Equal keys go to the lower index; experts with a bias of -infinity, the type's lowest value or
    NaN are chosen last."""
    w = _workload("f32", 4, E=12, k=3)
    L = S.make_layer(w, seed=9, device="cuda")
    L.W_r.zero_()
    L.b.copy_(torch.tensor([-float("inf"), 0.1, float("nan"), 0.2, 0.1, 0.1,
                            torch.finfo(torch.float32).min, 0.0, 0.0, 0.0, 0.0, 0.1]))
    out, _ = few(L)
    ref, _ = reference(L)  # experts 3, 1, 4
    compare(out, ref, torch.ones(4, device="cuda"))
    L.b.fill_(-float("inf"))
    out, _ = few(L)
    ref, _ = reference(L)  # nothing left: experts 0, 1, 2
    compare(out, ref, torch.ones(4, device="cuda"))


@pytest.mark.parametrize("kind", ["f32", "bf16", "fp8", "int4"])
def test_bad_values_stay_in_their_token(cuda_device, kind):
    """A token of NaN or infinities, and NaN in experts that only some tokens use, leave the other
    tokens' bits as they were."""
    L = S.make_layer(_workload(kind, 6, E=32, k=2), seed=10, device="cuda")
    clean, _ = few(L)
    clean = clean.clone()
    L.x[1] = float("nan")
    L.x[4] = float("inf")
    out, ws = few(L)
    assert B.moe_device_status(ws) == B.MOE_OK
    keep = torch.tensor([0, 2, 3, 5], device="cuda")
    assert torch.equal(out[keep], clean[keep])
    assert out[1].isnan().all()
    L = S.make_layer(_workload(kind, 6, E=32, k=2), seed=10, device="cuda")
    sig = torch.sigmoid(L.x.double() @ L.W_r.double().t()) + L.b.double()
    idx = sig.topk(2, dim=1).indices
    e = int(idx[0, 0])
    for m, s in ((L.W13, L.W13_scale), (L.W2, L.W2_scale)):
        if s is not None:
            s[e] = float("nan")
        else:
            m[e] = float("inf")
    out, _ = few(L)
    users = (idx == e).any(1)
    assert users.any() and not users.all()
    assert torch.equal(out[~users], clean[~users])
    assert out[users].isnan().any()


@pytest.mark.parametrize("kind", ["f32", "bf16", "fp8", "int4"])
def test_equal_calls_give_equal_bits_on_any_stream(cuda_device, kind):
    L = S.make_layer(_workload(kind, 11, d=512, E=24, I=384), seed=11, device="cuda")
    first, ws = few(L)
    first = first.clone()
    ws.fill_(0xA5)  # a workspace that no call has used
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(20):
        out = torch.full_like(first, float("nan"))
        side.wait_stream(torch.cuda.current_stream())
        out, _ = few(L, stream=side, ws=ws, out=out)
        side.synchronize()
        assert torch.equal(out, first)


def test_graph_replay_reads_the_new_tokens(cuda_device):
    L = S.make_layer(_workload("bf16", 4, d=512, E=24, I=384), seed=12, device="cuda")
    out, ws = few(L)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        few(L, ws=ws, out=out)
    for seed in (1, 2):
        L.x.copy_(torch.randn(L.x.shape, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        compare(out, *reference(L))
    assert B.moe_device_status(ws) == B.MOE_OK


def test_close_to_the_staged_layer(cuda_device):
    """moe_forward rounds h to bf16 (2^-9 of each, independent): 5 sigma of it, 2^-6.7 rms, and the
    two output roundings."""
    L = S.make_layer(_workload("bf16", 16, d=512, E=24, I=384), seed=13, device="cuda")
    out, _ = few(L)
    staged, _, _ = B.forward_layer(L)
    rms = staged.double().pow(2).mean().sqrt()
    err = (out.double() - staged.double()).abs()
    assert (err <= 2.0 ** -7 * staged.double().abs() + 2.0 ** -6.7 * rms).all()


def test_zero_tokens_and_one_launch(cuda_device):
    L = S.make_layer(_workload("bf16", 4), seed=14, device="cuda")
    cfg = B.config_for(L.w, T=0)
    ws = B.alloc_few_workspace(cfg)
    B.moe_forward_few(cfg, L.x[:0], *B.layer_weights(L), L.x[:0].clone(), ws)
    B.moe_reset_launch_count()
    few(L)
    assert B.moe_launch_count() == 1


def test_every_e4m3_code(cuda_device):
    """Weights of every finite e4m3 code, subnormals and both zeros among them."""
    L = S.make_layer(_workload("fp8", 3, d=256, E=4, k=2, I=128), seed=15, device="cuda")
    codes = torch.arange(256, device="cuda", dtype=torch.int16)
    codes = codes[(codes & 0x7F) != 0x7F].to(torch.uint8)
    g = torch.Generator(device="cuda").manual_seed(1)
    for m, s in ((L.W13, L.W13_scale), (L.W2, L.W2_scale), (L.Ws13, L.Ws13_scale),
                 (L.Ws2, L.Ws2_scale)):
        pick = torch.randint(0, codes.numel(), m.shape, generator=g, device="cuda")
        m.view(torch.uint8).copy_(codes[pick])
        s.copy_(torch.rand(s.shape, generator=g, device="cuda") * 2e-3)
    out, _ = few(L)
    compare(out, *reference(L))


@pytest.mark.parametrize("tokens", [3, 12])
def test_e4m3_nan_codes(cuda_device, tokens):
    """A NaN code makes the tokens of its expert NaN (W2: in its feature), the others keep their bits."""
    def run(edit):
        L = S.make_layer(_workload("fp8", tokens, d=256, E=32, k=2, I=128), seed=16, device="cuda")
        key = torch.sigmoid(L.x.double() @ L.W_r.double().t()) + L.b.double()
        idx = key.topk(2, dim=1).indices
        e = int(idx[0, 0])
        edit(L, e)
        return few(L)[0], (idx == e).any(1)

    clean, users = run(lambda L, e: None)
    assert users.any() and not users.all()

    def w13(L, e):
        L.W13.view(torch.uint8)[e, 200, 77] = 0xFF

    out, _ = run(w13)
    assert out[users].isnan().all() and torch.equal(out[~users], clean[~users])

    def w2(L, e):
        L.W2.view(torch.uint8)[e, 201, 3] = 0x7F

    out, _ = run(w2)
    other = torch.arange(256, device="cuda") != 201
    assert out[users][:, 201].isnan().all() and torch.equal(out[~users], clean[~users])
    assert torch.equal(out[:, other], clean[:, other])


def test_int4_scales_of_all_sizes(cuda_device):
    """Scales from subnormal to large, and zero: the weight is the product rounded to bf16."""
    L = S.make_layer(_workload("int4", 2, d=256, E=4, k=2, I=128), seed=17, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    for m, s in ((L.W13, L.W13_scale), (L.W2, L.W2_scale), (L.Ws13, L.Ws13_scale),
                 (L.Ws2, L.Ws2_scale)):
        m.copy_(torch.randint(0, 256, m.shape, generator=g, device="cuda").to(torch.uint8))
        e = torch.randint(-12, 0, s.shape, generator=g, device="cuda").float()
        s.copy_(torch.exp2(e) * (1 + torch.rand(s.shape, generator=g, device="cuda")))
        s.view(-1)[::7] = 0
        s.view(-1)[::11] = 1e-39
    out, _ = few(L)
    compare(out, *reference(L))


@pytest.mark.parametrize("scale", [1e-6, 1e6])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
def test_small_and_large_activations(cuda_device, kind, scale):
    """The 16 bits of h do not depend on its size."""
    L = S.make_layer(_workload(kind, 4), seed=18, device="cuda")
    L.x.mul_(scale)
    L.W_r.div_(scale)
    out, _ = few(L)
    compare(out, *reference(L))


def test_64_bit_weight_offsets(cuda_device):
    """Experts past 2^32 bytes of stacked weights."""
    w = replace(S.WORKLOADS["k2_decode_bf16"], T=2, E=100, k=2, w_init="fan_in")
    L = S.make_layer(w, seed=19, device="cuda")
    L.b.fill_(-2.0)
    L.b[-3:] = 2.0  # the last experts only
    out, _ = few(L)
    compare(out, *reference(L))


@pytest.mark.parametrize("kind,E", [("f32", 40), ("bf16", 1023), ("fp8", 64), ("int4", 33)])
def test_most_pairs(cuda_device, kind, E):
    """16 tokens of 32 experts each: 512 pairs."""
    check(_workload(kind, 16, d=128, E=E, k=32, I=128), seed=20)


@pytest.mark.parametrize("lo,hi", [(-12, -5), (-133, -120), (-6, -4), (100, 104)])
def test_int4_scales_of_a_range(cuda_device, lo, hi):
    """Scales of one range throughout: ordinary ones, subnormals, those about 2^-5, large ones."""
    L = S.make_layer(_workload("int4", 3, d=256, E=4, k=2, I=128), seed=18, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    for m, s in ((L.W13, L.W13_scale), (L.Ws13, L.Ws13_scale)):
        # the gate's rows keep ordinary scales: the output is of the other rows' size
        m.copy_(torch.randint(0, 256, m.shape, generator=g, device="cuda").to(torch.uint8))
        up = s[..., s.shape[-1] // 2:]
        e = torch.randint(lo, hi, up.shape, generator=g, device="cuda").double()
        up.copy_(torch.exp2(e) * (1 + torch.rand(up.shape, generator=g, device="cuda")))
    out, _ = few(L)
    compare(out, *reference(L))

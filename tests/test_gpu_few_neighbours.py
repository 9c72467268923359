"""A token of moe_forward_few beside other tokens: within the layer's tolerance of the formula whoever
shares its experts.  With bf16 activations the order of a token's sums, and so its last bits, may follow
the other tokens' experts (the planes of h in one product for up to four tokens of an expert, in turn
above; other cuts of the channels; other warps), so bits are not compared there; the fp32 layer's order
follows the number of tokens alone."""
import pytest
import torch

from test_gpu_few import _workload, compare, few, reference

from mixture_experts_ffn_gemm_gb300 import binding as B
from mixture_experts_ffn_gemm_gb300 import synthetic as S

pytestmark = pytest.mark.gpu

E, K = 16, 3
KINDS = [("f32", 0), ("bf16", 0), ("bf16", 128), ("fp8", 0), ("int4", 0)]


def _layer(kind, latent, users, seed):
    """`users` tokens that share expert 0 and three that do not; the choice is far from every border."""
    T = users + 3
    L = S.make_layer(_workload(kind, T, E=E, k=K, latent=latent), seed=seed, device="cuda")
    g = torch.Generator().manual_seed(seed)
    L.W_r.zero_()
    L.W_r[torch.arange(E), torch.arange(E)] = 8.0
    L.b.zero_()
    for t in range(T):
        others = (torch.randperm(E - 1, generator=g) + 1)[:K].tolist()
        L.x[t, :E] = -1.0
        for j, e in enumerate(([0] if t < users else []) + others):
            if j < K:
                L.x[t, e] = 1.0 + j / 16  # scores of the chosen from 0.9997, of the others below 0.001
    return L


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("users", [1, 4, 5, 8, 9, 13])
@pytest.mark.parametrize("kind,latent", KINDS)
def test_experts_of_any_number_of_tokens(cuda_device, kind, latent, users, seed):
    L = _layer(kind, latent, users, seed)
    ref, margin = reference(L)
    assert (margin > 0.5).all()
    out, ws = few(L)
    compare(out, ref, margin)
    tokens = L.x.clone()
    for t in (0, users - 1, users + 2):  # the same tokens alone
        L.x = tokens[t:t + 1].contiguous()
        alone, ws = few(L)
        compare(alone, ref[t:t + 1], margin[t:t + 1])
        assert B.moe_device_status(ws) == B.MOE_OK


@pytest.mark.parametrize("kind,latent", KINDS)
def test_replaced_neighbours(cuda_device, kind, latent):
    """Tokens that stay while others change their experts, over seeds."""
    for seed in range(12):
        L = S.make_layer(_workload(kind, 6, E=32, k=4, latent=latent), seed=seed, device="cuda")
        first = few(L)[0].clone()
        compare(first, *reference(L))
        g = torch.Generator().manual_seed(100 + seed)
        stay = torch.tensor([0, 2, 3, 5], device="cuda")
        for t in (1, 4):
            L.x[t] = torch.randn(L.x.shape[1], generator=g)
        out = few(L)[0]
        compare(out, *reference(L))
        if kind == "f32":
            assert torch.equal(out[stay], first[stay])

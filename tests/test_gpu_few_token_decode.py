"""The decode example: joins and layers together, eager and captured, against 64 bits.

Tolerances.  A block adds scale * gate * RMSNorm(y) w_post to an fp32 stream: the layer's input and
output carry one bf16 rounding each (2^-8 of a value at most, independent from value to value: 5 sigma
of the normed sum below 2^-6 of its rms 1), times the scale and the largest gate and weight,
0.5 * 1.2 * 1.2 < 0.75; two blocks add up, and the second block's routing is compared only while no
token is near a tie."""
import os
import sys

import pytest
import torch

from conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def _norm(v, w):
    return v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6) * w.double()


@pytest.mark.parametrize("tokens", [1, 5])
def test_two_blocks_eager_and_captured(cuda_device, tokens):
    import few_token_decode as F
    from test_gpu_few import reference

    stack = F.FewTokenStack(F.make_layers(2, tokens, seed=3))
    g = torch.Generator(device="cuda").manual_seed(5)
    resid = torch.randn(stack.resid.shape, generator=g, device="cuda")
    for buf in stack.attn:
        buf.copy_(torch.randn(buf.shape, generator=g, device="cuda"))

    r = resid.double()
    margin = torch.ones(tokens, device="cuda", dtype=torch.float64)
    for i, layer in enumerate(stack.layers):
        r = r + stack.attn[i].double()
        layer.x = _norm(r, stack.ffn_norm[i]).to(torch.bfloat16)
        y, m = reference(layer)
        margin = torch.minimum(margin, m)
        r = r + stack.branch_scale * stack.gate[i].double() * _norm(y, stack.post_norm[i])
    n = _norm(r, stack.next_norm[-1])
    # a rounding of the layer's input moves its keys by 2^-8 of a few
    keep = margin > 1e-3
    assert keep.any()

    def check():
        assert ((stack.resid.double() - r).abs() <= 2 * 0.75 * 2.0 ** -6)[keep].all()
        err = (stack.normed.double() - n).abs()
        assert (err <= 2.0 ** -8 * n.abs() + 1.2 * 2 * 0.75 * 2.0 ** -6)[keep].all()

    stack.resid.copy_(resid)
    stack.step()
    check()
    first = stack.resid.clone(), stack.normed.clone()
    stack.resid.copy_(resid)
    stack.capture()
    stack.resid.copy_(resid)
    stack.replay()
    torch.cuda.synchronize()
    assert torch.equal(stack.resid, first[0]) and torch.equal(stack.normed, first[1])

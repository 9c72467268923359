"""Decode steps of a few sequences through the FFN halves of a stack of blocks.

Each block's FFN half is three calls, captured once into a CUDA graph and replayed for every step:

  moe_block_join   r' = r + attn;  n = RMSNorm(r') w_ffn        (residual and norm before the layer)
  moe_forward_few  y = MoE(n)                                   (the whole layer, one launch)
  moe_block_join   r'' = r' + scale * gate * RMSNorm(y) w_post;  n' = RMSNorm(r'') w_next
                                                                (norm, gate and scale after it)

n' is what the next block's attention would read.  The attention itself is not part of this library:
its output is a given tensor of the step here.

  python examples/few_token_decode.py [--blocks 2] [--tokens 4] [--steps 20] [--full]
"""
import argparse
import os
import sys
from dataclasses import replace

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from mixture_experts_ffn_gemm_gb300 import binding as B  # noqa: E402
from mixture_experts_ffn_gemm_gb300 import synthetic as S  # noqa: E402


class FewTokenStack:
    """The FFN halves of len(layers) blocks for a fixed number of tokens, with their buffers."""

    def __init__(self, layers, branch_scale=0.5, seed=0):
        w = layers[0].w
        T, d, dt, dev = w.T, w.d, layers[0].x.dtype, layers[0].x.device
        g = torch.Generator(device=dev).manual_seed(seed)

        def vector():
            return (torch.rand(d, generator=g, device=dev) * 0.4 + 0.8).to(dt)

        self.layers = layers
        self.cfg = B.config_for(w)
        # a workspace a block: every call clears its workspace's status word, which `status` collects
        ws = torch.stack([B.alloc_few_workspace(self.cfg, dev) for _ in layers])
        self.ws = list(ws)
        self._flags = ws.view(torch.int32)[:, :1]
        self.status = torch.zeros(len(layers), 64, dtype=torch.int32, device=dev)
        self.ffn_norm = [vector() for _ in layers]
        self.post_norm = [vector() for _ in layers]
        self.next_norm = [vector() for _ in layers]
        self.gate = [vector() for _ in layers]
        self.before = B.make_join_config(T, d, dt, torch.float32, rms_eps=w.rms_eps)
        self.after = B.make_join_config(T, d, dt, torch.float32, gate="channel",
                                        branch_scale=branch_scale, rms_eps=w.rms_eps)
        self.branch_scale = branch_scale
        # the step's inputs and outputs: fp32 residual stream, one attention output per block
        self.resid = torch.zeros(T, d, dtype=torch.float32, device=dev)
        self.attn = [torch.zeros(T, d, dtype=dt, device=dev) for _ in layers]
        self.normed = torch.empty(T, d, dtype=dt, device=dev)
        self._n = torch.empty(T, d, dtype=dt, device=dev)
        self._y = torch.empty(T, d, dtype=dt, device=dev)
        self._graph = None

    def step(self):
        """One decode step in place: resid is the stream after the last block, normed its norm."""
        for i, layer in enumerate(self.layers):
            B.moe_block_join(self.before, self.resid, self.attn[i], None, None, self.ffn_norm[i],
                             self.resid, self._n)
            B.moe_forward_few(self.cfg, self._n, *B.layer_weights(layer), self._y, self.ws[i])
            B.moe_block_join(self.after, self.resid, self._y, self.post_norm[i], self.gate[i],
                             self.next_norm[i], self.resid, self.normed)
        self.status[:, :1].bitwise_or_(self._flags)

    def check(self):
        """Raises if a layer call of any step so far gave up a wait (synchronises)."""
        for i, word in enumerate(self.status):
            status = B.moe_device_status(word.view(torch.uint8))
            if status != B.MOE_OK:
                raise B.MoEError(status, f"block {i}")

    def capture(self):
        """Captures step() into a CUDA graph that replay() runs."""
        keep = self.resid.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.step()  # kernel attributes are set outside the capture
        torch.cuda.current_stream().wait_stream(side)
        self.resid.copy_(keep)
        self._graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self._graph):
            self.step()

    def replay(self):
        self._graph.replay()


def make_layers(blocks, tokens, full=False, seed=0):
    """Random-init layers: the K2 widths (384 experts: 34 GB a block) or a small stand-in."""
    w = S.WORKLOADS["k2_decode_bf16"]
    w = replace(w, T=tokens, w_init="fan_in")
    if not full:
        w = replace(w, d=1024, E=32, k=4, I=512, I_shared=512)
    return [S.make_layer(w, seed=seed + i, device="cuda") for i in range(blocks)]


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--blocks", type=int, default=2)
    ap.add_argument("--tokens", type=int, default=4)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--full", action="store_true", help="the K2 widths and 384 experts")
    a = ap.parse_args()
    stack = FewTokenStack(make_layers(a.blocks, a.tokens, a.full))
    stack.capture()
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for t in range(a.steps + 3):
        if t == 3:
            start.record()
        for i, buf in enumerate(stack.attn):
            buf.normal_()
        stack.replay()
    stop.record()
    torch.cuda.synchronize()
    stack.check()
    print(f"{a.blocks} blocks, {a.tokens} tokens: {start.elapsed_time(stop) / a.steps * 1e3:.1f} us "
          f"a step, |normed| rms {stack.normed.float().pow(2).mean().sqrt().item():.3f}")


if __name__ == "__main__":
    main()

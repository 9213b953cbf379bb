"""One mixture-of-experts layer: router, shared expert, routed experts, on one GPU.

    python examples/moe_layer.py                      # a decode batch of 64 tokens
    python examples/moe_layer.py --tokens 4096        # a prompt
    python examples/moe_layer.py --tokens 8 --experts 4 --top-k 2 --hidden 512 --intermediate 256 --check
    python examples/moe_layer.py --int8               # routed experts in 8-bit integers

The shared expert is bf16 (``mlp_swiglu_forward``); the routed experts are rounded once to e4m3 with a scale for each
block of 128 x 128 (``fp8_block_quantise``), as a program does when it loads a model.  With --int8 they are 8-bit integers with a
scale for each output channel (``int8_quantise``): the tokens are rounded and sorted by expert (``moe_sort``), go through
grouped products (``int8_grouped_matmul``) and the activation, and come back weighted on top of the shared expert's output
(``moe_unsort``).  Weights and tokens are random.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import __graft_entry__  # noqa: E402
import moe_shared_expert_gb300 as mse  # noqa: E402


class MoELayer:
    """Weights in the layouts the library takes, and the workspaces that every call of up to max_tokens reuses."""

    def __init__(self, hidden, intermediate, shared_intermediate, experts, top_k, max_tokens, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, generator=gen, device="cuda") / math.sqrt(shape[-1])).to(torch.bfloat16)

        H, I, E = hidden, intermediate, experts
        self.top_k = top_k
        self.router, self.bias = weight(E, H), 0.01 * torch.randn(E, generator=gen, device="cuda")
        self.shared_gate_up, self.shared_down = weight(2 * shared_intermediate, H), weight(H, shared_intermediate)
        # gate and up are rounded as two matrices, so that each has blocks of its own
        q, s = mse.fp8_block_quantise(weight(2 * E, I, H), block_rows=128)
        self.w_gate_up = q.as_strided((E, 2 * I, H), (2 * I * q.stride(1), q.stride(1), 1))
        self.s_gate_up = s.view(E, -1, s.shape[-1])
        self.w_down, self.s_down = mse.fp8_block_quantise(weight(E, H, I), block_rows=128)
        self.shared_workspace = mse.new_mlp_workspace(max_tokens, H, shared_intermediate)
        self.workspace = mse.new_moe_workspace(max_tokens, top_k, E, H, I)

    def route(self, x):
        return mse.moe_route(x @ self.router.t(), self.top_k, scoring="sigmoid", bias=self.bias)

    def shared(self, x):
        return mse.mlp_swiglu_forward(x, self.shared_gate_up, self.shared_down, workspace=self.shared_workspace)

    def __call__(self, x):
        ids, weights = self.route(x)
        y = self.shared(x)
        return mse.moe_experts_forward(x, ids, weights, self.w_gate_up, self.s_gate_up, self.w_down, self.s_down,
                                       shared=y, y=y, workspace=self.workspace)

    def experts(self):
        """The routed experts' weights [E, 2I, H] and [E, H, I] as the values they stand for."""
        def values(q, s):
            return q.float() * s.repeat_interleave(128, -2)[..., :q.shape[-2], :].repeat_interleave(128, -1)[..., :q.shape[-1]]

        E, _, H = self.w_gate_up.shape
        halves = self.w_gate_up.float().view(2 * E, -1, H), self.s_gate_up.view(2 * E, -1, self.s_gate_up.shape[-1])
        return values(*halves).view(E, -1, H), values(self.w_down, self.s_down)

    def plain(self, x):
        """The layer in elementary torch operations (8-bit weights as they are, activations not rounded)."""
        def swiglu(x, gate_up, down):
            g, u = (x @ gate_up.transpose(-1, -2)).chunk(2, -1)
            return (g / (1 + torch.exp(-g)) * u) @ down.transpose(-1, -2)

        x = x.float()
        score = torch.sigmoid((x.bfloat16() @ self.router.t()).float())
        ids = (score + self.bias).topk(self.top_k, 1).indices
        w = score.gather(1, ids)
        w = torch.zeros_like(score).scatter(1, ids, w / w.sum(1, keepdim=True))
        routed = swiglu(x, *self.experts())
        return swiglu(x, self.shared_gate_up.float(), self.shared_down.float()) + torch.einsum("te,eth->th", w, routed)


class Int8MoELayer(MoELayer):
    """The same layer with routed experts in 8-bit integers."""

    def __init__(self, hidden, intermediate, shared_intermediate, experts, top_k, max_tokens, seed=0):
        super().__init__(hidden, intermediate, shared_intermediate, experts, top_k, max_tokens, seed)
        gate_up, down = MoELayer.experts(self)
        self.gate_up, self.down = mse.int8_quantise(gate_up), mse.int8_quantise(down)
        del self.w_gate_up, self.s_gate_up, self.w_down, self.s_down, self.workspace
        pairs = max_tokens * top_k
        self.sort_workspace = mse.new_moe_sort_workspace(max_tokens, top_k, experts)
        self.workspaces = [mse.new_int8_workspace(pairs, w.shape[1], w.shape[2], experts) for w, _ in (self.gate_up, self.down)]

    def __call__(self, x):
        ids, weights = self.route(x)
        y = self.shared(x)
        q, scales = mse.int8_quantise(x)
        rows, place, offsets, scales = mse.moe_sort(q, ids, len(self.down[1]), scales=scales, workspace=self.sort_workspace)
        h = mse.int8_grouped_matmul(rows, scales, offsets, *self.gate_up, workspace=self.workspaces[0])
        h, scales = mse.int8_quantise(h, swiglu=True, offsets=offsets)
        o = mse.int8_grouped_matmul(h, scales, offsets, *self.down, workspace=self.workspaces[1])
        return mse.moe_unsort(o, place, weights, base=y, y=y)

    def experts(self):
        return [q.float() * s[..., None] for q, s in (self.gate_up, self.down)]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--hidden", type=int, default=7168)
    ap.add_argument("--intermediate", type=int, default=2048, help="of a routed expert")
    ap.add_argument("--shared-intermediate", type=int, default=None, help="of the shared expert (default 6144)")
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--top-k", type=int, default=8)
    ap.add_argument("--steps", type=int, default=50)
    ap.add_argument("--int8", action="store_true", help="routed experts in 8-bit integers")
    ap.add_argument("--check", action="store_true", help="compare with the layer in elementary operations")
    a = ap.parse_args()
    __graft_entry__.build()
    shared = a.shared_intermediate or (6144 if a.hidden == 7168 else 2 * a.intermediate)
    layer = (Int8MoELayer if a.int8 else MoELayer)(a.hidden, a.intermediate, shared, a.experts, a.top_k, a.tokens)
    x = torch.randn(a.tokens, a.hidden, device="cuda").to(torch.bfloat16)
    y = layer(x)
    if a.check:
        want = layer.plain(x)
        off = float((y.float() - want).norm() / want.norm())
        print(f"relative error against elementary operations: {off:.4f}")
        # x and h keep 3 fraction bits, about 2^-5 each in the mean square; 8-bit integers of a normal row more
        if not off < 0.06:
            raise SystemExit("the layer is off")
    for _ in range(3):
        layer(x)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(a.steps):
        layer(x)
    end.record()
    torch.cuda.synchronize()
    if mse.poll_device_error():
        raise SystemExit("device error")
    us = begin.elapsed_time(end) / a.steps * 1e3
    print(f"{a.tokens} tokens, {a.experts} experts of {a.hidden} x {a.intermediate}, top {a.top_k}, shared {shared}: "
          f"{us:.1f} us a layer, {a.tokens / us:.3f} M tokens/s")


if __name__ == "__main__":
    main()

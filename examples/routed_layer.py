"""One transformer block's routed feed-forward part as a serving process runs it: a
shared output projection on packed weights with the requests' low-rank adapters beside
it, then routing and the experts' gated feed-forward layer.

    python examples/routed_layer.py [tokens]

Prompts run eagerly; the decode step (few tokens, fixed buffers) is captured into a
graph and replayed.  Weights and inputs are random.
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from w4a8_quantized_gemm_quantize_amd import binding as w4a8  # noqa: E402


class RoutedLayer:
    """hidden -> shared projection + adapters -> router -> experts, residuals left out."""

    def __init__(self, hidden=1024, inter=512, experts=32, top_k=4, groups=4, topk_groups=2,
                 adapters=8, rank=16, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def rand(*shape):
            return torch.randn(shape, generator=g, device=device)

        def packed(rows, cols):
            return w4a8.pack_w4_grouped((0.02 * rand(rows, cols)).to(torch.bfloat16))

        self.hidden, self.inter, self.experts, self.top_k = hidden, inter, experts, top_k
        self.groups, self.topk_groups = groups, topk_groups
        self.proj = packed(hidden, hidden)
        self.lora_a = (rand(adapters, rank, hidden) * hidden ** -0.5).to(torch.bfloat16)
        self.lora_b = (rand(adapters, hidden, rank) * 0.1).to(torch.bfloat16)
        self.lora_scale = torch.full((adapters,), 0.5, device=device)
        self.router = (rand(hidden, experts) * hidden ** -0.5).to(torch.bfloat16)
        self.bias = 0.05 * rand(experts)
        self.w13 = packed(experts * 2 * inter, hidden)     # per expert: gate rows, then up rows
        self.w2 = packed(experts * hidden, inter)

    def buffers(self, tokens):
        """What a captured step keeps: outputs and workspaces of `tokens` rows."""
        dev = self.router.device
        h, k = self.hidden, self.top_k

        def space(n):
            return torch.empty(max(n, 16), dtype=torch.uint8, device=dev)

        return dict(
            y=torch.empty((tokens, h), dtype=torch.bfloat16, device=dev),
            logits=torch.empty((tokens, self.experts), dtype=torch.bfloat16, device=dev),
            ids=torch.empty((tokens, k), dtype=torch.int32, device=dev),
            weights=torch.empty((tokens, k), device=dev),
            out=torch.empty((tokens, h), dtype=torch.bfloat16, device=dev),
            proj_ws=space(w4a8.workspace_bytes(tokens, h, h)),
            lora_ws=space(w4a8.lora_workspace_bytes(tokens, *self.lora_a.shape)),
            moe_ws=space(w4a8.moe_ffn_workspace_bytes(tokens, self.experts, k, h, self.inter)))

    def __call__(self, x, adapter_ids, buf=None):
        """x bf16 [tokens, hidden], adapter_ids int32 [tokens] (-1: none) -> bf16."""
        b = buf if buf is not None else {}
        y = w4a8.w4a8_gemm_bf16act(x, *self.proj, self.hidden, out=b.get("y"),
                                   workspace=b.get("proj_ws"))
        w4a8.lora_add(x, self.lora_a, self.lora_b, adapter_ids, y, scale=self.lora_scale, out=y,
                      workspace=b.get("lora_ws"))
        logits = torch.mm(y, self.router, out=b.get("logits"))
        ids, weights = w4a8.moe_route(logits, self.top_k, bias=self.bias, score="sigmoid",
                                      groups=self.groups, topk_groups=self.topk_groups,
                                      ids=b.get("ids"), weights=b.get("weights"))
        return w4a8.w4a8_moe_ffn(y, ids, weights, self.w13, self.w2, self.inter,
                                 out=b.get("out"), workspace=b.get("moe_ws"))


def main(tokens=300, steps=4):
    layer = RoutedLayer()
    g = torch.Generator(device="cuda").manual_seed(1)

    def batch(t):
        x = torch.randn((t, layer.hidden), generator=g, device="cuda").to(torch.bfloat16)
        ids = torch.randint(-1, layer.lora_a.shape[0], (t,), generator=g, device="cuda")
        return x, ids.to(torch.int32)

    out = layer(*batch(tokens))
    torch.cuda.synchronize()
    print(f"prompt of {tokens} tokens: |out| rms {out.float().square().mean().sqrt():.4f}")

    # decode: fixed buffers, one graph
    x, ids = batch(5)
    buf = layer.buffers(5)
    layer(x, ids, buf)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(x, ids, buf)
    worst = 0.0
    for _ in range(steps):
        nx, nid = batch(5)
        x.copy_(nx)
        ids.copy_(nid)
        graph.replay()
        torch.cuda.synchronize()
        eager = layer(nx, nid)
        worst = max(worst, (eager.float() - buf["out"].float()).abs().max().item())
    print(f"decode of 5 tokens, {steps} replays: largest difference from eager {worst}")
    return out, worst


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 300)

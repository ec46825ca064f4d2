"""The feed-forward half of a decoder layer with routed experts on block-quantised weights.

    python examples/expert_layer.py [tokens]

The hidden states are added to the residual stream and normalised (rfp2_rms_norm), a router's logits choose
each token's experts (rfp2_moe_route), their gate and up rows are multiplied and joined (rfp2_moe_gemm with its
gated activation), their down rows after them (rfp2_moe_gemm with a row for every slot), and the experts'
rows are summed onto the residual stream (rfp2_moe_combine).  The step is captured as a CUDA graph and
replayed; a shared expert runs beside it on the same norm's Q8 blocks (rfp2_gemv_q8) for a few tokens.
The result is compared with the same layer in float64 over the weights that the blocks stand for.
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

HIDDEN, WIDTH, EXPERTS, TOP_K, GROUPS, KEEP = 512, 256, 32, 4, 4, 2


class Layer:
    """The packed weights and the workspace of a layer for up to `tokens` tokens."""

    def __init__(self, tokens, seed=0):
        import torch
        import gemm_rocmfp2_mul_gb300 as g
        self.g, self.tokens = g, tokens
        r = torch.Generator(device="cuda").manual_seed(seed)

        def packed(*shape):
            w = torch.randn(shape, generator=r, device="cuda") * shape[-1] ** -0.5
            return g.rfp2_pack_weights(w.flatten(0, -2)).view(*shape[:-1], shape[-1] // 32, 10)

        self.gate_up = packed(EXPERTS, 2 * WIDTH, HIDDEN)
        self.down = packed(EXPERTS, HIDDEN, WIDTH)
        self.shared = packed(HIDDEN, HIDDEN)
        self.router = torch.randn((EXPERTS, HIDDEN), generator=r, device="cuda") * HIDDEN ** -0.5
        self.balance = 0.05 * torch.randn(EXPERTS, generator=r, device="cuda")
        self.weight = 1.0 + 0.1 * torch.randn(HIDDEN, generator=r, device="cuda")
        self.ids = torch.empty((tokens, TOP_K), dtype=torch.int32, device="cuda")
        self.workspace = g.rfp2_moe_gemm_workspace(self.ids, EXPERTS)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def __call__(self, x, residual):
        """x, residual fp32 [T, HIDDEN] -> the residual stream after the experts, bf16 values in the products."""
        import torch
        g, T = self.g, x.shape[0]
        n = g.rfp2_rms_norm(x, self.weight, residual=residual, want="both", dtype=torch.bfloat16)
        logits = n.y.float() @ self.router.T
        ids, weights = g.rfp2_moe_route(logits, TOP_K, scoring="sigmoid", bias=self.balance, groups=GROUPS, keep=KEEP,
                                        group_top=2, scale=2.0, ids=self.ids[:T])
        h = g.rfp2_moe_gemm(self.gate_up, EXPERTS, 2 * WIDTH, HIDDEN, ids, n.y, activation="silu",
                            workspace=self.workspace, dev_status=self.status)
        y = g.rfp2_moe_gemm(self.down, EXPERTS, HIDDEN, WIDTH, ids, h, workspace=self.workspace, dev_status=self.status)
        out = g.rfp2_moe_combine(y, weights, ids=ids, residual=n.total)
        if T <= g.MAX_BATCH:
            out += g.rfp2_gemv_q8(self.shared, HIDDEN, HIDDEN, n.q, n.d)
        return out, logits, ids


def run(tokens=64, replays=3, seed=0):
    """(layer, [(x, residual, out, logits, ids)]) of a captured step, replayed on new inputs."""
    import torch
    if min(tokens, replays) < 1:
        raise ValueError(f"tokens and replays are needed, got {tokens} and {replays}")
    layer = Layer(tokens, seed)
    r = torch.Generator(device="cuda").manual_seed(seed + 1)
    x, residual = torch.zeros((2, tokens, HIDDEN), device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        layer(x, residual)      # what the first call sets up is not captured
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            found = layer(x, residual)
    torch.cuda.current_stream().wait_stream(stream)
    steps = []
    for _ in range(replays):
        x.copy_(torch.randn((tokens, HIDDEN), generator=r, device="cuda"))
        residual.copy_(2.0 * torch.randn((tokens, HIDDEN), generator=r, device="cuda"))
        graph.replay()
        steps.append(tuple(t.clone() for t in (x, residual, *found)))
    return layer, steps


def dequantised(packed):
    """float64 weights of ROCmFP2 blocks [..., K/32, 10]."""
    import torch
    codes = torch.stack([(packed[..., :8] >> (2 * i)) & 3 for i in range(4)], -1).flatten(-2)
    scale = packed[..., 8:].contiguous().view(torch.float8_e4m3fn).double() / 2
    levels = torch.tensor([-4.0, -1.0, 1.0, 4.0], dtype=torch.float64, device=packed.device)
    return (levels[codes.long()] * scale.repeat_interleave(16, -1)).flatten(-2)


def reference(layer, x, residual, logits, ids):
    """(the experts' part, the residual stream) in float64, of the experts in `ids`."""
    import torch
    total = x.double() + residual.double()
    y = total * (total.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * layer.weight.double()
    weights = torch.sigmoid(logits.double()).gather(1, ids.long())
    weights = 2.0 * weights / weights.sum(-1, keepdim=True)
    gate_up, down = dequantised(layer.gate_up)[ids.long()], dequantised(layer.down)[ids.long()]
    gate, up = torch.einsum("tjmk,tk->tjm", gate_up, y).chunk(2, -1)
    rows = torch.einsum("tjmk,tjk->tjm", down, gate * torch.sigmoid(gate) * up)
    out = torch.einsum("tj,tjm->tm", weights, rows)
    if x.shape[0] <= layer.g.MAX_BATCH:
        out = out + y @ dequantised(layer.shared).T
    return out, total


def main(argv):
    layer, steps = run(int(argv[0]) if argv else 64)
    for x, residual, out, logits, ids in steps:
        ref, total = reference(layer, x, residual, logits, ids)
        off = (out.double() - total - ref).norm(dim=-1) / ref.norm(dim=-1)
        print(f"status {int(layer.status)}; relative error a token of the experts' part: {float(off.max()):.4f} "
              "(bf16 values in the products against float64)")


if __name__ == "__main__":
    main(sys.argv[1:])

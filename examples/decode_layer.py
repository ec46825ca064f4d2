"""One attention layer of a decoder on block-quantised weights: a prompt, then tokens one at a time.

    python examples/decode_layer.py [prompt tokens] [new tokens]

The layer's two products run on ROCmFP2 weights (rfp2_gemm for the prompt, rfp2_gemv for a token); between
them the queries are rotated (rfp2_rope), the keys rotated and quantised into a paged cache with the values
(rfp2_kv_write), and the newest tokens attend over that cache (rfp2_attn_decode).  The step of a token is
captured once as a CUDA graph: the positions, slots and lengths that it reads are advanced on the GPU.
The result is compared with the same layer in float64 over the weights that the blocks stand for.
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

HIDDEN, HEADS, KV_HEADS, D, PAGE = 1024, 8, 2, 128, 16


class Layer:
    """The layer's packed weights, its cache and the buffers of a step, for `batch` sequences."""

    def __init__(self, batch, capacity, seed=0):
        import torch
        import gemm_rocmfp2_mul_gb300 as g
        self.g, self.batch = g, batch
        r = torch.Generator(device="cuda").manual_seed(seed)
        rows = (HEADS + 2 * KV_HEADS) * D
        self.qkv = g.rfp2_pack_weights(torch.randn((rows, HIDDEN), generator=r, device="cuda") * HIDDEN ** -0.5)
        self.out = g.rfp2_pack_weights(torch.randn((HIDDEN, HEADS * D), generator=r, device="cuda") * HIDDEN ** -0.5)
        # a context stretched fourfold over the trained length
        self.inv_freq, self.factor = g.rfp2_rope_frequencies(D, scaling="ramp", stretch=4.0, trained=4096.0)
        pages = -(-capacity // PAGE)
        self.cache = g.rfp2_kv_alloc(batch * pages, KV_HEADS, PAGE, D)
        order = torch.randperm(batch * pages, generator=r, device="cuda").int()
        self.table = order.view(batch, pages)
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        # for a prompt's tokens at once, and so for one
        longest = torch.empty(1, device="cuda").expand(batch, capacity, HEADS, D)
        self.workspace = g.rfp2_attn_decode_workspace(longest, KV_HEADS)
        self.gemv_workspace = [torch.empty(g.rfp2_gemv_workspace_bytes(batch, K), dtype=torch.uint8, device="cuda")
                               for K in (HIDDEN, HEADS * D)]

    def places(self, positions):
        """Slots of the tokens at positions [batch, n]."""
        page = self.table.gather(1, (positions // PAGE).long())
        return (page.long() * PAGE + positions % PAGE).flatten()

    def attend(self, qkv, new):
        """qkv fp32 [batch * new, rows] of each sequence's newest tokens -> [batch * new, HEADS * D]."""
        import torch
        g = self.g
        heads = qkv.view(-1, HEADS + 2 * KV_HEADS, D)
        q, k, v = heads.split([HEADS, KV_HEADS, KV_HEADS], dim=1)
        positions = self.lens[:, None] + torch.arange(new, dtype=torch.int32, device="cuda")
        at = positions.flatten()
        g.rfp2_rope(q, at, self.inv_freq, out=q, factor=self.factor)
        g.rfp2_kv_write(self.cache, k, v, self.places(positions), at, self.inv_freq, factor=self.factor,
                        dev_status=self.status)
        self.lens += new
        o, _ = g.rfp2_attn_decode(q.unflatten(0, (self.batch, new)), self.cache, self.table, self.lens,
                                  workspace=self.workspace, dev_status=self.status)
        return o.view(-1, HEADS * D)

    def prompt(self, x):
        """x bf16 [batch * new, HIDDEN], the sequences' tokens one after another."""
        g, rows = self.g, (HEADS + 2 * KV_HEADS) * D
        o = self.attend(g.rfp2_gemm(self.qkv, rows, HIDDEN, x), x.shape[0] // self.batch)
        return g.rfp2_gemm(self.out, HIDDEN, HEADS * D, o.bfloat16())

    def token(self, x):
        """x fp32 [batch, HIDDEN]: one token of each sequence."""
        g, rows = self.g, (HEADS + 2 * KV_HEADS) * D
        qkv = g.rfp2_gemv(self.qkv, rows, HIDDEN, x, workspace=self.gemv_workspace[0])
        return g.rfp2_gemv(self.out, HIDDEN, HEADS * D, self.attend(qkv, 1), workspace=self.gemv_workspace[1])


def run(prompt=300, new=20, batch=2, seed=0):
    """Outputs of the layer for a prompt and `new` tokens, one replayed step each, and their inputs."""
    if min(prompt, new, batch) < 1:
        raise ValueError(f"a prompt, new tokens and sequences are needed, got {prompt}, {new} and {batch}")
    import torch
    layer = Layer(batch, prompt + new, seed)
    r = torch.Generator(device="cuda").manual_seed(seed + 1)
    first = torch.randn((batch * prompt, HIDDEN), generator=r, device="cuda").bfloat16()
    tokens = torch.randn((new, batch, HIDDEN), generator=r, device="cuda")
    outputs = [layer.prompt(first).view(batch, prompt, HIDDEN)]
    x = torch.zeros((batch, HIDDEN), device="cuda")
    lens = layer.lens.clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        layer.token(x)          # what the first call sets up is not captured
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            y = layer.token(x)
    torch.cuda.current_stream().wait_stream(stream)
    layer.lens.copy_(lens)      # the trial step's token is written over by the first one
    for t in range(new):
        x.copy_(tokens[t])
        graph.replay()
        outputs.append(y.clone()[:, None])
    inputs = torch.cat([first.float().view(batch, prompt, HIDDEN), tokens.transpose(0, 1)], dim=1)
    return layer, inputs, torch.cat(outputs, dim=1)


def dequantised(packed, K):
    """float64 weights of ROCmFP2 blocks."""
    import torch
    blocks = packed.view(packed.shape[0], K // 32, 10)
    codes = torch.stack([(blocks[..., :8] >> (2 * i)) & 3 for i in range(4)], -1).flatten(-2)
    scale = blocks[..., 8:].contiguous().view(torch.float8_e4m3fn).double() / 2
    levels = torch.tensor([-4.0, -1.0, 1.0, 4.0], dtype=torch.float64, device=packed.device)
    return (levels[codes.long()] * scale.repeat_interleave(16, -1)).flatten(1)


def reference(layer, inputs):
    """The layer in float64: no blocks of activations, no cache, every token attending over all before it."""
    import torch
    B, T, _ = inputs.shape
    rows = inputs.double() @ dequantised(layer.qkv, HIDDEN).T
    q, k, v = rows.view(B, T, -1, D).split([HEADS, KV_HEADS, KV_HEADS], dim=2)
    theta = torch.outer(torch.arange(T, device="cuda").double(), layer.inv_freq.double())[:, None]
    c, s = layer.factor * theta.cos(), layer.factor * theta.sin()

    def turn(x):
        a, b = x[..., : D // 2], x[..., D // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    q, k = turn(q), turn(k).repeat_interleave(HEADS // KV_HEADS, 2)
    scores = torch.einsum("bihd,bjhd->bhij", q, k) * D ** -0.5
    scores = scores.masked_fill(torch.ones(T, T, device="cuda").triu(1).bool(), -float("inf"))
    o = torch.einsum("bhij,bjhd->bihd", scores.softmax(-1), v.repeat_interleave(HEADS // KV_HEADS, 2))
    return o.reshape(B, T, -1) @ dequantised(layer.out, HEADS * D).T


def main(argv):
    import torch
    prompt, new = (int(argv[0]) if argv else 300), (int(argv[1]) if len(argv) > 1 else 20)
    layer, inputs, y = run(prompt, new)
    ref = reference(layer, inputs)
    torch.cuda.synchronize()
    off = ((y.double() - ref).norm(dim=-1) / ref.norm(dim=-1))
    print(f"status {int(layer.status)}; relative error a token: prompt {off[:, :prompt].max():.4f}, "
          f"new tokens {off[:, prompt:].max():.4f} (8-bit activations and cache against float64)")


if __name__ == "__main__":
    main(sys.argv[1:])

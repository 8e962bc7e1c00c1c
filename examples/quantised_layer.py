"""One layer of a model with multi-head latent attention in 8 bits throughout: its products on E4M3 weights and rows, its
attention over the 8-bit latent cache.

Prompts go through the layer in one call, then token by token, as a server runs them: rows are normalised, quantised and
multiplied (latent and absorbed queries), the latents appended to the cache and attended, the outputs multiplied back onto
the residual stream, and the gated feed-forward block does the rest. Synthetic weights stand in for a model's. The last line
says how far 8 bits moved the layer's outputs from the same layer in 32 bits.

    python examples/quantised_layer.py [tokens]
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mla_block_diffusion_gb300 as M  # noqa: E402

HIDDEN, INTER, HEADS, KV, ROPE, PAGE = 1024, 2048, 8, 64, 16, 64
D = KV + ROPE
SCALE = 1 / math.sqrt(D)


def blocks(n: int) -> int:
    return -(-n // 128)


def linear(w: torch.Tensor) -> M.QLinear:
    """A weight matrix in the 8-bit format."""
    codes = torch.empty(w.shape, dtype=torch.uint8, device="cuda")
    scales = torch.empty(blocks(w.shape[0]), blocks(w.shape[1]), device="cuda")
    M.quantise_weight(w, codes, scales)
    return M.QLinear(codes, scales)


def norm(x: torch.Tensor) -> torch.Tensor:
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


class Layer:
    """The layer and its cache, for up to max_requests requests of max_tokens tokens."""

    def __init__(self, weights, max_requests: int, max_tokens: int, max_new: int):
        self.latent, self.query, self.out = (linear(weights[k]) for k in ("latent", "query", "out"))
        self.gated, self.down = M.QGated(linear(weights["gate"]), linear(weights["up"])), linear(weights["down"])
        pages = max_requests * -(-max_tokens // PAGE)
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.codes, self.scales = torch.zeros(pages, PAGE, D, dtype=torch.uint8, device="cuda"), torch.ones(pages, device="cuda")
        self.cache = M.QCache(KV, ROPE, [self.codes], [self.scales], i32(max_requests, -(-max_tokens // PAGE)), n_heads=HEADS)
        self.length, self.next_length = i32(max_requests), i32(max_requests)
        self.ring = torch.arange(pages, dtype=torch.int32, device="cuda")
        self.state, self.next_state = torch.tensor([0, pages], dtype=torch.int32, device="cuda"), i32(2)
        self.cu, self.slots, self.positions = i32(max_requests + 1), i32(max_new), i32(max_new)
        self.seg_row = i32(max_new // PAGE + 2 * max_requests + 1)

    @staticmethod
    def rows(x: torch.Tensor):
        """Rows in the 8-bit format."""
        q = torch.empty(x.shape, dtype=torch.uint8, device="cuda"), torch.empty(blocks(x.shape[1]), x.shape[0], device="cuda")
        M.quantise_rows(x, *q)
        return q

    def step(self, want: torch.Tensor, x: torch.Tensor) -> torch.Tensor:
        """The residual stream's new rows x [new, HIDDEN] (fp32) of requests that go to `want` tokens, through the layer, in
        place."""
        n = x.shape[0]
        self.cache.plan(self.length, want, self.ring, self.state, self.next_length, self.next_state, self.cu, self.slots,
                        self.positions, self.seg_row)
        self.length, self.next_length = self.next_length, self.length
        self.state, self.next_state = self.next_state, self.state
        bf16 = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        h = self.rows(norm(x))
        latent, query, o = bf16(n, D), bf16(n, HEADS, D), bf16(n, HEADS, KV)
        self.latent.matmul(*h, latent)
        self.query.matmul(*h, query.view(n, HEADS * D))
        self.cache.append(latent[None], self.slots, self.seg_row)
        self.cache.attend(0, query, self.cu, self.length, o, causal=True, scale=SCALE)
        self.out.matmul(*self.rows(o.view(n, HEADS * KV)), x, add=x)
        g = torch.empty(n, INTER, dtype=torch.uint8, device="cuda"), torch.empty(blocks(INTER), n, device="cuda")
        self.gated.forward(*self.rows(norm(x)), *g)
        self.down.matmul(*g, x, add=x)
        return x

    def check(self) -> bool:
        return not any(t.check() for t in (self.cache, self.latent, self.query, self.out, self.gated, self.down))


def exact(weights, x: torch.Tensor) -> torch.Tensor:
    """The layer over one request's rows in 32 bits."""
    h = norm(x)
    latent, query = h @ weights["latent"].t(), (h @ weights["query"].t()).view(-1, HEADS, D)
    s = torch.einsum("ihd,kd->ihk", query, latent) * SCALE
    n = x.shape[0]
    s.masked_fill_((torch.arange(n, device="cuda")[None] > torch.arange(n, device="cuda")[:, None])[:, None], float("-inf"))
    x = x + torch.einsum("ihk,kd->ihd", s.softmax(2), latent[:, :KV]).reshape(n, HEADS * KV) @ weights["out"].t()
    h = norm(x)
    return x + torch.nn.functional.silu(h @ weights["gate"].t()) * (h @ weights["up"].t()) @ weights["down"].t()


def main(tokens: int = 12, seed: int = 0):
    torch.backends.cuda.matmul.allow_tf32 = False
    g = torch.Generator(device="cuda").manual_seed(seed)
    draw = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    weights = {k: draw(n, m) / math.sqrt(m) for k, (n, m) in {
        "latent": (D, HIDDEN), "query": (HEADS * D, HIDDEN), "out": (HIDDEN, HEADS * KV), "gate": (INTER, HIDDEN),
        "up": (INTER, HIDDEN), "down": (HIDDEN, INTER)}.items()}
    prompts = [300, 64, 1]
    layer = Layer(weights, len(prompts), 512, max_new=512)
    inputs = [draw(n + tokens, HIDDEN) for n in prompts]
    outputs = [torch.empty_like(x) for x in inputs]
    at = [0] * len(prompts)
    for step in range(tokens + 1):
        to = [n + step for n in prompts]
        x = torch.cat([x[a:b] for x, a, b in zip(inputs, at, to)])
        y = layer.step(torch.tensor(to, dtype=torch.int32, device="cuda"), x)
        for i, part in enumerate(y.split([b - a for a, b in zip(at, to)])):
            outputs[i][at[i]:to[i]] = part
        at = to
    if not layer.check():
        raise RuntimeError("the kernels reported an error")
    worst = 0.0
    for x, y in zip(inputs, outputs):
        ref = exact(weights, x)
        worst = max(worst, float((y - ref).norm() / (ref - x).norm()))
    print(f"{sum(prompts)} tokens of prompts and {tokens} more of each; what the layer adds differs from 32 bits by {worst:.3f} "
          "of its size")
    return worst


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 12)

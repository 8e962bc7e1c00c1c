"""Serving attention from the 8-bit latent cache: prompts come in, are decoded token by token, grow and leave.

Every step is what a server runs for one attention layer of a model with multi-head latent attention: the page plan
(pages, slots and positions for the requests' new tokens, on the GPU), the quantising append of their latent entries,
and the attention of their queries over the cache. Synthetic latents and queries stand in for the model's; the same
tokens are kept unquantised, and the last line says how far the 8-bit cache moved the attention's outputs.

    python examples/quantised_cache.py [steps]
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mla_block_diffusion_gb300 as M  # noqa: E402

KV, ROPE, HEADS, PAGE = 512, 64, 64, 64


class Server:
    """One layer's cache for up to max_requests requests of max_tokens tokens, with room for n_pages pages."""

    def __init__(self, max_requests: int, max_tokens: int, n_pages: int, max_new: int):
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.codes = torch.zeros(n_pages, PAGE, KV + ROPE, dtype=torch.uint8, device="cuda")
        self.scales = torch.ones(n_pages, device="cuda")
        self.cache = M.QCache(KV, ROPE, [self.codes], [self.scales], i32(max_requests, -(-max_tokens // PAGE)), n_heads=HEADS)
        self.length, self.next_length = i32(max_requests), i32(max_requests)
        self.ring = torch.arange(n_pages, dtype=torch.int32, device="cuda")
        self.state, self.next_state = torch.tensor([0, n_pages], dtype=torch.int32, device="cuda"), i32(2)
        self.cu, self.slots, self.positions = i32(max_requests + 1), i32(max_new), i32(max_new)
        self.seg_row = i32(max_new // PAGE + 2 * max_requests + 1)

    def step(self, want: torch.Tensor, entries: torch.Tensor, queries: torch.Tensor):
        """Requests go to `want` tokens; entries [new, 576] and queries [new, heads, 576] of their new tokens, in order.
        A request of 0 tokens has ended and gives its pages back. Returns the new tokens' outputs [new, heads, 512]."""
        self.cache.plan(self.length, want, self.ring, self.state, self.next_length, self.next_state, self.cu, self.slots,
                        self.positions, self.seg_row)
        self.length, self.next_length = self.next_length, self.length
        self.state, self.next_state = self.next_state, self.state
        self.cache.append(entries[None], self.slots, self.seg_row)
        out = torch.empty(queries.shape[0], HEADS, KV, dtype=torch.bfloat16, device="cuda")
        self.cache.attend(0, queries, self.cu, self.length, out, causal=True, scale=1 / math.sqrt(192))
        return out


def exact(history: torch.Tensor, queries: torch.Tensor) -> torch.Tensor:
    """The same attention over the unquantised tokens of one request, in 32 bits."""
    n, seen = queries.shape[0], history.shape[0]
    s = torch.einsum("ihd,kd->ihk", queries.float(), history.float()) / math.sqrt(192)
    last = seen - n + torch.arange(n, device="cuda")
    s.masked_fill_((torch.arange(seen, device="cuda")[None] > last[:, None])[:, None], float("-inf"))
    return torch.einsum("ihk,kd->ihd", s.softmax(2), history[:, :KV].float())


def main(steps: int = 40, seed: int = 0):
    torch.backends.cuda.matmul.allow_tf32 = False
    g = torch.Generator(device="cuda").manual_seed(seed)
    draw = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    prompts = [700, 64, 1, 333, 1200]                        # admitted in steps 0, 1, 2, ...
    server = Server(len(prompts), 2048, n_pages=64, max_new=1500)
    history = [draw(0, KV + ROPE) for _ in prompts]
    worst = 0.0
    for step in range(steps):
        fresh = []
        for r, n in enumerate(prompts):
            if step < r or not history[r].shape[0] and step > r:
                fresh.append(0)                              # not here yet, or gone
            elif step == r:
                fresh.append(n)                              # its prompt
            elif r == 3 and step == steps // 2:
                fresh.append(-1)                             # it ends
            else:
                fresh.append(1)                              # one decoded token
        for r, n in enumerate(fresh):
            history[r] = history[r][:0] if n < 0 else torch.cat([history[r], draw(n, KV + ROPE)])
        fresh = [max(0, n) for n in fresh]
        want = torch.tensor([h.shape[0] for h in history], dtype=torch.int32, device="cuda")
        queries = draw(sum(fresh), HEADS, KV + ROPE)
        entries = torch.cat([h[h.shape[0] - n:] for h, n in zip(history, fresh)])
        out, at = server.step(want, entries, queries), 0
        assert server.length.tolist() == want.tolist(), "a request did not get its pages"
        for h, n in zip(history, fresh):
            if n:
                ref = exact(h, queries[at:at + n])
                worst = max(worst, float((out[at:at + n].float() - ref).norm() / ref.norm()))
            at += n
    if server.cache.check():
        raise RuntimeError("the kernels reported an error")
    free = int(server.state[1])
    held = sum(-(-h.shape[0] // PAGE) for h in history)
    print(f"{steps} steps, {sum(h.shape[0] for h in history)} tokens in {held} pages, {free} pages free; largest relative "
          f"difference of a request's outputs from the unquantised cache {worst:.3f}")
    return worst, held + free


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 40)

"""Products and gated products of quantised rows: CTAs that leave and come."""
import numpy as np
import pytest
import torch

import mla_block_diffusion_gb300 as M
from tests.test_gpu_qlinear import dev, rows_of, weight_of

pytestmark = pytest.mark.gpu


def blocks(n):
    return -(-n // 128)


@pytest.mark.parametrize("kb", [1, 4, 5, 6, 11, 12, 13, 25])
def test_kernels_that_follow_one_another(kb):
    """Every kernel has its barriers in another place of shared memory, and the next one's CTAs come as soon as one has left:
    rings that are not filled, just filled and filled again, results bit for bit those of calls that are waited for."""
    rng = np.random.default_rng(kb)
    k, n = 128 * kb - 16, 4112
    gate, up = (M.QLinear(*(dev(a) for a in weight_of(rng, n, k))) for _ in range(2))
    gated = M.QGated(gate, up)
    calls, outs = [], []
    for m in (1, 64, 17, 65, 32, 5):
        x = [dev(a) for a in rows_of(rng, m, k)]
        y = torch.zeros(m, n, device="cuda")
        h = torch.zeros(m, n, dtype=torch.uint8, device="cuda"), torch.zeros(blocks(n), m, device="cuda")
        calls += [lambda x=x, y=y: gate.matmul(*x, y), lambda x=x, h=h: gated.forward(*x, *h)]
        outs += [y, *h]
    for call in calls:
        call()
        torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    for t in outs:
        t.zero_()
    for _ in range(20):
        for call in calls:
            call()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    for t in outs:
        t.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for call in calls[::-1]:
            call()
    for _ in range(20):
        g.replay()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert gate.check() == 0


@pytest.mark.parametrize("m", [16, 32, 64])
def test_rings_around_their_length(m):
    """Few rows, up to 26 blocks of k: rings of 5 to 11 stages that are not filled, just filled, and filled again once and twice;
    the kernels lie close behind one another, and nothing of one may arrive in the next."""
    rng = np.random.default_rng(m)
    n, calls, outs = 272, [], []
    for kb in range(1, 27):
        k = 128 * kb
        gate, up = (M.QLinear(*(dev(a) for a in weight_of(rng, n, k))) for _ in range(2))
        x = [dev(a) for a in rows_of(rng, m, k)]
        y = torch.zeros(m, n, device="cuda")
        h = torch.zeros(m, n, dtype=torch.uint8, device="cuda"), torch.zeros(blocks(n), m, device="cuda")
        calls += [lambda a=gate, x=x, y=y: a.matmul(*x, y), lambda a=M.QGated(gate, up), x=x, h=h: a.forward(*x, *h)]
        outs += [y, *h]
    for call in calls:
        call()
        torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    for t in outs:
        t.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for call in calls:
            call()
        for call in calls[::-1]:
            call()
    for _ in range(30):
        g.replay()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert gate.check() == 0


@pytest.mark.parametrize("m", [1, 7, 64, 65, 300])
@pytest.mark.parametrize("n,k", [(272, 528), (2112, 1552)])
def test_columns_of_one_buffer(m, n, k):
    """A result, the residual and a stranger's column side by side; the scales of the rows and of h in one buffer: bit for bit
    what contiguous tensors give, and nothing else is written."""
    rng = np.random.default_rng(m * 7 + n)
    x, sx = (dev(a) for a in rows_of(rng, m, k))
    gate, up = (M.QLinear(*(dev(a) for a in weight_of(rng, n, k))) for _ in range(2))
    add = torch.randn(m, n, device="cuda") * 30
    want = {t: torch.empty(m, n, dtype=t, device="cuda") for t in (torch.float32, torch.bfloat16)}
    for y in want.values():
        gate.matmul(x, sx, y, add=add)
    hw = torch.empty(m, n, dtype=torch.uint8, device="cuda"), torch.empty(blocks(n), m, device="cuda")
    M.QGated(gate, up).forward(x, sx, *hw)
    for first in (0, n + 16):  # the result in front of the residual or behind it
        for t, y0 in want.items():
            buf = torch.full((m, 3 * n), 5.0, device="cuda")
            other = n + 16 - first
            buf[:, other:other + n] = add
            size = 4 // t.itemsize
            y = buf.view(t)[:, size * first:size * first + n]
            before = buf.clone()
            gate.matmul(x, sx, y, add=buf[:, other:other + n])
            assert torch.equal(y, y0)
            before.view(t)[:, size * first:size * first + n] = y0
            assert torch.equal(buf, before)
    scales = torch.full((max(blocks(k), blocks(n)), 2 * m + 3), 5.0, device="cuda")
    scales[:blocks(k), :m] = sx
    h = torch.empty_like(hw[0])
    before = scales.clone()
    M.QGated(gate, up).forward(x, scales[:blocks(k), :m], h, scales[:blocks(n), m + 1:2 * m + 1])
    before[:blocks(n), m + 1:2 * m + 1] = hw[1]
    assert torch.equal(h, hw[0]) and torch.equal(scales, before)
    assert gate.check() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,k,n", [(1, 512, 1040), (7, 7168, 272), (64, 2112, 1024), (65, 1536, 4112), (700, 1040, 2064)])
def test_feed_forward_chains(m, k, n, dtype):
    """Quantise, gated product, down onto the residual, quantise again, each kernel beginning before the last has ended: the bits of
    calls that are waited for, eager on two streams and replayed, for inputs that change between the passes."""
    g = torch.Generator(device="cuda").manual_seed(m)

    def linear(n, k):
        codes, scales = torch.empty(n, k, dtype=torch.uint8, device="cuda"), torch.empty(blocks(n), blocks(k), device="cuda")
        M.quantise_weight(torch.randn(n, k, device="cuda", generator=g) / k ** 0.5, codes, scales)
        return M.QLinear(codes, scales)

    class Chain:
        def __init__(self):
            self.x, self.y = torch.empty(m, k, dtype=dtype, device="cuda"), torch.empty(m, k, device="cuda")
            self.q, self.h, self.z = ((torch.empty(m, w, dtype=torch.uint8, device="cuda"), torch.empty(blocks(w), m, device="cuda"))
                                      for w in (k, n, k))

        def run(self, source, wait=lambda: None):
            self.x.copy_(source)
            self.y.copy_(source)
            for call in (lambda: M.quantise_rows(self.x, *self.q), lambda: gated.forward(*self.q, *self.h),
                         lambda: down.matmul(*self.h, self.y, add=self.y), lambda: M.quantise_rows(self.y, *self.z)):
                wait()
                call()

        def results(self):
            return [t.clone() for t in (self.y, *self.z)]

    gated, down = M.QGated(linear(n, k), linear(n, k)), linear(k, n)
    sources = [torch.randn(m, k, device="cuda", generator=g).to(dtype) for _ in range(3)]
    chain, want = Chain(), []
    for s in sources:
        chain.run(s, torch.cuda.synchronize)
        torch.cuda.synchronize()
        want.append(chain.results())
    same = lambda a, b: all(torch.equal(p, q) for p, q in zip(a, b))  # noqa: E731
    chains, streams = (Chain(), Chain()), (torch.cuda.Stream(), torch.cuda.Stream())
    torch.cuda.synchronize()
    got = []
    for i in range(12):
        for j in range(2):
            with torch.cuda.stream(streams[j]):
                chains[j].run(sources[(i + j) % 3])
                got.append((chains[j].results(), (i + j) % 3))
    torch.cuda.synchronize()
    assert all(same(r, want[i]) for r, i in got)
    source, graph = torch.empty_like(sources[0]), torch.cuda.CUDAGraph()
    source.copy_(sources[0])
    with torch.cuda.graph(graph):
        chain.run(source)
    for i in range(12):
        source.copy_(sources[i % 3])
        graph.replay()
        assert same(chain.results(), want[i % 3])
    assert gated.check() == 0 and down.check() == 0

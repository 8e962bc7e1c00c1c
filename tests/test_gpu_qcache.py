"""The 8-bit latent cache on the GPU against the float64 oracle.

Plan: every output equal. Append: codes and scales equal (scaling by a power of two is exact, the one rounding is to
nearest even on both sides). Attention, per element, with A = sum of weight * |v| and S = largest scale * sum |q||k|
of the row:
  output rounding to bf16                       2^-8 |o|
  weights kept to 8 bits at least               2^-8 A, and 2^-17 max|v| where a token's weight lies far below that of
                                                its neighbours (absolute error 2^-22 of theirs, 31 of them)
  scores: fp32 accumulation in at most 80 adds  2^-16 S   (80 * 2^-23, rounded up), the exponential and the products
                                                that form its argument included (a few 2^-23 of S)
  a query's bits below 2^-18 of its row's max   2^-18 max|q| * scale * sum|k|
A score error d moves a weight by d and the sum by d: twice that in o, once in lse.
"""
import numpy as np
import pytest
import torch

from oracle import qcache as Q
from oracle.formats import E4M3_TABLE

pytestmark = pytest.mark.gpu
LATENTS = [(512, 64), (256, 32), (128, 32), (64, 16)]


@pytest.fixture(scope="module")
def M():
    import mla_block_diffusion_gb300 as M
    from mla_block_diffusion_gb300 import build
    build.build()
    return M


def ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


# --- plan ----------------------------------------------------------------------------------------------------------
class Plan:
    def __init__(self, M, length, want, table, ring, state, max_new, max_seg):
        self.t, self.ring = ints(table), ints(ring)
        self.inputs = (ints(length), ints(want), self.ring, ints(state))
        bs = len(length)
        e = lambda n: torch.full((n,), -7, dtype=torch.int32, device="cuda")  # noqa: E731
        self.outs = (e(bs), e(2), e(bs + 1), e(max_new) if max_new else None, e(max_new) if max_new else None, e(max_seg + 1))
        self.cache = M.QCache(512, 64, (), (), self.t, n_pages=len(ring))

    def run(self):
        self.cache.plan(*self.inputs, *self.outs)
        return self.cache.check()


def check_plan(M, length, want, max_pages, n_pages, max_new, max_seg, seed=0, free=None, twice=True):
    rng = np.random.default_rng(seed)
    held = [Q._pages(n) if 0 <= n <= max_pages * 64 else 0 for n in length]
    pages = rng.permutation(n_pages).astype(np.int32)
    table = np.zeros((len(length), max_pages), dtype=np.int32)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = pages[at:at + h]
        at += h
    count = n_pages - at if free is None else free
    head = int(rng.integers(n_pages))
    ring = np.zeros(n_pages, dtype=np.int32)
    ring[(head + np.arange(count)) % n_pages] = pages[at:at + count]
    g = Plan(M, length, want, table, ring, (head, count), max_new, max_seg)
    st = g.run()
    t2, r2 = table.copy(), ring.copy()
    out, state, cu, slots, pos, seg = Q.plan(length, want, t2, r2, (head, count), max_new, max_seg)
    for _ in range(2 if twice else 1):  # a second call on the same inputs changes nothing
        got = [x.cpu().numpy() for x in g.outs if x is not None]
        assert np.array_equal(got[0], out) and tuple(got[1]) == state and np.array_equal(got[2], cu)
        if max_new:
            assert np.array_equal(got[3], slots) and np.array_equal(got[4], pos)
        assert np.array_equal(got[-1], seg)
        assert np.array_equal(g.t.cpu().numpy(), t2) and np.array_equal(g.ring.cpu().numpy(), r2)
        st |= g.run()
    return st


@pytest.mark.parametrize("length,want", [
    ([0], [1]), ([0], [0]), ([63], [64]), ([64], [65]), ([0], [64]), ([0], [65]), ([100], [0]), ([128], [64]), ([65], [63]),
    ([10, 64, 0, 200], [80, 64, 130, 5]), ([0] * 5, [0, 1, 0, 1, 0]),
])
def test_plan_small(M, length, want):
    new = sum(max(0, w - n) for n, w in zip(length, want))
    for room in {new, new + 1, new + 5}:
        assert check_plan(M, length, want, 8, 64, room, new + 3) == 0


@pytest.mark.parametrize("bs", [1, 3, 31, 32, 33, 255, 256, 257, 1000, 1024])
def test_plan_batches(M, bs):
    rng = np.random.default_rng(bs)
    length = rng.integers(0, 900, bs)
    want = np.where(rng.random(bs) < 0.25, rng.integers(0, 900, bs), length + rng.integers(0, 9, bs))
    new = int(np.maximum(want - length, 0).sum())
    assert check_plan(M, length.tolist(), want.tolist(), 16, 16 * bs + 64, new + 3, new // 64 + 2 * bs, seed=bs) == 0


def test_plan_long_prompts(M):
    rng = np.random.default_rng(5)
    want = rng.integers(1, 40000, 9)
    new = int(want.sum())
    assert check_plan(M, [0] * 9, want.tolist(), 700, 6000, new, new // 64 + 18) == 0


@pytest.mark.parametrize("free,room,spans", [(0, 1000, 99), (1, 1000, 99), (3, 1000, 99), (99, 0, 99), (99, 69, 99), (99, 70, 99),
                                             (99, 1000, 0), (99, 1000, 2), (99, 1000, 3)])
def test_plan_serves_in_order_while_there_is_room(M, free, room, spans):
    # what does not fit keeps its length, and so do the growing requests after it; shrinking ones are not held up
    assert check_plan(M, [60, 0, 128, 10, 7], [66, 64, 60, 11, 7], 4, 128, room, spans, free=free) == 0


def test_plan_reports_bad_lengths_and_rings(M):
    assert check_plan(M, [0, -1, 5, 600, 9], [64, 3, -2, 601, 70], 4, 64, 300, 99, twice=False) == 18
    g = Plan(M, [0], [64], np.zeros((1, 4)), np.zeros(8), (8, 1), 64, 4)      # the first free page lies outside the ring
    assert g.run() == 18 and g.outs[0].item() == 0 and g.outs[3].cpu().tolist() == [-1] * 64
    g = Plan(M, [0], [2], np.zeros((1, 4)), np.full(8, 8), (0, 1), 4, 4)      # no such page
    assert g.run() == 18 and g.outs[3].cpu().tolist() == [-1] * 4 and g.outs[4].cpu().tolist() == [0, 1, -1, -1]
    g = Plan(M, [128], [0], np.array([[3, 4, 0, 0]]), np.arange(8), (2, 7), 4, 4)  # one place for two pages
    assert g.run() == 18 and g.outs[1].cpu().tolist() == [2, 8] and g.ring.cpu().tolist() == [0, 3, 2, 3, 4, 5, 6, 7]


# --- append --------------------------------------------------------------------------------------------------------
def spans(length, want, table):
    slots, seg = [], []
    for b, (n, w) in enumerate(zip(length, want)):
        for p in range(n, w):
            if p == n or p % 64 == 0:
                seg.append(len(slots))
            slots.append(int(table[b, p // 64]) * 64 + p % 64)
    return np.array(slots, dtype=np.int32), np.array(seg + [len(slots)], dtype=np.int32)


def random_pages(rng, n_pages, D):
    codes = rng.integers(0, 256, (n_pages, 64, D), dtype=np.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x30
    return codes, (2.0 ** rng.integers(-9, -3, n_pages)).astype(np.float32)


@pytest.mark.parametrize("kv,rope", LATENTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("length,want", [
    ([0], [1]), ([0], [64]), ([0], [65]), ([63], [66]), ([1], [64]), ([10, 70, 0, 200, 64], [11, 70, 300, 328, 65]),
])
def test_append(M, kv, rope, dtype, length, want):
    D, layers, rng = kv + rope, 3, np.random.default_rng(kv + len(length))
    table = rng.permutation(40).astype(np.int32)[:len(length) * 6].reshape(len(length), 6)
    slots, seg = spans(length, want, table)
    pools = [random_pages(rng, 40, D) for _ in range(layers)]
    x = torch.from_numpy(rng.normal(0, 1, (layers, len(slots), D)) * 2.0 ** rng.integers(-3, 7, (layers, len(slots), 1))).to(dtype)
    x[1] = 0                                              # a layer of zeros
    pad = 3                                               # spare spans and rows that no span covers
    seg_d = ints(list(seg) + [seg[-1]] * pad)
    codes, scales = [torch.from_numpy(c).cuda() for c, _ in pools], [torch.from_numpy(s).cuda() for _, s in pools]
    cache = M.QCache(kv, rope, codes, scales, ints(table))
    cache.append(x.cuda(), ints(slots), seg_d)
    assert cache.check() == 0
    for l in range(layers):
        c, s = pools[l]
        Q.append(c, s, x[l].double().numpy(), slots, seg)
        assert np.array_equal(scales[l].cpu().numpy(), s)
        assert np.array_equal(E4M3_TABLE[codes[l].cpu().numpy()], E4M3_TABLE[c])


def test_append_strides_and_streams(M):
    kv, rope, D, rng = 128, 32, 160, np.random.default_rng(9)
    length, want = [5, 100], [70, 130]
    table = np.arange(8, dtype=np.int32).reshape(2, 4)
    slots, seg = spans(length, want, table)
    wide = torch.from_numpy(rng.normal(0, 1, (2, 2 * len(slots), D + 32))).to(torch.bfloat16).cuda()
    x = wide[:, ::2, 16:16 + D]                           # rows two apart, inside wider rows
    pools = [random_pages(rng, 8, D) for _ in range(2)]
    codes, scales = [torch.from_numpy(c).cuda() for c, _ in pools], [torch.from_numpy(s).cuda() for _, s in pools]
    cache = M.QCache(kv, rope, codes, scales, ints(table))
    s, e = ints(slots), ints(seg)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cache.append(x, s, e)
    side.synchronize()
    assert cache.check() == 0
    for l in range(2):
        c, sc = pools[l]
        Q.append(c, sc, x[l].double().cpu().numpy(), slots, seg)
        assert np.array_equal(codes[l].cpu().numpy(), c) and np.array_equal(scales[l].cpu().numpy(), sc)


def test_append_reports_bad_input(M):
    D, table = 80, np.arange(4, dtype=np.int32).reshape(1, 4)

    def go(x, slots, seg, scale=1.0):
        codes, scales = torch.zeros(4, 64, D, dtype=torch.uint8, device="cuda"), torch.full((4,), scale, device="cuda")
        cache = M.QCache(64, 16, [codes], [scales], ints(table))
        cache.append(x.cuda()[None], ints(slots), ints(seg))
        return cache.check(), E4M3_TABLE[codes.cpu().numpy()], scales.cpu().numpy()
    x = torch.ones(3, D, dtype=torch.bfloat16)
    x[1, 3], x[1, 4], x[2, 5] = float("nan"), float("inf"), float("-inf")
    st, c, s = go(x, [64, 65, 66], [0, 3])
    assert st == 17 and s[1] == 2.0 ** -8 and c[1, 1, 3] == 0 and c[1, 1, 4] == 448 and c[1, 2, 5] == -448 and c[1, 0, 0] == 256
    st, c, s = go(torch.full((1, D), 3e38, dtype=torch.float32), [0], [0, 1])
    assert st == 17 and s[0] == 2.0 ** 60 and np.all(c[0, 0] == 448)
    for scale in (0.3, 0.0, -1.0, float("nan"), 2.0 ** 61):
        assert go(torch.ones(1, D), [5], [0, 1], scale)[0] == 17     # the page holds tokens under no valid scale
        assert go(torch.ones(1, D), [0], [0, 1], scale)[0] == 0      # a page that starts over needs none
    one = torch.ones(3, D)
    for slots, seg in (([256], [0, 1]), ([-2], [0, 1]), ([62, 63, 64], [0, 3]), ([0, 1, 2], [0, 4]), ([0, 1, 2], [-1, 2]),
                       ([0, 1, 2], [2, 1])):
        st, c, s = go(one, slots, seg)
        assert st == 18 and not c.any() and np.all(s == 1)
    st, c, s = go(one, [-1, -1, -1], [0, 3])
    assert st == 0 and not c.any()


# --- attention -----------------------------------------------------------------------------------------------------
class Attend:
    """Inputs on the host and the device; unused pages and the places past a request's end hold NaN codes."""

    def __init__(self, M, kv, rope, H, length, nq, seed, sharp=1.0, exps=(-7, -4), max_pages=None, garbage=True):
        rng = np.random.default_rng(seed)
        self.kv, self.D, self.H, self.length, self.nq = kv, kv + rope, H, length, nq
        held = [Q._pages(n) for n in length]
        n_pages = sum(held) + 3
        order = rng.permutation(n_pages).astype(np.int32)
        self.table = np.zeros((len(length), max_pages or max(1, max(held))), dtype=np.int32)
        self.codes = np.full((n_pages, 64, self.D), 0x7F, dtype=np.uint8)
        self.scales = np.full(n_pages, 1.0, dtype=np.float32)
        at = 0
        for b, n in enumerate(length):
            self.table[b, :held[b]] = order[at:at + held[b]]
            self.table[b, held[b]:] = order[-1]          # an unused page of NaN
            for j in range(held[b]):
                pg, m = order[at + j], min(64, n - 64 * j)
                e = int(rng.integers(*exps))
                self.codes[pg, :m] = Q.e4m3_encode(rng.normal(0, 1, (m, self.D)) * 2.0 ** -e)
                self.scales[pg] = 2.0 ** e
            at += held[b]
        if not garbage:
            self.codes[self.codes == 0x7F] = 0
        self.cu = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
        q = rng.normal(0, sharp, (int(self.cu[-1]), H, self.D))
        self.q = torch.from_numpy(q).to(torch.bfloat16)
        self.scale = 1.3 / np.sqrt(self.D)
        self.dev = [torch.from_numpy(self.codes).cuda(), torch.from_numpy(self.scales).cuda(), ints(self.table)]
        self.cache = M.QCache(kv, rope, [self.dev[0]], [self.dev[1]], self.dev[2], n_heads=H)
        self.args = (ints(self.cu), ints(length))

    def run(self, causal, q=None, o=None):
        n = int(self.cu[-1])
        q = self.q.cuda() if q is None else q
        o = torch.full((n, self.H, self.kv), 9.0, dtype=torch.bfloat16, device="cuda") if o is None else o
        lse = torch.full((n, self.H), 9.0, device="cuda")
        self.cache.attend(0, q, *self.args, o, lse, causal=causal, scale=self.scale)
        return o, lse

    def check(self, causal, o, lse):
        o, lse, q = o.double().cpu().numpy(), lse.double().cpu().numpy(), self.q.double().numpy()
        for b, n in enumerate(self.length):
            a, z = self.cu[b], self.cu[b + 1]
            if a == z:
                continue
            wo, wl, absolute, top = Q.attend(self.codes, self.scales, self.table[b], n, q[a:z], self.kv, causal, self.scale)
            none = ~np.isfinite(wl)
            assert np.all(o[a:z][none] == 0) and np.all(lse[a:z][none] == -np.inf)
            k = np.concatenate([E4M3_TABLE[self.codes[p]] * self.scales[p] for p in self.table[b, :Q._pages(n)]])[:n] \
                if n else np.zeros((1, self.D))
            low = 2.0 ** -18 * np.abs(q[a:z]).max(2) * self.scale * np.abs(k).sum(1).max()
            ds = 2.0 ** -16 * top + low
            tol = 2.0 ** -8 * np.abs(wo) + (2.0 ** -8 + 2 * ds[..., None]) * absolute + 2.0 ** -17 * np.abs(k).max()
            assert np.all(np.abs(o[a:z] - wo) <= tol + 1e-30), (b, np.max(np.abs(o[a:z] - wo) / (tol + 1e-30)))
            fin = ~none
            assert np.all(np.abs(lse[a:z][fin] - wl[fin]) <= ds[fin] + 2.0 ** -22 * (1 + np.abs(wl[fin]))), b


@pytest.mark.parametrize("kv,rope", LATENTS)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("H,length,nq", [
    (8, [128], [7]), (1, [1], [1]), (64, [1], [1]), (64, [64], [1]), (64, [65], [1]), (64, [200], [7]), (5, [0], [3]),
    (64, [0, 70], [2, 0]), (40, [300, 0, 63, 129], [3, 5, 1, 0]), (128, [90, 257], [1, 2]), (16, [1000, 20], [9, 20]),
    (3, [50], [50]), (64, [191, 192, 193], [1, 1, 1]), (12, [2000], [1]),
])
def test_attend(M, kv, rope, causal, H, length, nq):
    t = Attend(M, kv, rope, H, length, nq, seed=H + sum(length))
    o, lse = t.run(causal)
    assert t.cache.check() == 0
    t.check(causal, o, lse)


@pytest.mark.parametrize("kv,rope", LATENTS)
@pytest.mark.parametrize("H,length,nq", [
    (64, [300], [200]), (100, [130, 77, 2], [60, 77, 9]),  # more tiles than CTAs
    (7, [40 * i % 700 for i in range(300)], [i % 3 for i in range(300)]),  # many small requests
    (64, [12000, 100, 100, 100], [1, 1, 1, 1]),            # one request far longer than the others
])
def test_attend_divisions_of_the_work(M, kv, rope, H, length, nq):
    t = Attend(M, kv, rope, H, length, nq, seed=13)
    o, lse = t.run(True)
    assert t.cache.check() == 0
    t.check(True, o, lse)


@pytest.mark.parametrize("kv,rope", LATENTS)
def test_attend_rows_of_every_magnitude(M, kv, rope):
    # neighbouring query rows 2^-120 .. 2^8 times unit size, one all zero: none disturbs another
    t = Attend(M, kv, rope, 20, [333], [4], seed=14)
    e = torch.linspace(-120, 8, 80)[torch.randperm(80, generator=torch.Generator().manual_seed(1))].round()
    q = t.q.float().reshape(80, t.D) * torch.exp2(e)[:, None]
    q[17] = 0
    t.q = q.reshape(4, 20, t.D).to(torch.bfloat16)
    o, lse = t.run(False)
    assert t.cache.check() == 0
    t.check(False, o, lse)


@pytest.mark.parametrize("kv,rope", LATENTS)
def test_attend_queries_before_the_cache(M, kv, rope):
    # causal with more queries than cached tokens: the first ones see nothing
    t = Attend(M, kv, rope, 9, [5, 64, 1], [12, 70, 2], seed=3)
    o, lse = t.run(True)
    assert t.cache.check() == 0 and torch.isinf(lse[:7]).all() and not torch.isinf(lse[7:12]).any()
    t.check(True, o, lse)


@pytest.mark.parametrize("kv,rope", LATENTS)
def test_attend_long_and_ragged(M, kv, rope):
    # split over many CTAs, requests that end in every part of a page, one empty
    t = Attend(M, kv, rope, 16, [9001, 3, 0, 4999, 640, 1], [1, 1, 1, 2, 1, 1], seed=4)
    o, lse = t.run(True)
    assert t.cache.check() == 0
    t.check(True, o, lse)
    o2, lse2 = t.run(True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)  # the same result every time


@pytest.mark.parametrize("kv,rope", LATENTS)
@pytest.mark.parametrize("sharp", [8.0, 60.0])
def test_attend_sharp_and_far_apart_scales(M, kv, rope, sharp):
    # scores of hundreds, page scales many binades apart: the running reference moves a long way
    t = Attend(M, kv, rope, 8, [700, 150], [2, 1], seed=5, sharp=sharp, exps=(-12, 4))
    o, lse = t.run(False)
    assert t.cache.check() == 0
    t.check(False, o, lse)


@pytest.mark.parametrize("kv,rope", LATENTS)
@pytest.mark.parametrize("H,length,nq", [
    (64, [20000], [1]), (20, [9000, 5000], [1, 2]), (5, [7000, 0, 64], [1, 1, 1]), (33, [4500], [3]), (64, [9000, 2049], [1, 1]),
])
def test_attend_few_long_requests(M, kv, rope, H, length, nq):
    # one to four tiles in many pieces each: several warps add up a row
    t = Attend(M, kv, rope, H, length, nq, seed=16)
    o, lse = t.run(True)
    assert t.cache.check() == 0
    t.check(True, o, lse)
    o2, lse2 = t.run(True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kv,rope", LATENTS)
@pytest.mark.parametrize("size", [2.0 ** 13, 2.0 ** 18, 2.0 ** 23])
def test_attend_huge_scores(M, kv, rope, size):
    # every query looks at the last element alone, which is 1 or -1: scores are size * scale or its negative, equal weights
    # for the tokens on the winning side. Products and the exponent's differences are exact; the weights' two terms and the
    # output round (2^-9 each), the score's factors, sum and logarithm in fp32 (eight roundings of 2^-24).
    t = Attend(M, kv, rope, 6, [700, 130, 90], [3, 1, 2], seed=15)
    for b, n in enumerate(t.length):
        for j in range(n):
            pg = t.table[b, j // 64]
            up = (j >= 500, j < 64, True)[b]
            t.codes[pg, j % 64, -1] = Q.e4m3_encode(np.float64((1 if up else -1) / t.scales[pg]))
    t.dev[0].copy_(torch.from_numpy(t.codes))
    t.q = torch.zeros_like(t.q)
    t.q[..., -1] = size * torch.tensor([1.0, -1.0]).repeat(3)
    o, lse = t.run(False)
    assert t.cache.check() == 0
    for b, n in enumerate(t.length):
        a, z = t.cu[b], t.cu[b + 1]
        wo, wl, absolute, _ = Q.attend(t.codes, t.scales, t.table[b], n, t.q[a:z].double().numpy(), kv, False, t.scale)
        assert np.all(np.abs(o[a:z].double().cpu().numpy() - wo) <= 2.0 ** -8 * (np.abs(wo) + absolute))
        assert np.all(np.abs(lse[a:z].double().cpu().numpy() - wl) <= 2.0 ** -21 * (1 + np.abs(wl)))


@pytest.mark.parametrize("kv,rope", LATENTS)
def test_attend_one_token_outweighs_the_rest(M, kv, rope):
    # the first token takes half of every row's weight, thousands of others share the rest
    t = Attend(M, kv, rope, 8, [6000], [1], seed=6, sharp=0.4, exps=(-4, -3))
    q = t.q.double().numpy()
    want = np.log(6000.0) / t.scale
    first = q[0].mean(0)
    first *= want / (first @ first)
    pg = t.table[0, 0]
    t.codes[pg, 0] = Q.e4m3_encode(first / t.scales[pg])
    t.dev[0].copy_(torch.from_numpy(t.codes))
    t.q = torch.from_numpy(np.repeat(q.mean(1, keepdims=True), 8, axis=1)).to(torch.bfloat16)
    o, lse = t.run(False)
    assert t.cache.check() == 0
    t.check(False, o, lse)


@pytest.mark.parametrize("kv,rope", LATENTS)
def test_attend_strides_and_streams(M, kv, rope):
    t = Attend(M, kv, rope, 6, [100, 77], [3, 2], seed=7)
    wq = torch.zeros(5, 7 * t.D + 8, dtype=torch.bfloat16, device="cuda")
    q = wq[:, 8:8 + 6 * t.D].unflatten(1, (6, t.D))
    q.copy_(t.q.cuda())
    wo = torch.full((5, 6 * kv + 40), 5.0, dtype=torch.bfloat16, device="cuda")
    o = wo[:, 16:16 + 6 * kv].unflatten(1, (6, kv))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _, lse = t.run(True, q=q, o=o)
    side.synchronize()
    assert t.cache.check() == 0
    t.check(True, o, lse)
    assert torch.all(wo[:, :16] == 5) and torch.all(wo[:, 16 + 6 * kv:] == 5)


def test_attend_without_lse_and_with_no_queries(M):
    t = Attend(M, 512, 64, 64, [100], [1], seed=8)
    o, lse = t.run(False)
    o2 = torch.zeros_like(o)
    t.cache.attend(0, t.q.cuda(), *t.args, o2, None, causal=False, scale=t.scale)
    assert t.cache.check() == 0 and torch.equal(o, o2)
    t = Attend(M, 512, 64, 64, [100, 3], [0, 0], seed=8)
    t.run(True)
    assert t.cache.check() == 0


@pytest.mark.parametrize("kv,rope", [(512, 64), (64, 16)])
def test_attend_in_a_graph_with_other_lengths(M, kv, rope):
    # captured once, replayed with lengths that change on the device
    t = Attend(M, kv, rope, 64, [900, 400], [1, 1], seed=9)
    o, lse = t.run(True)
    g = torch.cuda.CUDAGraph()
    q = t.q.cuda()
    o, lse = torch.zeros_like(o), torch.zeros_like(lse)
    with torch.cuda.graph(g):
        t.cache.attend(0, q, *t.args, o, lse, causal=True, scale=t.scale)
    for length in ([900, 400], [1, 399], [0, 65], [770, 0]):
        t.args[1].copy_(ints(length))
        g.replay()
        torch.cuda.synchronize()
        t.length = length
        t.check(True, o, lse)
    assert t.cache.check() == 0


@pytest.mark.parametrize("kv,rope", LATENTS)
def test_attend_reports_bad_input(M, kv, rope):
    t = Attend(M, kv, rope, 4, [100, 80, 60], [2, 2, 1], seed=10)
    o, lse = t.run(False)
    q = t.q.clone()
    q[1, 2, 5] = float("nan")
    q[3, 0, 0] = float("-inf")
    o2, lse2 = t.run(False, q=q.cuda())
    assert t.cache.check() == 17
    hit = torch.zeros(5, 4, dtype=torch.bool, device="cuda")
    hit[1, 2] = hit[3, 0] = True
    assert torch.isnan(o2[hit]).all() and torch.isnan(lse2[hit]).all()      # those rows, and no others
    assert torch.equal(o2[~hit], o[~hit]) and torch.equal(lse2[~hit], lse[~hit])
    for cu, length in (([0, 2, 4, 6], [100, 80, 60]), ([0, 2, 1, 1], [100, 80, 60]), ([0, 2, 4, 5], [100, 129, 60]),
                       ([0, 2, 4, 5], [100, -1, 60]), ([-1, 2, 4, 5], [100, 80, 60])):
        t.args[0].copy_(ints(cu))
        t.args[1].copy_(ints(length))
        o3, _ = t.run(False)
        assert t.cache.check() == 18
        ok = [b for b in range(3) if 0 <= cu[b] <= cu[b + 1] <= 5 and 0 <= length[b] <= 128]
        for b in ok:                                                       # the other requests are served
            if (cu[b], cu[b + 1]) == (t.cu[b], t.cu[b + 1]):
                assert torch.equal(o3[cu[b]:cu[b + 1]], o[cu[b]:cu[b + 1]])
    t.args[0].copy_(ints(t.cu))
    t.args[1].copy_(ints(t.length))
    for value in (-1, len(t.scales), 1 << 30):
        t.dev[2][1, 1] = value
        o3, _ = t.run(False)
        assert t.cache.check() == 18 and torch.equal(o3[:2], o[:2])
    t.dev[2].copy_(ints(t.table))
    t.dev[1][int(t.table[2, 0])] = 0.75
    t.run(False)
    assert t.cache.check() == 17


def test_binding_refuses_what_does_not_fit(M):
    t = Attend(M, 64, 16, 4, [100, 80], [2, 1], seed=15)
    q, o, lse = t.q.cuda(), torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, 4, device="cuda")
    cu, length = t.args
    bad = [dict(q=q.half()), dict(q=q[:, :, :72]), dict(q=q.cpu()), dict(o=o[:2]), dict(o=o.float()), dict(lse=lse[:2]),
           dict(lse=lse.double()), dict(cu=cu.long()), dict(cu=cu[:2]), dict(length=length.long()), dict(length=length.cpu()),
           dict(q=q.transpose(0, 1)[:3]), dict(q=torch.zeros(3, 4, 160, dtype=torch.bfloat16, device="cuda")[:, :, ::2]),
           dict(length=ints([1, 1, 1]), cu=ints([0, 1, 2, 3]))]
    for kw in bad:
        a = dict(q=q, cu=cu, length=length, o=o, lse=lse) | kw
        with pytest.raises(ValueError):
            t.cache.attend(0, a["q"], a["cu"], a["length"], a["o"], a["lse"])
    with pytest.raises(M.DSparkError):
        t.cache.attend(1, q, cu, length, o, lse)                       # no such layer
    with pytest.raises(M.DSparkError):
        t.cache.attend(0, q, cu, length, o, lse, scale=-1.0)
    x, slots, seg = torch.zeros(1, 3, 80, device="cuda"), ints([0, 1, 2]), ints([0, 3])
    for kw in (dict(x=x[0]), dict(x=x.half()), dict(x=x.cpu()), dict(x=x[:, :, :64]), dict(x=x.expand(2, 3, 80)),
               dict(slots=slots.long()), dict(seg=seg.cpu()), dict(x=torch.zeros(1, 3, 160, device="cuda")[:, :, ::2])):
        a = dict(x=x, slots=slots, seg=seg) | kw
        with pytest.raises(ValueError):
            t.cache.append(a["x"], a["slots"], a["seg"])
    with pytest.raises(M.DSparkError):
        t.cache.append(torch.zeros(1, 3, 82, device="cuda")[:, :, :80], slots, seg)  # rows off the 16-byte grid
    g = Plan(M, [5, 6], [7, 8], np.zeros((2, 4)), np.zeros(8), (0, 8), 4, 4)
    for i in range(9):                                                   # each argument in turn too short or of another type
        args = list(g.inputs + g.outs)
        for other in (args[i].long(), args[i][:0] if i not in (7, 8) else args[i].cpu()):
            if other.numel() == 0 and i == 0:
                continue                                                 # no requests at all: the library's own refusal
            with pytest.raises(ValueError):
                g.cache.plan(*(args[:i] + [other] + args[i + 1:]))
    with pytest.raises(M.DSparkError):
        g.cache.plan(ints([]), ints([]), *g.inputs[2:], *g.outs)
    with pytest.raises(ValueError):
        M.QCache(64, 16, [t.dev[0]], [], t.dev[2])
    with pytest.raises(ValueError):
        M.QCache(128, 32, [t.dev[0]], [t.dev[1]], t.dev[2])
    with pytest.raises(ValueError):
        M.QCache(64, 16, [t.dev[0]], [t.dev[1].double()], t.dev[2])
    with pytest.raises(M.DSparkError):
        M.QCache(64, 32, (), (), t.dev[2], n_pages=4)                    # no such latent width


def test_attend_pages_past_32_bits(M):
    # a pool of 4.8 GB whose used pages lie past byte 2^32
    kv, rope, n, rng = 512, 64, 130_000, np.random.default_rng(11)
    codes = torch.empty(n, 64, 576, dtype=torch.uint8, device="cuda")
    scales = torch.ones(n, device="cuda")
    table = ints([[n - 1, n - 7, 121_000]])
    x = torch.from_numpy(rng.normal(0, 1, (1, 150, 576))).to(torch.bfloat16)
    cache = M.QCache(kv, rope, [codes], [scales], table, n_heads=64)
    slots, seg = spans([0], [150], table.cpu().numpy())
    cache.append(x.cuda(), ints(slots), ints(seg))
    t = Attend(M, kv, rope, 64, [150], [1], seed=12)
    used = table[0].cpu().numpy()
    c, s = np.zeros((3, 64, 576), dtype=np.uint8), np.ones(3, dtype=np.float32)
    near, _ = spans([0], [150], np.arange(3, dtype=np.int32)[None])
    Q.append(c, s, x[0].double().numpy(), near, seg)
    assert np.array_equal(codes[used.tolist()].cpu().numpy()[:2], c[:2])
    t.codes, t.scales, t.table = c, s, np.arange(3, dtype=np.int32)[None]
    t.cache = cache
    o, lse = t.run(True)
    assert cache.check() == 0
    t.check(True, o, lse)

"""The 8-bit latent cache on the GPU at the ends of its documented ranges, and where it reports instead of answering.

Attention is compared at the tolerances of test_gpu_qcache.Attend.check, which that file derives."""
import numpy as np
import pytest
import torch

from oracle import qcache as Q
from oracle.formats import E4M3_TABLE
from test_gpu_qcache import LATENTS, Attend, M, Plan, ints  # noqa: F401

pytestmark = pytest.mark.gpu


class Laid(Attend):
    """Attention inputs from given pages: codes [n, 64, D], scales [n], table [bs, pages], q [total, H, D]."""

    def __init__(self, M, kv, codes, scales, table, length, nq, q):
        self.kv, self.D, self.H, self.length, self.nq = kv, codes.shape[2], q.shape[1], length, nq
        self.codes, self.scales, self.table = codes, np.asarray(scales, dtype=np.float32), np.asarray(table, dtype=np.int32)
        self.cu = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
        self.q, self.scale = torch.from_numpy(q).to(torch.bfloat16), 1.3 / np.sqrt(self.D)
        self.dev = [torch.from_numpy(codes).cuda(), torch.from_numpy(self.scales).cuda(), ints(self.table)]
        self.cache = M.QCache(kv, self.D - kv, [self.dev[0]], [self.dev[1]], self.dev[2], n_heads=self.H)
        self.args = (ints(self.cu), ints(length))


def page(rng, kv, D, e, last, size=1.0):
    """A page at scale 2^e: normal values, zero key-only elements but for the last, which steers the scores."""
    v = np.zeros((64, D))
    v[:, :kv] = rng.normal(0, size, (64, kv))
    v[:, -1] = last
    return Q.e4m3_encode(v * 2.0 ** -e)


def check_steered(t, o, lse):
    """Like Attend.check, for queries whose last element alone is not zero: both its terms are exact, so that the scores
    lose only what fp32 does."""
    o, lse, q = o.double().cpu().numpy(), lse.double().cpu().numpy(), t.q.double().numpy()
    for b, n in enumerate(t.length):
        a, z = t.cu[b], t.cu[b + 1]
        wo, wl, absolute, top = Q.attend(t.codes, t.scales, t.table[b], n, q[a:z], t.kv, False, t.scale)
        ds, v = 2.0 ** -16 * top, (E4M3_TABLE[t.codes] * t.scales[:, None, None])[:, :, :t.kv]
        tol = 2.0 ** -8 * np.abs(wo) + (2.0 ** -8 + 2 * ds[..., None]) * absolute + 2.0 ** -17 * np.abs(v).max()
        assert np.all(np.abs(o[a:z] - wo) <= tol), b
        assert np.all(np.abs(lse[a:z] - wl) <= ds + 2.0 ** -22 * (1 + np.abs(wl))), b


# Divisions of the work on 152 SMs: with 304 requests of 11 chunks every CTA holds whole requests; 76 requests of 24
# chunks are cut in two pieces of 12 chunks.
@pytest.mark.parametrize("kv,rope", LATENTS)
@pytest.mark.parametrize("H", [2, 34])
def test_attend_references_that_move_with_every_chunk(M, kv, rope, H):
    # Scores of the first two heads grow by 2^70 from chunk to chunk, so that what came before is scaled away, while the
    # others' stay at zero: the warps of those rows fall behind the others', whose references stay. The result is right,
    # and the same every time.
    D, bs, rng = kv + rope, 76, np.random.default_rng(20)
    levels = [-(448 - 32 * i) / 256 for i in range(12)]
    codes = np.stack([page(rng, kv, D, -8, x) for x in levels])
    row = np.repeat(list(range(12)) * 2, 2)
    q = np.zeros((bs, H, D))
    q[:, :2, -1] = 14 * 70 * np.log(2) / (1.75 * 1.3 / np.sqrt(D))
    t = Laid(M, kv, codes, [2.0 ** -8] * 12, [row] * bs, [3067] * bs, [1] * bs, q)
    o, lse = t.run(False)
    assert t.cache.check() == 0
    check_steered(t, o, lse)
    for _ in range(20):
        o2, lse2 = t.run(False)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert t.cache.check() == 0




@pytest.mark.parametrize("kv,rope", LATENTS)
@pytest.mark.parametrize("bs,chunks", [(304, 11), (76, 24)])
def test_attend_zero_pages_behind_low_scores(M, kv, rope, bs, chunks):
    # Scores of 2^-110 on pages of scale 2^-8, then 1280 tokens and more on all-zero pages (scale 2^-60), where the
    # scores are zero; one normal page at the end of the longer ones. The zero pages outweigh what comes first by 2^110,
    # and value scales are 2^52 apart.
    D, H, rng = kv + rope, 2, np.random.default_rng(21)
    codes = np.stack([page(rng, kv, D, -8, -1.75), page(rng, kv, D, -8, -1.75), np.zeros((64, D), dtype=np.uint8),
                      page(rng, kv, D, -7, 0.0)])
    row = [0, 1] + [2] * (2 * chunks - 2)
    if chunks == 24:
        row[-1] = 3
    q = np.zeros((bs, H, D))
    q[:, :, -1] = np.linspace(76.0, 76.9, bs * H).reshape(bs, H) / (1.75 * 1.3 / np.sqrt(D))
    t = Laid(M, kv, codes, [2.0 ** -8, 2.0 ** -8, 2.0 ** -60, 2.0 ** -7], [row] * bs, [128 * chunks - 5] * bs, [1] * bs, q)
    o, lse = t.run(False)
    assert t.cache.check() == 0 and torch.isfinite(lse).all()
    check_steered(t, o, lse)


@pytest.mark.parametrize("kv,rope", LATENTS)
def test_attend_pieces_at_both_ends_of_the_page_scales(M, kv, rope):
    # The first of two pieces begins with a page of scale 2^60 and scores of zero, the second with scores of 2^-67 on a
    # page of 2^-8 and goes on with 2^-8: together those tokens weigh a sixteenth of the first page.
    D, H, bs, rng = kv + rope, 2, 76, np.random.default_rng(22)
    codes = np.stack([page(rng, kv, D, 60, 0.0, size=2.0 ** 60), page(rng, kv, D, -8, -1.75), page(rng, kv, D, -8, -56 / 256)])
    row = [0, 1] + [2] * 22 + [1, 1] + [2] * 22
    q = np.zeros((bs, H, D))
    q[:, :, -1] = np.linspace(46.5, 46.9, bs * H).reshape(bs, H) / (1.75 * 1.3 / np.sqrt(D))
    t = Laid(M, kv, codes, [2.0 ** 60, 2.0 ** -8, 2.0 ** -8], [row] * bs, [3067] * bs, [1] * bs, q)
    o, lse = t.run(False)
    assert t.cache.check() == 0
    check_steered(t, o, lse)


@pytest.mark.parametrize("kv,rope", LATENTS)
@pytest.mark.parametrize("length", [[700, 130, 90], [9000, 130, 90]])
def test_attend_reports_scores_beyond_the_range(M, kv, rope, length):
    # A query that looks at the last element alone, which is 1 or -1: scores of +-12 million or infinite. Its row is NaN
    # and reported; no other row changes.
    t = Attend(M, kv, rope, 6, length, [3, 1, 2], seed=23)
    for b, n in enumerate(t.length):
        for j in range(n):
            pg = t.table[b, j // 64]
            up = (j >= 500, j < 64, True)[b]
            t.codes[pg, j % 64, -1] = Q.e4m3_encode(np.float64((1 if up else -1) / t.scales[pg]))
    t.dev[0].copy_(torch.from_numpy(t.codes))
    o, lse = t.run(True)
    assert t.cache.check() == 0
    t.check(True, o, lse)
    hit = torch.zeros(6, 6, dtype=torch.bool, device="cuda")
    for i, h, value in ((0, 1, 1.2e7), (1, 5, -1.2e7), (2, 0, 3e38 * t.scale), (3, 3, -3e38 * t.scale), (4, 2, 1.2e7), (5, 4, -1.2e7)):
        t.q[i, h] = 0
        t.q[i, h, -1] = value / t.scale
        hit[i, h] = True
    o2, lse2 = t.run(True)
    assert t.cache.check() == 17
    assert torch.isnan(o2[hit]).all() and torch.isnan(lse2[hit]).all()
    assert torch.equal(o2[~hit], o[~hit]) and torch.equal(lse2[~hit], lse[~hit])


@pytest.mark.parametrize("kv,rope", LATENTS)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("length,nq,at", [
    ([80, 200, 100], [1, 150, 2], 2),          # many tiles; causal: the first 78 queries end before the bad page
    ([80, 20000, 100], [1, 1, 2], 100),        # one request in many pieces
    ([80, 65, 100], [1, 3, 2], 1),             # the last page, one token
])
def test_attend_marks_rows_over_bad_pages(M, kv, rope, causal, length, nq, at):
    # a page number outside the pool, or a scale that is no power of two in range: the rows that see that page are NaN,
    # and no others
    t = Attend(M, kv, rope, 4, length, nq, seed=24)
    o, lse = t.run(causal)
    assert t.cache.check() == 0
    t.check(causal, o, lse)
    i = np.arange(nq[1])
    sees = length[1] - nq[1] + i + 1 if causal else np.full(nq[1], length[1])
    hit = torch.zeros(sum(nq), dtype=torch.bool, device="cuda")
    hit[1:1 + nq[1]] = torch.from_numpy(sees > 64 * at).cuda()

    def check(status):
        o2, lse2 = t.run(causal)
        assert t.cache.check() == status
        assert torch.isnan(o2[hit]).all() and torch.isnan(lse2[hit]).all()
        assert torch.equal(o2[~hit], o[~hit]) and torch.equal(lse2[~hit], lse[~hit])
    for number in (-1, len(t.scales), 1 << 30, -(1 << 31)):
        t.dev[2][1, at] = number
        check(18)
    t.dev[2].copy_(ints(t.table))
    for scale in (0.75, 0.0, -1.0, float("nan"), float("inf"), 2.0 ** 61, 2.0 ** -61):
        t.dev[1][int(t.table[1, at])] = scale
        check(17)


def test_plan_reports_a_bad_page_when_it_comes_back(M):
    # a ring that holds a page outside the pool: reported when it is taken, and again when its request gives it back
    g = Plan(M, [0], [2], np.zeros((1, 4)), np.full(8, 8), (0, 1), 4, 4)
    assert g.run() == 18 and g.outs[0].item() == 2 and g.outs[3].cpu().tolist() == [-1] * 4
    h = Plan(M, [2], [0], g.t.cpu().numpy(), g.ring.cpu().numpy(), tuple(g.outs[1].tolist()), 4, 4)
    assert h.run() == 18 and h.outs[0].item() == 0


@pytest.mark.parametrize("kv,rope", LATENTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_refuses_spans_that_are_not_one_run_of_slots(M, kv, rope, dtype):
    # rows of a span whose slots do not follow one another: reported, and nothing of that page is written
    D, rng = kv + rope, np.random.default_rng(25)
    x = torch.from_numpy(rng.normal(0, 1, (1, 64, D))).to(dtype).cuda()

    def go(slots, seg):
        codes, scales = torch.zeros(4, 64, D, dtype=torch.uint8, device="cuda"), torch.ones(4, device="cuda")
        cache = M.QCache(kv, rope, [codes], [scales], ints([[0, 1, 2, 3]]))
        cache.append(x, ints(slots), ints(seg))
        return cache.check(), codes.cpu().numpy(), scales.cpu().numpy()
    whole = list(range(64, 128))
    assert go(whole, [0, 64])[0] == 0
    for at, value in ((1, -1), (63, -1), (63, 126), (5, 70), (40, 1 << 30), (2, 66 + 64), (1, 64), (7, -(1 << 31))):
        slots = list(whole)
        slots[at] = value
        st, c, s = go(slots, [0, 64])
        assert st == 18 and not c.any() and np.all(s == 1), (at, value)
    st, c, s = go([-1, 65, 66], [0, 3])                      # a skipped first row takes no others with it unseen
    assert st == 18 and not c.any()
    st, c, s = go([-1, -1, -1, 130, 131, 9, 11], [0, 3, 5, 7])
    assert st == 18 and not c[0].any() and not c[1].any() and c[2, 2:4].any(1).all()
    assert np.all(s == 1)                                    # page 2 holds tokens under the larger scale of 1
    st, c, s = go([-1, -1, 130, 131], [0, 2, 4])
    assert st == 0 and c[2, 2:4].any(1).all()


def test_plan_fills_the_largest_slot_map_exactly(M):
    # max_new at its limit, 2^30: one request takes all of it, the next must wait (its one token has no slot)
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB of free device memory")
    most, n_pages = 1 << 30, (1 << 24) + 8
    e = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = M.QCache(512, 64, (), (), torch.zeros(2, 1 << 24, dtype=torch.int32, device="cuda"), n_pages=n_pages)
    out, state, cu, slots, pos, seg = e(2), e(2), e(3), e(most), e(most), e((1 << 24) + 9)
    cache.plan(ints([0, 0]), ints([most, 5]), torch.arange(n_pages, dtype=torch.int32, device="cuda"), ints([0, n_pages]),
               out, state, cu, slots, pos, seg)
    assert cache.check() == 0
    assert out.tolist() == [most, 0] and state.tolist() == [1 << 24, 8] and cu.tolist() == [0, most, most]
    assert slots[-1].item() == most - 1 and pos[-1].item() == most - 1 and seg[-8:].tolist() == [most] * 8


# --- forms that a server meets -------------------------------------------------------------------------------------
def test_append_take_back_and_append_again(M):
    # a draft-and-verify loop: tokens are drafted, some are taken back, others come in their place. A page's scale never
    # falls while the page holds tokens, and its codes are those of the same steps on the host.
    kv, rope, D, rng = 128, 32, 160, np.random.default_rng(26)
    codes, scales = np.zeros((6, 64, D), dtype=np.uint8), np.ones(6, dtype=np.float32)
    dev = [torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()]
    table, ring = np.zeros((1, 3), dtype=np.int32), np.array([3, 1, 5, 0, 2, 4], dtype=np.int32)
    cache = M.QCache(kv, rope, [dev[0]], [dev[1]], ints(table))
    ring_d, length, state = ints(ring), ints([0]), ints([0, 6])
    host_length, host_state = [0], (0, 6)
    want = 0
    kept = []                                                # the tokens as they came
    for step in range(40):
        new = int(rng.integers(1, 9))
        fresh = [want + new, max(0, want + new - int(rng.integers(0, new + 1)))]   # drafted, then what is accepted
        for w in fresh:
            outs = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (1, 2, 2, 8, 8, 4)]
            cache.plan(length, ints([w]), ring_d, state, *outs)
            got = Q.plan(host_length, [w], table, ring, host_state, 8, 3)
            assert cache.check() == 0
            for a, b in zip(outs, got):
                assert a.cpu().tolist() == list(b)
            if w > host_length[0]:
                x = rng.normal(0, 1, (1, 8, D)) * 2.0 ** rng.integers(-6, 6)
                x = torch.from_numpy(x).to(torch.bfloat16)
                cache.append(x.cuda(), outs[3], outs[5])
                assert cache.check() == 0
                Q.append(codes, scales, x[0].double().numpy(), got[3], got[5])
                kept = kept[:host_length[0]] + list(x[0, :w - host_length[0]].double().numpy())
            length, state, host_length, host_state, want = outs[0], outs[1], [w], got[1], w
            assert np.array_equal(dev[1].cpu().numpy(), scales)
            assert np.array_equal(E4M3_TABLE[dev[0].cpu().numpy()], E4M3_TABLE[codes])
    # what all raises together cost: one rounding, 2^-4 of an element, and less than 2^(e - 9) once it is below the
    # normal range of its page (each raise to 2^e' rounds by at most half the smallest step, 2^(e' - 10), and e' differ)
    for p in range(want):
        pg = table[0, p // 64]
        got, s = E4M3_TABLE[codes[pg, p % 64]] * scales[pg], float(scales[pg])
        assert np.all(np.abs(got - kept[p]) <= 2.0 ** -4 * np.abs(kept[p]) + s * 2.0 ** -9)


def test_whole_step_in_a_graph(M):
    # plan, append and attention captured together, replayed while the wanted lengths change on the device
    kv, rope, H, bs, most, D = 256, 32, 16, 3, 96, 288
    rng = np.random.default_rng(27)
    n_pages, width = 20, 8
    codes, scales = torch.zeros(n_pages, 64, D, dtype=torch.uint8, device="cuda"), torch.ones(n_pages, device="cuda")
    table = torch.zeros(bs, width, dtype=torch.int32, device="cuda")
    cache = M.QCache(kv, rope, [codes], [scales], table, n_heads=H)
    length, state, want, ring = ints([0] * bs), ints([3, n_pages]), ints([0] * bs), ints(rng.permutation(n_pages))
    e = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    after, state_after, cu, slots, pos, seg = e(bs), e(2), e(bs + 1), e(most), e(most), e(10)
    x = torch.zeros(1, most, D, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(most, H, D, dtype=torch.bfloat16, device="cuda")
    o, lse = torch.zeros(most, H, kv, dtype=torch.bfloat16, device="cuda"), torch.zeros(most, H, device="cuda")
    host = {"length": [0] * bs, "state": (3, n_pages), "table": np.zeros((bs, width), dtype=np.int32), "ring": ring.cpu().numpy(),
            "codes": codes.cpu().numpy(), "scales": scales.cpu().numpy()}

    def step():
        cache.plan(length, want, ring, state, after, state_after, cu, slots, pos, seg)
        cache.append(x, slots, seg)
        cache.attend(0, q, cu, after, o, lse, causal=True, scale=0.07)
        length.copy_(after)
        state.copy_(state_after)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                               # nothing wanted: nothing changes
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for wanted in ([70, 0, 3], [71, 20, 4], [72, 21, 60], [60, 0, 70], [64, 33, 129], [128, 34, 130], [0, 200, 131], [1, 35, 0]):
        want.copy_(ints(wanted))
        x.copy_(torch.from_numpy(rng.normal(0, 1, (1, most, D)) * 2.0 ** rng.integers(-2, 3)))
        q.copy_(torch.from_numpy(rng.normal(0, 1, (most, H, D))))
        g.replay()
        assert cache.check() == 0
        before = host["length"]
        out, host["state"], host_cu, host_slots, _, host_seg = Q.plan(before, wanted, host["table"], host["ring"], host["state"], most, 9)
        host["length"] = out.tolist()
        Q.append(host["codes"], host["scales"], x[0].double().cpu().numpy(), host_slots, host_seg)
        assert length.tolist() == host["length"] and state.tolist() == list(host["state"]) and cu.tolist() == host_cu.tolist()
        assert np.array_equal(codes.cpu().numpy(), host["codes"]) and np.array_equal(scales.cpu().numpy(), host["scales"])
        total = int(host_cu[-1])
        t = Laid(M, kv, host["codes"], host["scales"], host["table"], host["length"], np.diff(host_cu).tolist(),
                 q[:total].double().cpu().numpy())
        t.scale = 0.07
        t.check(True, o[:total], lse[:total])


@pytest.mark.parametrize("kv,rope", LATENTS)
def test_attend_a_thousand_requests(M, kv, rope):
    # several requests a thread where the work is divided
    rng = np.random.default_rng(28)
    t = Attend(M, kv, rope, 5, rng.integers(0, 200, 1000).tolist(), rng.integers(0, 3, 1000).tolist(), seed=28)
    o, lse = t.run(True)
    assert t.cache.check() == 0
    t.check(True, o, lse)


def test_attend_any_layer(M):
    t = Attend(M, 128, 32, 8, [300, 90], [2, 1], seed=29)
    empty = torch.full_like(t.dev[0], 0x7F)
    cache = M.QCache(128, 32, [empty, empty, t.dev[0], empty], [t.dev[1] * 3, t.dev[1], t.dev[1], t.dev[1]], t.dev[2], n_heads=8)
    o, lse = t.run(False)
    t.cache = cache
    o2, lse2 = torch.zeros_like(o), torch.zeros_like(lse)
    cache.attend(2, t.q.cuda(), *t.args, o2, lse2, causal=False, scale=t.scale)
    assert cache.check() == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)
    t.check(False, o2, lse2)


def test_attend_more_chunks_than_32_bit_divisions_hold(M):
    # 1024 requests of 524300 tokens, 4.2 million chunks; the pages repeat, so that 4096 tokens with multiplicities are the
    # reference. Row sums add 4097 weights a thread and the output's accumulators four products of 32 tokens a chunk:
    # at most 4 * 4097 roundings of 2^-23 in sequence.
    kv, rope, D, H, bs, n = 64, 16, 80, 64, 1024, 524_300
    rng = np.random.default_rng(30)
    codes = np.stack([Q.e4m3_encode(rng.normal(0, 32, (64, D))) for _ in range(64)])
    row = rng.integers(0, 64, -(-n // 64)).astype(np.int32)
    q = torch.from_numpy(rng.normal(0, 1, (bs, H, D))).to(torch.bfloat16)
    dev = [torch.from_numpy(codes).cuda(), torch.full((64,), 2.0 ** -5, device="cuda")]
    cache = M.QCache(kv, rope, [dev[0]], [dev[1]], ints(row)[None].expand(bs, -1).contiguous(), n_heads=H)
    o, lse = torch.zeros(bs, H, kv, dtype=torch.bfloat16, device="cuda"), torch.zeros(bs, H, device="cuda")
    scale = 1.3 / np.sqrt(D)
    cache.attend(0, q.cuda(), ints(np.arange(bs + 1)), ints([n] * bs), o, lse, causal=True, scale=scale)
    assert cache.check() == 0
    count = np.zeros((64, 64))
    for j, pg in enumerate(row):
        count[pg, :min(64, n - 64 * j)] += 1
    k, count = E4M3_TABLE[codes].reshape(-1, D) * 2.0 ** -5, count.reshape(-1)
    for b in (0, 1, 7, 150, 511, 512, 1000, 1022, 1023):
        s = scale * q[b].double().numpy() @ k.T
        top = scale * (np.abs(q[b].double().numpy()) @ np.abs(k).T).max(1)
        m = s.max(1, keepdims=True)
        w = np.exp(s - m) * count
        want, absolute = w @ k[:, :kv] / w.sum(1)[:, None], w @ np.abs(k[:, :kv]) / w.sum(1)[:, None]
        ds = 2.0 ** -16 * top + 2.0 ** -18 * np.abs(q[b].double().numpy()).max(1) * scale * np.abs(k).sum(1).max()
        sums = 4 * 4097 * 2.0 ** -23
        tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2 * ds[:, None] + 2 * sums) * absolute + 2.0 ** -17 * np.abs(k).max()
        assert np.all(np.abs(o[b].double().cpu().numpy() - want) <= tol)
        assert np.all(np.abs(lse[b].double().cpu().numpy() - (m[:, 0] + np.log(w.sum(1)))) <= ds + sums + 2.0 ** -20)


@pytest.mark.parametrize("kv,rope", LATENTS)
@pytest.mark.parametrize("bs,length,nq", [(1, 12000, 1), (5, 3000, 2), (200, 700, 1), (2, 5, 3), (20, 200, 30)])
def test_attend_pages_of_all_scales(M, kv, rope, bs, length, nq):
    # zero pages, pages whose tokens score far below and far above them, value scales 2^63 apart, in any order
    D, H, rng = kv + rope, 3, np.random.default_rng(31 + bs)
    kinds = [(-8, -1.75, 1.0), (-60, 0.0, 0.0), (-7, 0.0, 1.0), (3, 0.0, 1000.0), (-9, 0.75, 0.3), (-50, 0.0, 2.0 ** -45)]
    codes = np.stack([page(rng, kv, D, e, last, size) for e, last, size in kinds])
    rows = rng.integers(0, len(kinds), (bs, -(-length // 64)))
    q = np.zeros((bs * nq, H, D))
    q[:, :, -1] = rng.choice([0.0, 60.0, 800.0, -800.0, 5000.0], (bs * nq, H))
    t = Laid(M, kv, codes, [2.0 ** e for e, _, _ in kinds], rows, [length] * bs, [nq] * bs, q)
    o, lse = t.run(False)
    assert t.cache.check() == 0
    check_steered(t, o, lse)
    o2, lse2 = t.run(False)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kv,rope", LATENTS)
@pytest.mark.parametrize("H", [333, 1024])
def test_attend_many_heads(M, kv, rope, H):
    t = Attend(M, kv, rope, H, [130, 0, 77], [2, 1, 1], seed=32)
    o, lse = t.run(True)
    assert t.cache.check() == 0
    t.check(True, o, lse)

"""8-bit layers with a scale for each block of 128 against the oracle in 64 bits: quantisers bit for bit, products and the
gated product within bounds that follow from the number of roundings."""
import numpy as np
import pytest
import torch

import mla_block_diffusion_gb300 as M
from oracle import qlinear as O

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    return t.cpu().numpy()


def rows_of(rng, m, k):
    """Random quantised rows: codes without NaN, scales any positive fp32 numbers."""
    codes = rng.integers(0, 255, (m, k)).astype(np.uint8)
    codes[(codes & 127) == 127] = 3
    return codes, np.exp2(rng.uniform(-12, 2, (-(-k // 128), m))).astype(np.float32)


def weight_of(rng, n, k):
    codes = rng.integers(0, 255, (n, k)).astype(np.uint8)
    codes[(codes & 127) == 127] = 3
    return codes, np.exp2(rng.uniform(-14, -4, (-(-n // 128), -(-k // 128)))).astype(np.float32)


def product_bound(mag, k):
    """Of an fp32 product against the exact one, mag the sum of the terms' magnitudes. The products of two codes are exact;
    a block's 128 terms are summed in the tensor core, which adds 32 at a time aligned to the largest: four such
    additions, each off by at most 2^-21 of the magnitudes that it has seen; the two scales' product and the FMA of every
    block are off by 2^-24 each, sums of all blocks likewise."""
    blocks = -(-k // 128)
    return mag * (4 * 2.0 ** -21 + (2 + blocks + 8) * 2.0 ** -24) + 1e-30


ROWS = [1, 7, 16, 17, 33, 64, 65, 127, 129, 300]
SHAPES = [(16, 16), (128, 128), (144, 272), (576, 720), (272, 4112)]  # (n, k)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,k", [(1, 16), (1, 7168), (7, 128), (9, 144), (33, 1040), (200, 2112)])
def test_quantise_rows(m, k, dtype):
    rng = np.random.default_rng(m * 10007 + k)
    x = torch.from_numpy(rng.standard_normal((m, k)) * np.exp2(rng.integers(-30, 30, (m, k)))).to(dtype)
    x[rng.integers(0, m), :16] = 0
    codes = torch.full((m, k), 77, dtype=torch.uint8, device="cuda")
    scales = torch.full((-(-k // 128), m), 5.0, device="cuda")
    M.quantise_rows(x.cuda(), codes, scales)
    c, s = O.quantise_rows(x.double().numpy())
    assert np.array_equal(host(scales), s)
    assert np.array_equal(host(codes), c)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,k", [(16, 16), (128, 128), (144, 272), (400, 720)])
def test_quantise_weight(n, k, dtype):
    rng = np.random.default_rng(n * 10007 + k)
    w = torch.from_numpy(rng.standard_normal((n, k)) * np.exp2(rng.integers(-8, 8, (n, k)))).to(dtype)
    codes = torch.empty(n, k, dtype=torch.uint8, device="cuda")
    scales = torch.empty(-(-n // 128), -(-k // 128), device="cuda")
    M.quantise_weight(w.cuda(), codes, scales)
    c, s = O.quantise_weight(w.double().numpy())
    assert np.array_equal(host(scales), s)
    assert np.array_equal(host(codes), c)


def test_quantise_edges():
    """Every binade's ends, powers of two times 448, subnormals, zeros, the largest number; NaN and infinities."""
    for dtype in (torch.float32, torch.bfloat16):
        rows = []
        for e in (-149, -130, -126, -110, -109, -108, -92, -91, -20, -1, 0, 1, 8, 9, 60, 120, 127):
            for f in (1.0, 1.75, 1.7578125, 1.9921875):
                x = np.zeros(128)
                x[5], x[9], x[17] = f * 2.0 ** e, -f * 2.0 ** (e - 3), f * 2.0 ** (e - 16)
                rows.append(x)
        x = torch.from_numpy(np.stack(rows)).to(dtype)
        bad = torch.ones(4, 128).to(dtype)
        bad[0, 3], bad[1, 3], bad[2, 3] = float("nan"), float("inf"), float("-inf")
        bad[3] = float("nan")
        x = torch.cat([x, bad])
        codes = torch.empty(x.shape, dtype=torch.uint8, device="cuda")
        scales = torch.empty(1, x.shape[0], device="cuda")
        M.quantise_rows(x.cuda(), codes, scales)
        c, s = O.quantise_rows(x.double().numpy())
        got = host(codes)
        nan = (c & 127) == 127
        assert np.array_equal(host(scales), s)
        assert np.array_equal((got & 127) == 127, nan)
        assert np.array_equal(got[~nan], c[~nan])


def test_quantise_strides_and_untouched_neighbours():
    g = torch.Generator().manual_seed(3)
    big = torch.randn(20, 320, generator=g).cuda()
    x = big[3:13, 16:16 + 144]
    codes = torch.full((12, 144), 9, dtype=torch.uint8, device="cuda")
    scales = torch.full((2, 12), 9.0, device="cuda")
    M.quantise_rows(x, codes[1:11], scales[:, 1:11])
    c, s = O.quantise_rows(x.double().cpu().numpy())
    assert np.array_equal(host(codes[1:11]), c) and np.array_equal(host(scales[:, 1:11]), s)
    assert bool((codes[0] == 9).all() and (codes[11] == 9).all() and (scales[:, 0] == 9).all() and (scales[:, 11] == 9).all())


@pytest.mark.parametrize("m", ROWS)
@pytest.mark.parametrize("n,k", SHAPES)
@pytest.mark.parametrize("out", ["bf16", "fp32", "add"])
def test_matmul(m, n, k, out):
    rng = np.random.default_rng(m * 1009 + n * 13 + k)
    x, sx = rows_of(rng, m, k)
    w, sw = weight_of(rng, n, k)
    lin = M.QLinear(dev(w), dev(sw))
    y = torch.full((m + 1, n), 7.0, dtype=torch.bfloat16 if out == "bf16" else torch.float32, device="cuda")
    add = rng.standard_normal((m, n)).astype(np.float32) * 30 if out == "add" else None
    lin.matmul(dev(x), dev(sx), y[:m], add=None if add is None else dev(add))
    assert lin.check() == 0
    want, mag = O.matmul(O.rows_values(x, sx), O.weight_values(w, sw))
    bound = product_bound(mag, k)
    if add is not None:
        want = want + add
        bound = bound + np.abs(want) * 2.0 ** -24
    if out == "bf16":
        # 8 significant bits: numbers of [1, 2) are 2^-7 apart, so a rounding is off by up to 2^-8 of the value
        bound = bound + (np.abs(want) + bound) * 2.0 ** -8
    got = host(y[:m].double())
    assert bool((y[m] == 7).all())
    off = np.abs(got - want)
    assert (off <= bound).all(), (off / bound).max()


@pytest.mark.parametrize("m,n,k", [(300, 9744, 272), (65, 19472, 144), (1000, 9744, 16), (64, 20496, 4112), (320, 2112, 7168)])
@pytest.mark.parametrize("out", ["bf16", "add"])
def test_matmul_of_many_tiles(m, n, k, out):
    """Tiles of the full width, several a CTA."""
    test_matmul(m, n, k, out)


@pytest.mark.parametrize("m,n,k", [(300, 9744, 272), (1300, 4112, 144), (64, 20496, 4112), (3, 20496, 4112), (30, 12304, 2576)])
def test_gated_of_many_tiles(m, n, k):
    test_gated(m, n, k)


@pytest.mark.parametrize("m,n", [(16, 20496), (60, 2112), (320, 2112), (150, 576)])
def test_calls_in_a_row_give_the_same(m, n):
    """Results do not depend on timing: calls that overlap in their prologues, eager and replayed, bit for bit."""
    rng = np.random.default_rng(m)
    k = 2576
    x, sx = (dev(a) for a in rows_of(rng, m, k))
    ws = [M.QLinear(*(dev(a) for a in weight_of(rng, n, k))) for _ in range(4)]
    ys = torch.empty(4, m, n, device="cuda")
    hs = [(torch.empty(m, n, dtype=torch.uint8, device="cuda"), torch.empty(-(-n // 128), m, device="cuda")) for _ in range(4)]

    def calls():
        for i in range(4):
            ws[i].matmul(x, sx, ys[i])
            M.QGated(ws[i], ws[(i + 1) % 4]).forward(x, sx, *hs[i])

    def results():
        return [ys.clone()] + [t.clone() for h in hs for t in h]
    calls()
    first = results()
    for _ in range(10):
        calls()
    assert all(torch.equal(a, b) for a, b in zip(first, results()))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    ys.zero_()
    for _ in range(10):
        g.replay()
    assert all(torch.equal(a, b) for a, b in zip(first, results()))
    assert all(w.check() == 0 for w in ws)


@pytest.mark.parametrize("m", ROWS)
@pytest.mark.parametrize("n,k", SHAPES)
def test_gated(m, n, k):
    """The scale is the least that holds the block's largest value, or off by a factor of two where that is at a border; every
    value within half an E4M3 step of the exact one, plus what the sums and the exponential are off by."""
    rng = np.random.default_rng(m * 1009 + n * 13 + k + 1)
    x, sx = rows_of(rng, m, k)
    wg, sg = weight_of(rng, n, k)
    wu, su = weight_of(rng, n, k)
    xv = O.rows_values(x, sx)
    (g, gm), (u, um) = O.matmul(xv, O.weight_values(wg, sg)), O.matmul(xv, O.weight_values(wu, su))
    unit = 2.0 ** np.round(np.log2(np.abs(g).std() + 1e-30))  # gates of a few units
    sg, g, gm = (sg / unit).astype(np.float32), g / unit, gm / unit
    gate = M.QGated(M.QLinear(dev(wg), dev(sg)), M.QLinear(dev(wu), dev(su)))
    hc = torch.full((m + 1, n), 9, dtype=torch.uint8, device="cuda")
    hs = torch.full((-(-n // 128), m + 1), 9.0, device="cuda")
    gate.forward(dev(x), dev(sx), hc[:m], hs[:, :m])
    assert gate.check() == 0
    assert bool((hc[m] == 9).all() and (hs[:, m] == 9).all())
    want = O.gated(g, u)
    eg, eu = product_bound(gm, k), product_bound(um, k)
    # |d silu / dg| <= 1.1; exp, division and products: 2^-20 relative with room
    off = 1.1 * eg * (np.abs(u) + eu) + np.abs(O.gated(g, np.ones_like(g))) * eu + np.abs(want) * 2.0 ** -20
    scales = host(hs[:, :m]).astype(np.float64)
    assert (np.exp2(np.round(np.log2(scales))) == scales).all()
    for b in range(scales.shape[0]):
        at = np.s_[:, b * 128:(b + 1) * 128]
        low, high = (np.abs(want[at]) - off[at]).max(1), (np.abs(want[at]) + off[at]).max(1)
        assert (low <= 448 * scales[b]).all()
        assert ((scales[b] == 2.0 ** -100) | (high > 224 * scales[b])).all()
    s = np.repeat(scales.T, 128, 1)[:, :n]
    got = O.rows_values(host(hc[:m]), scales)
    # half a step: 2^-4 of the value, and 2^-10 scales below the normal numbers
    assert (np.abs(got - want) <= off + np.maximum((np.abs(want) + off) * 2.0 ** -4, s * 2.0 ** -10)).all()


# 11 blocks of k stay whole; 12 and more are shared by clusters, not evenly where they are no multiple, the last block short
SHARED = [(16, 1408), (144, 1424), (144, 1536), (272, 1552), (1040, 2064), (2112, 3600), (576, 14336)]


@pytest.mark.parametrize("m", [1, 2, 16, 31, 64])
@pytest.mark.parametrize("n,k", SHARED)
@pytest.mark.parametrize("out", ["bf16", "add"])
def test_matmul_of_shared_blocks(m, n, k, out):
    test_matmul(m, n, k, out)


@pytest.mark.parametrize("m", [1, 17, 64])
@pytest.mark.parametrize("n,k", SHARED)
def test_gated_of_shared_blocks(m, n, k):
    test_gated(m, n, k)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,k", [(430, 7168), (435, 7184), (3001, 1040), (6001, 528)])
def test_quantise_rows_of_long_calls(m, k, dtype):
    """Either number of blocks a half-warp, around the border between them; blocks that are no multiple of it."""
    test_quantise_rows(m, k, dtype)


@pytest.mark.parametrize("m", [5, 64, 300])
def test_two_streams_and_two_graphs_of_one_workspace(m):
    """Calls on two streams, and two graphs replayed at once, that share an error word and weights."""
    rng = np.random.default_rng(m)
    n, k = 1040, 2064
    x, sx = (dev(a) for a in rows_of(rng, m, k))
    a = M.QLinear(*(dev(v) for v in weight_of(rng, n, k)))
    b = M.QLinear(*(dev(v) for v in weight_of(rng, n, k)), workspace=a.ws)
    want = [torch.empty(m, n, device="cuda") for _ in range(2)]
    a.matmul(x, sx, want[0])
    b.matmul(x, sx, want[1])
    torch.cuda.synchronize()
    ys = [torch.zeros(m, n, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for lin, y, s in zip((a, b), ys, streams):
            with torch.cuda.stream(s):
                lin.matmul(x, sx, y)
    torch.cuda.synchronize()
    assert all(torch.equal(y, w) for y, w in zip(ys, want))
    graphs = []
    for lin, y in zip((a, b), ys):
        y.zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lin.matmul(x, sx, y)
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(y, w) for y, w in zip(ys, want))
    assert a.check() == 0

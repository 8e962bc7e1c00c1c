"""Products and gated products of quantised rows: strides, results in place, NaN and values that are not finite, scales of any
sign and zero, more than 2^32 elements."""
import numpy as np
import pytest
import torch

import mla_block_diffusion_gb300 as M
from oracle import qlinear as O
from tests.test_gpu_qlinear import dev, host, product_bound, rows_of, weight_of

pytestmark = pytest.mark.gpu
ROWS = [1, 7, 64, 65, 300]
SHAPES = [(16, 16), (272, 528), (2112, 1552)]


def blocks(n):
    return -(-n // 128)


def empty_rows(m, n):
    return torch.empty(m, n, dtype=torch.uint8, device="cuda"), torch.empty(blocks(n), m, device="cuda")


def is_nan(codes):
    return (codes & 127) == 127


@pytest.mark.parametrize("m", ROWS)
@pytest.mark.parametrize("n,k", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides(m, n, k, dtype):
    """Result, residual and scales with strides of their own: bit for bit what contiguous ones give, and what lies between the
    rows stays."""
    rng = np.random.default_rng(m * 1009 + n * 13 + k)
    x, sx = (dev(a) for a in rows_of(rng, m, k))
    lin = M.QLinear(*(dev(a) for a in weight_of(rng, n, k)))
    add = torch.randn(m, n, device="cuda") * 30
    scales = torch.full((blocks(k), m + 5), float("nan"), device="cuda")
    scales[:, 2:m + 2] = sx
    wide = torch.full((m, n + 48), float("nan"), device="cuda")
    wide[:, 32:n + 32] = add
    for a, b in ((None, None), (add, wide[:, 32:n + 32])):
        want = torch.empty(m, n, dtype=dtype, device="cuda")
        lin.matmul(x, sx, want, add=a)
        out = torch.full((m + 2, n + 16), 7.0, dtype=dtype, device="cuda")
        lin.matmul(x, scales[:, 2:m + 2], out[1:m + 1, 8:n + 8], add=b)
        assert torch.equal(out[1:m + 1, 8:n + 8], want)
        assert bool((out[0] == 7).all() and (out[-1] == 7).all() and (out[:, :8] == 7).all() and (out[:, n + 8:] == 7).all())
    assert lin.check() == 0


@pytest.mark.parametrize("m", ROWS)
@pytest.mark.parametrize("n,k", SHAPES)
def test_onto_the_residual(m, n, k):
    """The residual is the result itself, contiguous and as columns of a buffer: the bits of a separate one."""
    rng = np.random.default_rng(m * 1009 + n * 13 + k + 2)
    x, sx = (dev(a) for a in rows_of(rng, m, k))
    lin = M.QLinear(*(dev(a) for a in weight_of(rng, n, k)))
    add = torch.randn(m, n, device="cuda") * 30
    want = torch.empty(m, n, device="cuda")
    lin.matmul(x, sx, want, add=add)
    y = add.clone()
    lin.matmul(x, sx, y, add=y)
    assert torch.equal(y, want)
    buf = torch.full((m, n + 32), 7.0, device="cuda")
    y = buf[:, 16:n + 16]
    y.copy_(add)
    lin.matmul(x, sx, y, add=y)
    assert torch.equal(y, want) and bool((buf[:, :16] == 7).all() and (buf[:, n + 16:] == 7).all())
    assert lin.check() == 0


@pytest.mark.parametrize("m", ROWS)
@pytest.mark.parametrize("n,k", SHAPES)
def test_nan_codes_in_products(m, n, k):
    """A NaN in a row's codes makes that row NaN, one in a weight's that output, and nothing else moves."""
    rng = np.random.default_rng(m * 1009 + n * 13 + k + 3)
    x, sx = rows_of(rng, m, k)
    w, sw = weight_of(rng, n, k)
    row, out = m // 2, 3 * n // 4
    add = torch.randn(m, n, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        clean = torch.empty(m, n, dtype=dtype, device="cuda")
        M.QLinear(dev(w), dev(sw)).matmul(dev(x), dev(sx), clean, add=add)
        x2, w2 = x.copy(), w.copy()
        x2[row, k // 3], w2[out, k - 1] = 0x7f, 0xff
        for a, b, bad in ((x2, w, np.s_[row]), (x, w2, np.s_[:, out])):
            y = torch.empty(m, n, dtype=dtype, device="cuda")
            lin = M.QLinear(dev(b), dev(sw))
            lin.matmul(dev(a), dev(sx), y, add=add)
            assert bool(torch.isnan(y[bad]).all())
            y[bad] = clean[bad]
            assert torch.equal(y, clean)
            assert lin.check() == 0


@pytest.mark.parametrize("m", ROWS)
@pytest.mark.parametrize("n,k", SHAPES)
def test_nan_codes_in_gated_products(m, n, k):
    """A NaN makes NaN codes where it enters; the scales are those of the finite values, 2^-100 where there is none."""
    rng = np.random.default_rng(m * 1009 + n * 13 + k + 4)
    x, sx = rows_of(rng, m, k)
    (wg, sg), (wu, su) = weight_of(rng, n, k), weight_of(rng, n, k)
    row, out = m // 2, 3 * n // 4
    wu[out] = 0  # where the NaN comes the value is zero without it, and no scale depends on it
    clean, h = empty_rows(m, n), empty_rows(m, n)
    M.QGated(M.QLinear(dev(wg), dev(sg)), M.QLinear(dev(wu), dev(su))).forward(dev(x), dev(sx), *clean)
    assert not bool(is_nan(clean[0]).any())
    for name in ("gate", "up"):
        g2, u2 = wg.copy(), wu.copy()
        (g2 if name == "gate" else u2)[out, k // 2] = 0x7f
        gated = M.QGated(M.QLinear(dev(g2), dev(sg)), M.QLinear(dev(u2), dev(su)))
        gated.forward(dev(x), dev(sx), *h)
        assert bool(is_nan(h[0][:, out]).all()) and torch.equal(h[1], clean[1])
        h[0][:, out] = clean[0][:, out]
        assert torch.equal(h[0], clean[0])
    x2 = x.copy()
    x2[row, k - 1] = 0xff
    gated = M.QGated(M.QLinear(dev(wg), dev(sg)), M.QLinear(dev(wu), dev(su)))
    gated.forward(dev(x2), dev(sx), *h)
    assert bool(is_nan(h[0][row]).all()) and bool((h[1][:, row] == 2.0 ** -100).all())
    h[0][row], h[1][:, row] = clean[0][row], clean[1][:, row]
    assert torch.equal(h[0], clean[0]) and torch.equal(h[1], clean[1])
    assert gated.check() == 0


@pytest.mark.parametrize("m", [7, 65])
def test_gated_values_that_are_not_finite(m):
    """Sums beyond fp32 in the second of three blocks of outputs: NaN codes there, the scale of the finite ones."""
    n, k = 384, 128
    x, sx = np.full((m, k), 0x7e, np.uint8), np.ones((1, m), np.float32)     # 448
    wg, wu = np.full((n, k), 0x38, np.uint8), np.full((n, k), 0x38, np.uint8)  # 1
    wu[128:256] = 0
    wu[128:200:2], wu[129:200:2] = 0x7e, 0xfe                                # 448, -448: sums of +-2^24.6
    wu[200:256] = 0x38
    wu[255] = 0
    sg, su = np.full((3, 1), 2.0 ** -14, np.float32), np.ones((3, 1), np.float32)  # gates of 3.5
    su[1] = 2.0 ** 104                                                       # +-2^128.6: beyond; 2^15.8 2^104: held
    h = empty_rows(m, n)
    gated = M.QGated(M.QLinear(dev(wg), dev(sg)), M.QLinear(dev(wu), dev(su)))
    gated.forward(dev(x), dev(sx), *h)
    assert gated.check() == 0
    c = h[0].cpu().numpy()
    assert ((c[:, 128:200] & 127) == 127).all()
    rest = np.r_[0:128, 200:384]
    g = 448.0 * 128 * 2.0 ** -14
    u = np.where((rest >= 200) & (rest < 255), 448.0 * 128 * 2.0 ** 104, np.where(rest == 255, 0.0, 448.0 * 128))
    want = np.tile(O.gated(np.full(u.shape, g), u), (m, 1))
    scales = host(h[1]).astype(np.float64)
    assert (scales == np.array([[O.scale_of(O.gated(np.array([g]), np.array([v])))] for v in (448.0 * 128, 448.0 * 128 * 2.0 ** 104,
                                                                                            448.0 * 128)])).all()
    got = O.rows_values(c, scales)[:, rest]
    # half a step of E4M3 and what the gate is off by
    assert (np.abs(got - want) <= np.abs(want) * (2.0 ** -4 + 2.0 ** -14)).all()


@pytest.mark.parametrize("m", ROWS)
@pytest.mark.parametrize("n,k", SHAPES)
def test_scales_of_any_sign_and_zero(m, n, k):
    rng = np.random.default_rng(m * 1009 + n * 13 + k + 5)
    x, sx = rows_of(rng, m, k)
    w, sw = weight_of(rng, n, k)
    for s in (sx, sw):
        s *= rng.choice([1, -1], s.shape)
        s[rng.random(s.shape) < 0.2] = 0
    y = torch.empty(m, n, device="cuda")
    lin = M.QLinear(dev(w), dev(sw))
    lin.matmul(dev(x), dev(sx), y)
    assert lin.check() == 0
    xv, wv = O.rows_values(x, sx), O.weight_values(w, sw)
    want, mag = O.matmul(xv, wv)
    assert (np.abs(host(y).astype(np.float64) - want) <= product_bound(mag, k)).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_more_than_2_to_32_elements(dtype):
    """Rows, results and scales behind 2^32 elements and 2^34 bytes: the last rows have the bits of a call over them alone."""
    m, n, k, tail = 300000, 16384, 144, 700
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(m, n, dtype=dtype, device="cuda")
    x[:tail].normal_(generator=g)
    x[-tail:].normal_(generator=g)
    x[tail:-tail] = 1
    q, part = empty_rows(m, n), empty_rows(tail, n)
    M.quantise_rows(x, *q)
    for at in (slice(0, tail), slice(m - tail, m)):
        M.quantise_rows(x[at], *part)
        assert torch.equal(q[0][at], part[0]) and torch.equal(q[1][:, at], part[1])
    weights = []
    for _ in range(2):
        w = torch.randn(n, k, device="cuda", generator=g) / 12
        codes, scales = torch.empty(n, k, dtype=torch.uint8, device="cuda"), torch.empty(blocks(n), blocks(k), device="cuda")
        M.quantise_weight(w, codes, scales)
        weights.append(M.QLinear(codes, scales))
    s = empty_rows(m, k)
    M.quantise_rows(torch.randn(m, k, device="cuda", generator=g), *s)
    y = x  # its rows are quantised
    weights[0].matmul(*s, y)
    gated = M.QGated(*weights)
    gated.forward(*s, *q)
    yt = torch.empty(tail, n, dtype=dtype, device="cuda")
    for at in (slice(0, tail), slice(m - tail, m)):
        rows = s[0][at].contiguous(), s[1][:, at]
        weights[0].matmul(*rows, yt)
        assert torch.equal(y[at], yt)
        gated.forward(*rows, *part)
        assert torch.equal(q[0][at], part[0]) and torch.equal(q[1][:, at], part[1])
    assert gated.check() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,k", [(9, 528), (2100, 1552)])
def test_quantise_rows_of_columns(m, k, dtype):
    """Source rows and scales with strides, both forms of the bf16 quantiser."""
    g = torch.Generator(device="cuda").manual_seed(m)
    wide = torch.randn(m, k + 64, device="cuda", generator=g).to(dtype)
    x = wide[:, 32:k + 32]
    want, codes = empty_rows(m, k), torch.empty(m, k, dtype=torch.uint8, device="cuda")
    M.quantise_rows(x.contiguous(), *want)
    scales = torch.full((blocks(k), m + 3), 7.0, device="cuda")
    M.quantise_rows(x, codes, scales[:, 1:m + 1])
    assert torch.equal(codes, want[0]) and torch.equal(scales[:, 1:m + 1], want[1])
    assert bool((scales[:, 0] == 7).all() and (scales[:, m + 1:] == 7).all())
    c, s = O.quantise_rows(x[-40:].double().cpu().numpy())
    assert np.array_equal(host(codes[-40:]), c) and np.array_equal(host(scales[:, 1:m + 1])[:, -40:], s)

"""8-bit rows on the GPU: quantise, load, the gated activation forward and backward, against the 64-bit
definitions. Bytes and scales are equal bit for bit; values are within their type's rounding.

Tolerances. An output of type t is rounded once: eps(t) / 2 relative, half the smallest subnormal absolute.
Before that comes 32-bit arithmetic: e^-g is documented within 2 + 1.173 |g| ulp, a fast quotient within 2, each
product half: silu and its slope within (1.173 |g| + 8) 2^-23 relative (to the sum of the magnitudes where terms
are added). Where e^-g overflows (g < -88) the result is below 1e-36 |u|.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from lossless_entropy_coding_fixed_b200 import hx  # noqa: E402

from . import _rows as ref  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FMT = {"e4m3": hx.ROWS_E4M3, "int8": hx.ROWS_INT8}
SUB = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}


@pytest.fixture(scope="module")
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def half_step(dt):
    return torch.finfo(DT[dt]).eps / 2


def make(rows, cols, dt, seed, cuda):
    """Rows of many levels; the first ones of zeros, tiny and huge values where there are enough."""
    rng = np.random.default_rng(seed)
    x = rng.laplace(0, 0.3, (rows, cols)) * np.exp(rng.normal(0, 1, (rows, 1)))
    x[rng.random((rows, cols)) < 0.05] *= 20
    if rows > 8:
        x[0] = 0
        x[1] *= 1e-30
        x[2] *= 1e-5
        x[3] = np.where(rng.random(cols) < 0.5, -0.0, 0.0)
        x[4, 0] = 3e4
        if dt != "f16":
            x[5] *= 1e30
    return torch.from_numpy(x).to(DT[dt]).to(cuda)


def placed(x, pad, shift):
    """x inside a wider buffer, `pad` columns more and `shift` elements from an aligned start."""
    rows, cols = x.shape
    buf = torch.full((rows * (cols + pad) + shift + 8,), 7.0, dtype=x.dtype, device=x.device)
    v = buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    v.copy_(x)
    return v, buf


def check_rows(x, b, s, fmt):
    rb, rs = ref.quantize(x.double().cpu().numpy(), fmt)
    assert (s.double().cpu().numpy() == rs).all()
    assert (b.cpu().numpy().reshape(rb.shape) == rb).all()


SHAPES = [(1, 1), (3, 2), (9, 7), (9, 8), (33, 31), (12, 255), (10, 1000), (9, 1024), (9, 1025), (9, 1032), (9, 4104),
          (9, 8192), (9, 16384), (9, 16392), (9, 4097), (2, 40001), (2, 40000), (9, 1002), (9, 4100), (2, 20002), (2, 20004)]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_quantize_and_load(cuda, shape, dt, fmt):
    x = make(*shape, dt, sum(shape), cuda)
    b, s = hx.quantize_rows(x, FMT[fmt])
    check_rows(x, b, s, fmt)
    for out in DT:
        y = hx.dequantize_rows(b, s, FMT[fmt], dtype=DT[out]).double().cpu().numpy()
        v = ref.values(b.cpu().numpy(), s.cpu().numpy(), fmt)
        if out == "f16":
            v = np.clip(v, -65504, 65504)
        # the product rounds to 32 bits (INT8), then to the type
        tol = np.abs(v) * (half_step(out) + (2.0 ** -24 if fmt == "int8" else 0)) + SUB[out] / 2
        assert (np.abs(y - v) <= tol).all()
        if fmt == "e4m3" and out != "f16":
            assert (y == v).all()


@pytest.mark.parametrize("pad,shift", [(0, 1), (1, 0), (8, 0), (8, 4), (3, 3), (24, 8)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_strides_and_alignment(cuda, dt, pad, shift):
    x = make(21, 520, dt, 5, cuda)
    v, _ = placed(x, pad, shift)
    b = torch.full((21 * 520 + 64,), 99, dtype=torch.uint8, device=cuda)
    for off in (0, 1, 8):
        out = b[off:off + 21 * 520].view(21, 520)
        _, s = hx.quantize_rows(v, hx.ROWS_INT8, out=out)
        check_rows(x, out, s, "int8")
        assert (b[off + 21 * 520:] == 99).all() and (b[:off] == 99).all()
        y, buf = placed(torch.zeros_like(x), pad, shift)
        hx.dequantize_rows(out, s, hx.ROWS_INT8, out=y)
        assert torch.equal(y, hx.dequantize_rows(out.clone(), s, hx.ROWS_INT8, dtype=x.dtype))
        rest = buf.clone()
        rest[shift:shift + 21 * (520 + pad)].view(21, 520 + pad)[:, :520] = 7
        assert (rest == 7).all()  # nothing beside the matrix was written
        b.fill_(99)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_rows_that_are_not_finite(cuda, dt, fmt):
    for cols in (16, 13, 5000):
        x = make(6, cols, dt, 2, cuda)
        x[1, 3] = float("nan")
        x[2, cols - 1] = float("inf")
        x[4, 0] = -float("inf")
        b, s = hx.quantize_rows(x, FMT[fmt])
        good = [0, 3, 5]
        check_rows(x[good], b[good], s[good], fmt)
        for r in (1, 2, 4):
            assert torch.isnan(s[r]) and (b[r] == 0).all()
        y = hx.dequantize_rows(b, s, FMT[fmt], dtype=DT[dt])
        assert torch.isnan(y[[1, 2, 4]]).all() and torch.isfinite(y[good]).all()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_extreme_rows_stay_finite(cuda, dt, fmt):
    big, small = torch.finfo(DT[dt]).max, torch.finfo(DT[dt]).smallest_normal
    x = torch.tensor([[big, -big, big / 2, 1], [small, 0, -small, 0], [small / 4, 0, 0, -small / 4],
                      [448, 447, 449, -448], [127, 0.5, 1.5, -126.5], [2.5, 254, -2.5, 3]], dtype=DT[dt], device=cuda)
    b, s = hx.quantize_rows(x, FMT[fmt])
    check_rows(x, b, s, fmt)
    assert torch.isfinite(hx.dequantize_rows(b, s, FMT[fmt], dtype=DT[dt])).all()
    assert torch.isfinite(hx.dequantize_rows(b, s, FMT[fmt], dtype=torch.float32)).all()


def test_int8_ties_and_neighbours(cuda):
    """Quotients at and next to a half: decided as the 32-bit division decides them."""
    rng = np.random.default_rng(8)
    rows = []
    for top in (127.0, 63.5, 1.0, 0.3, 5e-20, 7e20):
        s = np.float32(top) / np.float32(127)
        k = rng.integers(-126, 126, 500)
        h = ((k + 0.5) * np.float64(s)).astype(np.float32)
        near = np.concatenate([h, np.nextafter(h, np.float32(0)), np.nextafter(h, np.float32(np.inf)),
                               np.nextafter(h, np.float32(-np.inf)), [np.float32(top)]])
        rows.append(near)
    x = torch.from_numpy(np.stack(rows)).to(cuda)
    b, sc = hx.quantize_rows(x, hx.ROWS_INT8)
    check_rows(x, b, sc, "int8")


@pytest.mark.parametrize("dt, e", [("f16", 0), ("f16", -13)] + [("bf16", e) for e in (-124, -110, 0, 69, 70, 71, 72, 73, 127)])
def test_int8_every_pair_of_a_16_bit_type(cuda, dt, e):
    """Every significand of a value under every significand of the row's largest, at the nine exponents that reach half
    a step: the bytes are the 32-bit division's. Scales from 2^-126 on, around 2^64, and up to 2^121."""
    n = 128 if dt == "bf16" else 1024
    m = torch.arange(n, 2 * n, dtype=torch.float64) / n
    x = torch.cat([torch.ldexp(m, torch.tensor(-k)) for k in range(9)])[None].repeat(n, 1)
    x[:, 1::2] *= -1
    x[x.abs() > m[:, None]] = 0
    x = (torch.cat([m[:, None], x], 1) * 2.0 ** e).to(DT[dt])
    b, s = hx.quantize_rows(x.to(cuda), hx.ROWS_INT8)
    check_rows(x, b, s, "int8")


def gated_check(h, g, u, dt):
    want = ref.gated(g, u)
    tol = np.abs(want) * (half_step(dt) + 2.0 ** -23 * (1.173 * np.abs(g) + 8)) + SUB[dt] + 1e-36 * np.abs(u)
    got = h.double().cpu().numpy()
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1), (9, 8), (5, 33), (9, 256), (3, 1031), (2, 8192), (2, 16392), (2, 20001),
                                   (5, 1002), (5, 4100), (2, 20002), (2, 20004)])
def test_gated_forward_and_backward(cuda, shape, dt, fmt):
    rows, cols = shape
    rng = np.random.default_rng(cols)
    x = torch.from_numpy(rng.laplace(0, 1.5, (rows, 2 * cols))).to(DT[dt]).to(cuda)
    x[0, 0] = -100  # e^-g overflows
    h, b, s = hx.gated_forward(x, FMT[fmt])
    xs = x.double().cpu().numpy().reshape(rows, 2, cols)
    gated_check(h, xs[:, 0], xs[:, 1], dt)
    check_rows(x.view(rows, 2, cols), b, s, fmt)
    h2, none, none2 = hx.gated_forward(x, FMT[fmt], save=False)
    assert none is None and none2 is None and torch.equal(h, h2)

    dh = torch.from_numpy(rng.normal(0, 0.1, (rows, cols))).to(DT[dt]).to(cuda)
    dx, again = hx.gated_backward(dh, b, s, FMT[fmt], need_h=True)
    dx2, no_h = hx.gated_backward(dh, b, s, FMT[fmt])
    assert no_h is None and torch.equal(dx, dx2)
    v = ref.values(b.cpu().numpy(), s.cpu().numpy(), fmt)
    g, u, d = v[:, 0], v[:, 1], dh.double().cpu().numpy()
    gated_check(again, g, u, dt)
    dg, du = ref.gated_grad(g, u, d)
    got = dx.double().cpu().numpy().reshape(rows, 2, cols)
    slack = 2.0 ** -23 * (1.173 * np.abs(g) + 8)
    p = ref.sigmoid(g)
    terms = np.abs(d * u) * (p + np.abs(g) * p * (1 - p))
    assert (np.abs(got[:, 0] - dg) <= np.abs(dg) * half_step(dt) + terms * (slack + 2.0 ** -22) + SUB[dt] + 1e-36).all()
    assert (np.abs(got[:, 1] - du) <= np.abs(du) * (half_step(dt) + slack) + SUB[dt] + 1e-36).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(70001, 3), (40001, 17), (9001, 34), (9000, 100), (5000, 248), (3001, 1001), (2000, 2050)])
def test_many_rows(cuda, shape, dt):
    """Enough rows for several units per thread and several rows per warp, in every width of unit."""
    rows, cols = shape
    g = torch.Generator(device=cuda).manual_seed(cols)
    x = (torch.randn(rows, 2 * cols, generator=g, device=cuda) * 2).to(DT[dt])
    x[::97] = 0
    h, b, s = hx.gated_forward(x, hx.ROWS_E4M3)
    xs = x.double().cpu().numpy().reshape(rows, 2, cols)
    gated_check(h, xs[:, 0], xs[:, 1], dt)
    check_rows(x.view(rows, 2, cols), b, s, "e4m3")
    assert torch.equal(hx.gated_forward(x, save=False)[0], h)
    v = ref.values(b.cpu().numpy(), s.cpu().numpy(), "e4m3")
    back = hx.dequantize_rows(b.view(2 * rows, cols), s.view(-1), dtype=torch.float32)
    assert (back.cpu().numpy().reshape(v.shape) == v).all()
    q, qs = hx.quantize_rows(x, hx.ROWS_INT8)
    check_rows(x, q, qs, "int8")
    dh = torch.randn(rows, cols, generator=g, device=cuda).to(DT[dt])
    dx, again = hx.gated_backward(dh, b, s, need_h=True)
    gated_check(again, v[:, 0], v[:, 1], dt)
    dg, du = ref.gated_grad(v[:, 0], v[:, 1], dh.double().cpu().numpy())
    got = dx.double().cpu().numpy().reshape(rows, 2, cols)
    # values of a normal law, |g| < 16: slope and activation within 27 ulp of terms that are at most 1.1 |dh u| and |dh g|
    d, u = np.abs(dh.double().cpu().numpy()), np.abs(v[:, 1])
    assert (np.abs(got[:, 0] - dg) <= np.abs(dg) * half_step(dt) + 1.1 * d * u * 2.0 ** -18 + 1e-37).all()
    assert (np.abs(got[:, 1] - du) <= np.abs(du) * (half_step(dt) + 2.0 ** -18) + 1e-37).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_gates_whose_exponential_is_huge(cuda, dt):
    """e^-g between 2^126 and 2^128 and beyond, with an up value that makes the result an ordinary number. e^-|g| is then
    below 2^-126: its last place is 2^-149, 2^-20 of it down to g = -89."""
    g = np.array([-86, -87, -87.5, -88, -88.5, -89.0, 86, 87.5, 88])
    u = np.array([1e30, -1e30, 2.0 ** 120])
    gg, uu = (v.reshape(-1) for v in np.meshgrid(g, u))
    x = torch.from_numpy(np.stack([np.concatenate([gg, uu])] * 3)).to(DT[dt]).to(cuda)
    xs = x.double().cpu().numpy().reshape(3, 2, -1)
    near = half_step(dt) + 2.0 ** -23 * (1.173 * 89 + 8) + 2.0 ** -20
    for save in (True, False):
        h = hx.gated_forward(x, save=save)[0].double().cpu().numpy()
        want = ref.gated(xs[:, 0], xs[:, 1])
        assert (np.abs(h - want) <= near * np.abs(want)).all()
    for fmt, name in ((hx.ROWS_E4M3, "e4m3"), (hx.ROWS_INT8, "int8")):
        _, b, s = hx.gated_forward(x, fmt)
        dx, h = hx.gated_backward(torch.full((3, gg.size), 0.5, dtype=DT[dt], device=cuda), b, s, fmt, need_h=True)
        v = ref.values(b.cpu().numpy(), s.cpu().numpy(), name)
        want = ref.gated(v[:, 0], v[:, 1])
        assert (np.abs(h.double().cpu().numpy() - want) <= near * np.abs(want)).all()
        dg, du = ref.gated_grad(v[:, 0], v[:, 1], 0.5)
        dx = dx.double().cpu().numpy().reshape(3, 2, -1)
        assert (np.abs(dx[:, 0] - dg) <= near * np.abs(dg)).all()
        assert (np.abs(dx[:, 1] - du) <= near * np.abs(du) + SUB[dt]).all()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_large_gates_are_linear(cuda, dt):
    """1 + e^-g rounds to 1 from g = 18 on (e^-18 < 2^-25), so the result is g u, rounded once: at a half to even."""
    g = (18 + 2 * torch.arange(40, device=cuda)).to(DT[dt])
    u = torch.cat([torch.arange(129, 256, 2, device=cuda) / 128, -torch.arange(129, 256, 6, device=cuda) / 64]).to(DT[dt])
    x = torch.stack([g.repeat_interleave(u.numel()), u.repeat(g.numel())]).view(1, -1)
    want = (x[0, :x.shape[1] // 2].float() * x[0, x.shape[1] // 2:].float()).to(DT[dt])
    for save in (True, False):
        assert torch.equal(hx.gated_forward(x, save=save)[0][0], want)


def test_gated_in_32_bits(cuda):
    """f32: e = e^-|g| is within 2 units of the last place (4 2^-24), of which 1 + e takes over the part e / (1 + e), so that
    e / (1 + e) is at most 4 off for it; the sum rounds (1), the reciprocal is within 2 units (4), the product of the two,
    the one with g and the one with u round (3): 12 2^-24; 1 / (1 + e) within 7. Held to 14."""
    g = torch.Generator(device=cuda).manual_seed(5)
    gate = 160 * torch.rand(64, 4096, generator=g, device=cuda) - 80
    up = torch.randn(64, 4096, generator=g, device=cuda)
    for save in (True, False):
        h = hx.gated_forward(torch.cat((gate, up), 1), save=save)[0].double().cpu().numpy()
        want = ref.gated(gate.double().cpu().numpy(), up.double().cpu().numpy())
        assert (np.abs(h - want) <= 14 * 2.0 ** -24 * np.abs(want)).all()
    b, s = hx.quantize_rows(torch.stack((gate, up), 1).view(128, 4096), hx.ROWS_INT8)
    dh = torch.randn(64, 4096, generator=g, device=cuda)
    b, s = b.view(64, 2, 4096), s.view(64, 2)
    # the values that the kernel reads: byte times scale, rounded to 32 bits
    v = hx.dequantize_rows(b.view(128, 4096), s.view(128), hx.ROWS_INT8, dtype=torch.float32).double().cpu().numpy()
    v = v.reshape(64, 2, 4096)
    d = dh.double().cpu().numpy()
    dx, h = hx.gated_backward(dh, b, s, hx.ROWS_INT8, need_h=True)
    want = ref.gated(v[:, 0], v[:, 1])
    assert (np.abs(h.double().cpu().numpy() - want) <= 14 * 2.0 ** -24 * np.abs(want)).all()
    dg, du = ref.gated_grad(v[:, 0], v[:, 1], d)
    dx = dx.double().cpu().numpy().reshape(64, 2, 4096)
    p = ref.sigmoid(v[:, 0])
    terms = np.abs(d * v[:, 1]) * (p + np.abs(v[:, 0]) * p * ref.sigmoid(-v[:, 0]))
    assert (np.abs(dx[:, 1] - du) <= 14 * 2.0 ** -24 * np.abs(du)).all()
    # silu is within 11, 1 - p within 10, their product is added in the same operation (1), then dh u (2): 24, held to 28
    assert (np.abs(dx[:, 0] - dg) <= 28 * 2.0 ** -24 * terms).all()


def test_gated_output_given(cuda):
    """An output of the caller's on a start that is not aligned; nothing beside it is written."""
    x = make(11, 2 * 264, "bf16", 6, cuda)
    want = hx.gated_forward(x)[0]
    buf = torch.full((11 * 264 + 16,), 5.0, dtype=torch.bfloat16, device=cuda)
    for off in (0, 1, 2, 8):
        out = buf[off:off + 11 * 264].view(11, 264)
        for save in (True, False):
            got = hx.gated_forward(x, save=save, out=out)[0]
            assert same_bits([got], [want]) and got.data_ptr() == out.data_ptr()
            assert (buf[:off] == 5).all() and (buf[off + 11 * 264:] == 5).all()
            buf.fill_(5)


def test_gated_strided_input(cuda):
    """x and dh as slices of wider buffers, on starts that are not aligned."""
    x = make(17, 2 * 264, "bf16", 3, cuda)
    want = hx.gated_forward(x, hx.ROWS_E4M3)
    dh = make(17, 264, "bf16", 4, cuda)
    grads = hx.gated_backward(dh, want[1], want[2], hx.ROWS_E4M3, need_h=True)
    for pad, shift in ((8, 0), (3, 1)):
        v, _ = placed(x, pad, shift)
        for a, b in zip(hx.gated_forward(v, hx.ROWS_E4M3), want):
            assert torch.equal(a, b)
        d, _ = placed(dh, pad, shift)
        for a, b in zip(hx.gated_backward(d, want[1], want[2], hx.ROWS_E4M3, need_h=True), grads):
            assert torch.equal(a, b)


def test_gated_not_finite(cuda):
    x = make(4, 64, "bf16", 3, cuda)
    x[1, 5] = float("nan")   # a gate
    x[2, 40] = float("inf")  # an up
    h, b, s = hx.gated_forward(x, hx.ROWS_E4M3)
    assert torch.isnan(h[1, 5]) and torch.isinf(h[2, 8]) and torch.isfinite(h[[0, 3]]).all()
    assert torch.isnan(s[1, 0]) and torch.isfinite(s[1, 1]) and torch.isnan(s[2, 1])
    dx, _ = hx.gated_backward(torch.ones(4, 32, dtype=torch.bfloat16, device=cuda), b, s, hx.ROWS_E4M3)
    assert torch.isnan(dx[1]).all() and torch.isfinite(dx[[0, 3]]).all()


def test_no_rows(cuda):
    x = torch.empty(0, 16, dtype=torch.bfloat16, device=cuda)
    b, s = hx.quantize_rows(x)
    assert b.shape == (0, 16) and s.shape == (0,)
    assert hx.dequantize_rows(b, s).shape == (0, 16)
    h, b, s = hx.gated_forward(x)
    assert h.shape == (0, 8) and hx.gated_backward(h, b, s)[0].shape == (0, 16)


def test_more_values_than_31_bits(cuda):
    """Offsets beyond 2^31 and 2^32 values: a few rows of a large matrix."""
    rows, cols = (1 << 17) + 3, 1 << 15
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=cuda)
    at = [0, 1, 65535, 65536, 65537, 131071, 131072, rows - 1]
    x[at] = make(len(at), cols, "bf16", 9, cuda)
    b, s = hx.quantize_rows(x, hx.ROWS_E4M3)
    check_rows(x[at], b[at], s[at], "e4m3")
    assert int((s != 1).sum()) <= len(at) and int(b[65538:131000].max()) == 0
    y = hx.dequantize_rows(b, s, hx.ROWS_E4M3, out=x)
    assert (y[at].double().cpu().numpy() == ref.values(b[at].cpu().numpy(), s[at].cpu().numpy(), "e4m3")).all()
    del y
    dx, h = hx.gated_backward(x[:rows // 2], b[:rows // 2 * 2].view(rows // 2, 2, cols),
                              s[:rows // 2 * 2].view(rows // 2, 2), hx.ROWS_E4M3, need_h=True)
    last = rows // 2 - 1
    one, h1 = hx.gated_backward(x[last:last + 1].clone(), b[2 * last:2 * last + 2].clone().view(1, 2, cols),
                                s[2 * last:2 * last + 2].clone().view(1, 2), hx.ROWS_E4M3, need_h=True)
    assert torch.equal(dx[last], one[0]) and torch.equal(h[last], h1[0])


def same_bits(a, b):
    """Equal bit for bit, NaN included."""
    return all(torch.equal(u.contiguous().view(torch.uint8), v.contiguous().view(torch.uint8)) for u, v in zip(a, b))


def test_captured_and_replayed(cuda):
    """Save, forward and backward inside a CUDA graph: replays with new contents, and eager calls beside it."""
    x = make(40, 2 * 768, "bf16", 1, cuda)
    x2 = make(40, 2 * 768, "bf16", 2, cuda)
    dh = make(40, 768, "bf16", 3, cuda)

    def step():
        h, b, s = hx.gated_forward(x, hx.ROWS_INT8)
        dx, again = hx.gated_backward(dh, b, s, hx.ROWS_INT8, need_h=True)
        q, qs = hx.quantize_rows(h, hx.ROWS_E4M3)
        return h, b, s, dx, again, hx.dequantize_rows(q, qs, hx.ROWS_E4M3)

    first = [t.clone() for t in step()]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = step()
    g.replay()
    assert same_bits(held, first)
    x.copy_(x2)
    second = [t.clone() for t in step()]
    g.replay()
    assert same_bits(held, second)


def test_on_another_stream_and_device(cuda):
    x = make(64, 1024, "bf16", 1, cuda)
    want = hx.quantize_rows(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = hx.quantize_rows(x)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    if torch.cuda.device_count() > 1:  # the tensors' device is not the current one
        x1 = x.to("cuda:1")
        got = hx.quantize_rows(x1)
        assert got[0].device == x1.device and torch.equal(got[0].cpu(), want[0].cpu())


def test_binding_refusals(cuda):
    x = torch.zeros(4, 8, dtype=torch.bfloat16, device=cuda)
    b, s = hx.quantize_rows(x)
    for call, err in ((lambda: hx.quantize_rows(x.t()), ValueError), (lambda: hx.quantize_rows(x.long()), TypeError),
                      (lambda: hx.quantize_rows(x[0]), ValueError),
                      (lambda: hx.quantize_rows(x[:1].expand(4, 8)), ValueError),
                      (lambda: hx.quantize_rows(x, out=b[:3]), ValueError),
                      (lambda: hx.quantize_rows(x, 2), hx.HxError),
                      (lambda: hx.dequantize_rows(b, s[:3]), ValueError),
                      (lambda: hx.dequantize_rows(b.t(), s), ValueError),
                      (lambda: hx.dequantize_rows(b, s.cpu()), TypeError),
                      (lambda: hx.gated_forward(x[:, :7]), ValueError),
                      (lambda: hx.gated_backward(x, b, s), ValueError)):
        with pytest.raises(err):
            call()

"""Per-head norm with rotation, forward and backward, against the 64-bit definition; saved rows bit for bit.

Tolerances. Outputs are rounded once (eps / 2 relative). Before: 32-bit arithmetic, a sum of at most 512 terms in
chains of 16 and a butterfly (21 additions deep), a root and a quotient: below 2^-19 of the sum of the terms'
magnitudes. A weight gradient adds at most `chain` terms one after another, (chain + 32) 2^-24 of their magnitudes.
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
EPS = 1e-5


@pytest.fixture(scope="module")
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def setup(T, nq, nk, D, R, dt, cuda, seed=0, wdt=torch.float32, places=None, pdt=torch.int64):
    rng = np.random.default_rng(seed)
    H = nq + nk
    x = rng.laplace(0, 0.5, (T, H, D)) * np.exp(rng.normal(0, 1, (T, H, 1)))
    if T > 2:
        x[1, 0] = 0  # eps alone
        x[2] *= 1e-4
    dy = rng.normal(0, 0.05, (T, H, D))
    places = places or 2 * T + 5
    ang = np.arange(places)[:, None] * 10000.0 ** (-np.arange(0, R, 2) / max(R, 1))
    to = lambda a, d: torch.from_numpy(np.ascontiguousarray(a)).to(d).to(cuda)  # noqa: E731
    return dict(x=to(x, DT[dt]), dy=to(dy, DT[dt]), wq=to(rng.normal(1, 0.3, D), wdt), wk=to(rng.normal(1, 0.3, D), wdt),
                cos=to(np.cos(ang), torch.float32), sin=to(np.sin(ang), torch.float32),
                pos=to(rng.integers(0, places, T), pdt))


def half(dt):
    return torch.finfo(DT[dt]).eps / 2


def args(p, nq):
    return (nq, p["wq"], p["wk"], p["cos"], p["sin"], p["pos"])


def f64(t):
    return t.double().cpu().numpy()


def angles(p):
    pos = p["pos"].cpu().numpy()
    return f64(p["cos"])[pos], f64(p["sin"])[pos]


def check_forward(y, p, nq, dt, inter):
    x, (c, s) = f64(p["x"]), angles(p)
    want = ref.head_norm_rope(x, nq, f64(p["wq"]), f64(p["wk"]), c, s, EPS, inter)
    mags = ref.turned(np.abs(x / np.sqrt(np.mean(x * x, -1, keepdims=True) + EPS)
                             * ref.head_weights(x.shape[1], nq, f64(p["wq"]), f64(p["wk"]))),
                      np.abs(c), np.abs(s), inter)
    # |a c| + |b s| for both of a pair
    a, b = ref.pair_places(2 * c.shape[1], inter)
    n = np.abs(x / np.sqrt(np.mean(x * x, -1, keepdims=True) + EPS)
               * ref.head_weights(x.shape[1], nq, f64(p["wq"]), f64(p["wk"])))
    mags = n.copy()
    mags[..., a] = mags[..., b] = n[..., a] + n[..., b]
    half = torch.finfo(DT[dt]).eps / 2
    assert (np.abs(f64(y) - want) <= np.abs(want) * half + mags * 2.0 ** -19 + SUB[dt]).all()


def check_backward(dx, dwq, dwk, b, s8, p, nq, dt, inter, fmt):
    x, dy, (c, s) = ref.values(b.cpu().numpy(), f64(s8), fmt), f64(p["dy"]), angles(p)
    wq, wk = f64(p["wq"]), f64(p["wk"])
    want, wdq, wdk = ref.head_norm_rope_grad(dy, x, nq, wq, wk, c, s, EPS, inter)
    r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + EPS)
    i, j = ref.pair_places(2 * c.shape[1], inter)
    g = np.abs(dy).copy()
    g[..., i] = g[..., j] = np.abs(dy[..., i]) + np.abs(dy[..., j])
    d = g * np.abs(ref.head_weights(x.shape[1], nq, wq, wk))
    xn = np.abs(x * r)
    mags = r * (d + xn * np.mean(d * xn, -1, keepdims=True))
    half = torch.finfo(DT[dt]).eps / 2
    assert (np.abs(f64(dx) - want) <= np.abs(want) * half + mags * 2.0 ** -19 + SUB[dt]).all()
    T = x.shape[0]
    for got, w, lo, hi in ((dwq, wdq, 0, nq), (dwk, wdk, nq, x.shape[1])):
        if hi == lo:
            continue
        terms = (g * xn)[:, lo:hi].sum((0, 1))
        chain = min(T * (hi - lo), 512 + T * (hi - lo) // 100)
        assert (np.abs(f64(got) - w) <= terms * ((chain + 32) * 2.0 ** -24) + 1e-37).all()


CASES = [  # tokens, q, k, dim, rot
    (1, 1, 0, 2, 2), (1, 4, 2, 64, 64), (3, 0, 2, 16, 8), (7, 3, 1, 128, 128), (5, 9, 3, 128, 64), (33, 2, 2, 80, 80),
    (6, 4, 1, 96, 32), (4, 2, 1, 18, 6), (3, 5, 2, 100, 100), (3, 2, 2, 256, 64), (2, 2, 1, 512, 512), (2, 1, 1, 510, 2),
    (9, 2, 1, 36, 0), (300, 17, 2, 32, 32), (2000, 8, 4, 64, 48)]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", CASES)
def test_forward_and_backward(cuda, case, dt, inter):
    T, nq, nk, D, R = case
    fmt = "e4m3" if (T + D) % 2 else "int8"
    p = setup(T, nq, nk, D, R, dt, cuda, seed=D + T)
    y, b, s = hx.head_norm_rope_forward(p["x"], *args(p, nq), eps=EPS, interleaved=inter, fmt=FMT[fmt])
    check_forward(y, p, nq, dt, inter)
    rb, rs = ref.quantize(f64(p["x"]), fmt)
    assert (b.cpu().numpy() == rb).all() and (f64(s) == rs).all()
    y2, n1, n2 = hx.head_norm_rope_forward(p["x"], *args(p, nq), eps=EPS, interleaved=inter, save=False)
    assert n1 is None and n2 is None and torch.equal(y, y2)
    got = hx.head_norm_rope_backward(p["dy"], b, s, *args(p, nq), eps=EPS, interleaved=inter, fmt=FMT[fmt])
    check_backward(*got, b, s, p, nq, dt, inter, fmt)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("level", [-30, -60, -64, -66, -68])
def test_backward_of_tiny_heads_without_eps(cuda, level, dt, fmt):
    """Rows whose scale squared is below 32 bits' numbers, but not their mean square. That is at least 2^-137 here; its
    last place is 2^-149, so that it is within 2^-13 where it is below 2^-126, and its inverse root within 2^-14: three of
    those in dx, one in a weight gradient."""
    p = setup(6, 2, 1, 64, 32, dt, cuda, seed=9)
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.choice([-1, 1], (18, 64)) * rng.uniform(0.8, 1.2, (18, 64)) * 2.0 ** level).to(DT[dt]).to(cuda)
    b, s = hx.quantize_rows(x, FMT[fmt])
    b, s = b.view(6, 3, 64), s.view(6, 3)
    dx, dwq, dwk = hx.head_norm_rope_backward(p["dy"], b, s, *args(p, 2), eps=0.0, fmt=FMT[fmt])
    v, dy, (c, sn) = ref.values(b.cpu().numpy(), f64(s), fmt), f64(p["dy"]), angles(p)
    wq, wk = f64(p["wq"]), f64(p["wk"])
    want, wdq, wdk = ref.head_norm_rope_grad(dy, v, 2, wq, wk, c, sn, 0.0, False)
    r = 1 / np.sqrt(np.mean(v * v, -1, keepdims=True))
    i, j = ref.pair_places(32, False)
    g = np.abs(dy).copy()
    g[..., i] = g[..., j] = np.abs(dy[..., i]) + np.abs(dy[..., j])
    d = g * np.abs(ref.head_weights(3, 2, wq, wk))
    xn = np.abs(v * r)
    lost = 2.0 ** -14 if level < -62 else 0
    assert (np.abs(f64(dx) - want) <= np.abs(want) * half(dt) + r * (d + xn * np.mean(d * xn, -1, keepdims=True)) *
            (2.0 ** -19 + 3 * lost)).all()
    for got, w, lo, hi in ((dwq, wdq, 0, 2), (dwk, wdk, 2, 3)):
        assert (np.abs(f64(got) - w) <= (g * xn)[:, lo:hi].sum((0, 1)) * (2.0 ** -18 + lost)).all()


@pytest.mark.parametrize("wdt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pdt", [torch.int32, torch.int64])
def test_weight_and_position_types(cuda, wdt, pdt):
    p = setup(11, 4, 2, 64, 64, "bf16", cuda, wdt=wdt, pdt=pdt)
    y, b, s = hx.head_norm_rope_forward(p["x"], *args(p, 4), eps=EPS)
    check_forward(y, p, 4, "bf16", False)
    got = hx.head_norm_rope_backward(p["dy"], b, s, *args(p, 4), eps=EPS)
    check_backward(*got, b, s, p, 4, "bf16", False, "e4m3")


@pytest.mark.parametrize("D,shift", [(128, 0), (128, 4), (128, 1), (48, 0)])
def test_packed_in_place_and_other_layouts(cuda, D, shift):
    """Read out of and written into a packed projection; heads before tokens; starts that are not aligned. Another
    alignment is read in other vectors, whose sums have another order: values are held to the definition, not to
    the aligned call's last bit."""
    T, nq, nk = 13, 4, 2
    p = setup(T, nq, nk, D, D, "bf16", cuda, seed=shift)
    want = hx.head_norm_rope_forward(p["x"], *args(p, nq), eps=EPS)
    back = hx.head_norm_rope_backward(p["dy"], want[1], want[2], *args(p, nq), eps=EPS)
    check_forward(want[0], p, nq, "bf16", False)
    H = nq + 2 * nk
    buf = torch.full((T * H * D + 8,), 5.0, dtype=torch.bfloat16, device=cuda)
    packed = buf[shift:shift + T * H * D].view(T, H, D)
    packed[:, :nq + nk] = p["x"]
    got = hx.head_norm_rope_forward(packed[:, :nq + nk], *args(p, nq), eps=EPS, out=packed[:, :nq + nk])
    check_forward(packed[:, :nq + nk], p, nq, "bf16", False)
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    assert (packed[:, nq + nk:] == 5).all() and (buf[:shift] == 5).all() and (buf[shift + T * H * D:] == 5).all()
    packed[:, :nq + nk] = p["dy"]
    dx, dwq, dwk = hx.head_norm_rope_backward(packed[:, :nq + nk], want[1], want[2], *args(p, nq), eps=EPS,
                                              out=packed[:, :nq + nk])
    assert (packed[:, nq + nk:] == 5).all()
    for a, w, k in ((packed[:, :nq + nk], dwq, dwk), back):
        check_backward(a, w, k, want[1], want[2], p, nq, "bf16", False, "e4m3")
    heads_first = p["x"].transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(hx.head_norm_rope_forward(heads_first, *args(p, nq), eps=EPS)[0], want[0])


def test_positions_outside_the_tables(cuda):
    p = setup(6, 4, 2, 64, 32, "bf16", cuda)
    st = hx.new_status(cuda)
    want = hx.head_norm_rope_forward(p["x"], *args(p, 4), eps=EPS, status=st)
    assert int(st.item()) == 0
    p["pos"][2], p["pos"][4] = -1, p["cos"].shape[0]
    y, b, s = hx.head_norm_rope_forward(p["x"], *args(p, 4), eps=EPS, status=st)
    assert int(st.item()) == hx.HX_ERR_ARG
    good = [0, 1, 3, 5]
    assert torch.equal(y[good], want[0][good]) and torch.isnan(y[[2, 4]]).all()
    assert torch.equal(b, want[1]) and torch.equal(s, want[2])
    st.zero_()
    dx, dwq, dwk = hx.head_norm_rope_backward(p["dy"], b, s, *args(p, 4), eps=EPS, status=st)
    assert int(st.item()) == hx.HX_ERR_ARG
    assert torch.isfinite(dx[good]).all() and torch.isnan(dx[[2, 4]]).all() and torch.isnan(dwq).all()
    hx.head_norm_rope_forward(p["x"], *args(p, 4), eps=EPS)  # not reported, and not fatal


def test_heads_that_are_not_finite(cuda):
    p = setup(4, 4, 2, 64, 64, "bf16", cuda)
    clean = hx.head_norm_rope_forward(p["x"], *args(p, 4), eps=EPS)
    p["x"][1, 2, 7] = float("nan")
    p["x"][3, 5, 0] = float("inf")
    y, b, s = hx.head_norm_rope_forward(p["x"], *args(p, 4), eps=EPS)
    hit = torch.zeros(4, 6, dtype=torch.bool, device=cuda)
    hit[1, 2] = hit[3, 5] = True
    assert torch.equal(y[~hit], clean[0][~hit]) and torch.isnan(y[1, 2]).all()
    assert torch.isnan(s[hit]).all() and (b[hit] == 0).all() and torch.equal(b[~hit], clean[1][~hit])
    dx, dwq, dwk = hx.head_norm_rope_backward(p["dy"], b, s, *args(p, 4), eps=EPS)
    assert torch.isnan(dx[hit]).all() and torch.isfinite(dx[~hit]).all()


@pytest.mark.parametrize("fmt", [hx.ROWS_E4M3, hx.ROWS_INT8])
@pytest.mark.parametrize("D,inter", [(128, False), (128, True), (48, False), (6, True), (2, False)])
def test_saved_heads_of_every_level(cuda, D, inter, fmt):
    """The bytes and scales of a head are the row's, up to bf16's largest values, also when the outputs go where the
    heads were."""
    p = setup(40, 4, 2, D, D, "bf16", cuda, seed=D)
    level = torch.tensor([2.0 ** e for e in (-120, -60, 0, 61, 69, 70, 71, 72, 100, 126)], device=cuda)
    p["x"] = (p["x"].float().clamp(-1, 1) * level.repeat(4)[:, None, None]).bfloat16()
    p["x"][:, :, 0] = p["x"][:, :, 0].sign() * (level.repeat(4)[:, None] * 1.5).bfloat16()
    p["x"][9, 3, 0] = torch.finfo(torch.bfloat16).max
    want = hx.quantize_rows(p["x"].reshape(-1, D), fmt)
    y, b, s = hx.head_norm_rope_forward(p["x"], *args(p, 4), eps=EPS, interleaved=inter, fmt=fmt)
    assert torch.equal(b.reshape(-1, D), want[0]) and torch.equal(s.reshape(-1), want[1].reshape(-1))
    x = p["x"].clone()
    y2, b, s = hx.head_norm_rope_forward(x, *args(p, 4), eps=EPS, interleaved=inter, fmt=fmt, out=x)
    assert torch.equal(b.reshape(-1, D), want[0]) and torch.equal(s.reshape(-1), want[1].reshape(-1))
    small = level.repeat(4) < 2.0 ** 60
    assert torch.equal(y2[small], y[small]) and torch.isfinite(y[small]).all()


def test_more_values_than_32_bits(cuda):
    """Offsets beyond 2^32 values, in place: a few tokens of a large batch against a small one of the same."""
    T, H, D = (1 << 17) + 3, 128, 256
    p = setup(6, 96, 32, D, D, "bf16", cuda, places=64)
    at = torch.tensor([0, 1, 65536, 131071, 131072, T - 1], device=cuda)
    want = hx.head_norm_rope_forward(p["x"], *args(p, 96), eps=EPS)
    back = hx.head_norm_rope_backward(p["dy"], want[1], want[2], *args(p, 96), eps=EPS)
    x = torch.zeros(T, H, D, dtype=torch.bfloat16, device=cuda)
    x[at] = p["x"]
    pos = torch.zeros(T, dtype=torch.int64, device=cuda)
    pos[at] = p["pos"]
    big = dict(p, pos=pos)
    y, b, s = hx.head_norm_rope_forward(x, *args(big, 96), eps=EPS, out=x)
    assert torch.equal(y[at], want[0]) and torch.equal(b[at], want[1]) and torch.equal(s[at], want[2])
    assert int(torch.count_nonzero(s != 1)) <= want[2].numel()
    x.zero_()
    x[at] = p["dy"]
    dx, dwq, dwk = hx.head_norm_rope_backward(x, b, s, *args(big, 96), eps=EPS, out=x)
    assert torch.equal(dx[at], back[0])
    for got, w in ((dwq, back[1]), (dwk, back[2])):  # the same terms in another order, and zeros
        assert float((got - w).abs().max()) <= float(w.abs().max()) * 2.0 ** -14


def test_gradients_that_are_broadcast(cuda):
    """dy with strides of zero: one gradient for every head, or for every token."""
    p = setup(9, 4, 2, 64, 64, "bf16", cuda)
    _, b, s = hx.head_norm_rope_forward(p["x"], *args(p, 4), eps=EPS)
    for dy in (p["dy"][:, :1].expand(9, 6, 64), p["dy"][:1].expand(9, 6, 64)):
        got = hx.head_norm_rope_backward(dy, b, s, *args(p, 4), eps=EPS)
        want = hx.head_norm_rope_backward(dy.contiguous(), b, s, *args(p, 4), eps=EPS)
        assert all(torch.equal(a, c) for a, c in zip(got, want))


def test_no_tokens(cuda):
    p = setup(0, 4, 2, 64, 64, "bf16", cuda, places=4)
    y, b, s = hx.head_norm_rope_forward(p["x"], *args(p, 4))
    assert y.shape == (0, 6, 64) and b.shape == (0, 6, 64) and s.shape == (0, 6)
    dx, dwq, dwk = hx.head_norm_rope_backward(p["dy"], b, s, *args(p, 4))
    assert (dwq == 0).all() and (dwk == 0).all()


def test_repeated_captured_and_two_at_once(cuda):
    """The same bits every time: eager, replayed, and beside another call on another stream."""
    p = setup(700, 8, 2, 128, 128, "bf16", cuda)

    def step():
        y, b, s = hx.head_norm_rope_forward(p["x"], *args(p, 8), eps=EPS)
        return (y, b, s, *hx.head_norm_rope_backward(p["dy"], b, s, *args(p, 8), eps=EPS))

    first = [t.clone() for t in step()]
    g, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = step()
    with torch.cuda.graph(g2):
        held2 = step()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s1):
            g.replay()
        with torch.cuda.stream(s2):
            g2.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, first))
    assert all(torch.equal(a, b) for a, b in zip(held2, first))
    assert all(torch.equal(a, b) for a, b in zip(step(), first))


def test_binding_refusals(cuda):
    p = setup(4, 4, 2, 64, 64, "bf16", cuda)
    f = hx.head_norm_rope_forward
    _, b, s = f(p["x"], *args(p, 4))
    for call, err in ((lambda: f(p["x"], 7, *args(p, 4)[1:]), ValueError),
                      (lambda: f(p["x"], 4, None, *args(p, 4)[2:]), ValueError),
                      (lambda: f(p["x"], 4, p["wq"][:32], *args(p, 4)[2:]), ValueError),
                      (lambda: f(p["x"], 4, p["wq"].half(), p["wk"].half(), *args(p, 4)[3:]), hx.HxError),
                      (lambda: f(p["x"], 4, p["wq"], p["wk"], p["cos"].double(), p["sin"], p["pos"]), TypeError),
                      (lambda: f(p["x"], 4, p["wq"], p["wk"], p["cos"], p["sin"][:3], p["pos"]), ValueError),
                      (lambda: f(p["x"], 4, p["wq"], p["wk"], p["cos"], p["sin"], p["pos"].float()), TypeError),
                      (lambda: f(p["x"], 4, p["wq"], p["wk"], p["cos"], p["sin"], p["pos"][:3]), ValueError),
                      (lambda: f(p["x"], 4, p["wq"], p["wk"], p["cos"], p["sin"], p["pos"].cpu()), TypeError),
                      (lambda: f(p["x"].transpose(1, 2), *args(p, 4)), ValueError),
                      (lambda: f(p["x"], *args(p, 4), out=p["x"][:1].expand(4, 6, 64)), ValueError),
                      (lambda: hx.head_norm_rope_backward(p["dy"], b[:, :5], s, *args(p, 4)), ValueError),
                      (lambda: hx.head_norm_rope_backward(p["dy"], b, s.double(), *args(p, 4)), TypeError)):
        with pytest.raises(err):
            call()

"""Weight gradient from 8-bit rows, against the 64-bit product.

Tolerances. The result is rounded once to its type (eps / 2 relative). The products of dY with e4m3 rows in bf16 are
exact in 32 bits, and each of `tokens` additions loses at most one unit of the last place of 32 bits (2^-23 of the
sum so far, at most 2^-23 of the sum of the terms' magnitudes); the splits' join adds at most 32 more. INT8 rows are
held as two values of dY's type: the rest of the rest is within (eps / 2)^2 of each. In f16 a value can fall below the normal
range: half the smallest subnormal, 2^-25, absolute.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from lossless_entropy_coding_fixed_b200 import hx  # noqa: E402

from . import _rows as ref  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FMT = {"e4m3": hx.ROWS_E4M3, "int8": hx.ROWS_INT8}


@pytest.fixture(scope="module")
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def setup(T, n, k, dt, fmt, cuda, seed=0):
    g = torch.Generator(device=cuda).manual_seed(seed)
    x = torch.randn(T, k, generator=g, device=cuda) * torch.exp(torch.randn(T, 1, generator=g, device=cuda))
    if T > 4:
        x[2] = 0
    dy = (0.05 * torch.randn(T, n, generator=g, device=cuda)).to(DT[dt])
    b, s = hx.quantize_rows(x, FMT[fmt])
    return dy, b, s


def check(dw, dy, b, s, dt, fmt, old=None):
    """All on the GPU in 64 bits: the bytes' values come from a table made on the host."""
    T = dy.shape[0]
    table = (ref.values(np.arange(256, dtype=np.uint8)[None], np.ones(1), fmt))[0]
    table[~np.isfinite(table)] = 0
    x = torch.from_numpy(table).to(dy.device)[b.long()] * s.double()[:, None]
    d = dy.double()
    want, mags = d.T @ x, d.abs().T @ x.abs()
    if old is not None:
        want, mags = want + old.double(), mags + old.double().abs()
    tol = want.abs() * torch.finfo(dw.dtype).eps / 2 + mags * ((T + 64) * 2.0 ** -23)
    if fmt == "int8":
        tol = tol + mags * (torch.finfo(DT[dt]).eps / 2) ** 2
    if dt == "f16":
        tol = tol + (d.abs().sum(0) * 2.0 ** -25)[:, None]
    if dw.dtype is torch.float16:
        tol = tol + 2.0 ** -25
    assert torch.isfinite(dw).all()
    assert ((dw.double() - want).abs() <= tol).all()


SIZES = [(1, 1, 1), (1, 128, 128), (2, 8, 3), (63, 64, 64), (64, 128, 128), (65, 130, 136), (64, 256, 256), (200, 257, 300),
         (1000, 515, 261), (513, 1024, 512), (5000, 8, 16), (5000, 17, 9), (4096, 64, 64), (20000, 128, 128),
         (70, 3328, 3200), (129, 3331, 3201), (300, 200, 40000)]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("size", SIZES)
def test_against_the_product(cuda, size, dt, fmt):
    T, n, k = size
    dy, b, s = setup(T, n, k, dt, fmt, cuda, seed=T)
    for out in (dt, "f32"):
        dw = hx.weight_grad(dy, b, s, FMT[fmt], dtype=DT[out])
        assert dw.dtype is DT[out] and dw.shape == (n, k)
        check(dw, dy, b, s, dt, fmt)
        old = torch.randn(n, k, device=cuda).to(DT[out])
        dw = hx.weight_grad(dy, b, s, FMT[fmt], out=old.clone(), accumulate=True)
        check(dw, dy, b, s, dt, fmt, old)


@pytest.mark.parametrize("fmt,size", [  # tile and splits of the tokens by the estimate: 128 x 128 ..
    ("e4m3", (300, 22, 4)), ("int8", (640, 641, 922)), ("int8", (640, 517, 770)), ("e4m3", (640, 1036, 261)),  # 1 2 3 4
    ("e4m3", (640, 8, 7)), ("e4m3", (1000, 933, 132)), ("e4m3", (3000, 3, 6)),  # 5 6 8
    ("e4m3", (2000, 772, 1316)), ("e4m3", (3000, 771, 784)), ("int8", (2000, 650, 897))])  # 256 x 256: 2 3 4
def test_every_number_of_splits(cuda, fmt, size):
    dy, b, s = setup(*size, "bf16", fmt, cuda, seed=size[1])
    n, k = size[1:]
    for out in ("bf16", "f32"):
        check(hx.weight_grad(dy, b, s, FMT[fmt], dtype=DT[out]), dy, b, s, "bf16", fmt)
    old = torch.randn(n, k, device=cuda)
    check(hx.weight_grad(dy, b, s, FMT[fmt], out=old.clone(), accumulate=True), dy, b, s, "bf16", fmt, old)


def test_scales_that_are_no_powers_of_two(cuda):
    """e4m3 rows of a caller's own scales: rounded once in the product, not the scale."""
    dy, b, s = setup(200, 136, 264, "bf16", "e4m3", cuda, seed=8)
    s = s * 1.2345
    table = (ref.values(np.arange(256, dtype=np.uint8)[None], np.ones(1), "e4m3"))[0]
    table[~np.isfinite(table)] = 0
    x = (torch.from_numpy(table).to(cuda)[b.long()].float() * s[:, None]).bfloat16().double()
    want, mags = dy.double().T @ x, dy.double().abs().T @ x.abs()
    dw = hx.weight_grad(dy, b, s, dtype=torch.float32).double()
    assert ((dw - want).abs() <= mags * ((200 + 64) * 2.0 ** -23)).all()


@pytest.mark.parametrize("T", [40, 3000])
@pytest.mark.parametrize("pad,shift", [(0, 1), (8, 0), (8, 8), (1, 0), (16, 4)])
def test_strides_and_alignment(cuda, T, pad, shift):
    """dY and dW as parts of wider buffers, bytes on any address; nothing beside dW is written."""
    n, k = 264, 192
    dy, b, s = setup(T, n, k, "bf16", "e4m3", cuda, seed=3)
    want = {o: hx.weight_grad(dy, b, s, dtype=DT[o]) for o in ("bf16", "f32")}

    def inside(rows, cols, dtype, fill):
        buf = torch.full((rows * (cols + pad) + shift + 16,), fill, dtype=dtype, device=cuda)
        return buf, buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]

    _, v = inside(T, n, torch.bfloat16, float("nan"))  # what lies beside is not read as a value
    v.copy_(dy)
    raw = torch.full((T * k + 64,), 0x7f, dtype=torch.uint8, device=cuda)  # NaN's byte
    at = raw[shift:shift + T * k].view(T, k)
    at.copy_(b)
    for o in want:
        buf, out = inside(n, k, DT[o], 3.0)
        hx.weight_grad(v, at, s, out=out)
        assert torch.equal(out, want[o])
        out.fill_(3.0)
        assert (buf == 3).all()


def test_no_tokens(cuda):
    dy, b, s = setup(0, 40, 24, "bf16", "e4m3", cuda)
    assert (hx.weight_grad(dy, b, s) == 0).all()
    old = torch.randn(40, 24, device=cuda).bfloat16()
    assert torch.equal(hx.weight_grad(dy, b, s, out=old.clone(), accumulate=True), old)


@pytest.mark.parametrize("n,k", [(1664, 1664), (4096, 4096)])  # pairs of CTAs: 256 x 256, 512 x 256
def test_no_tokens_of_a_large_product(cuda, n, k):
    dy = torch.empty(0, n, dtype=torch.bfloat16, device=cuda)
    b, s = torch.empty(0, k, dtype=torch.uint8, device=cuda), torch.empty(0, device=cuda)
    for fmt in FMT.values():
        for dt in ("bf16", "f32"):
            out = torch.full((n, k), 3.0, dtype=DT[dt], device=cuda)
            st = hx.new_status(cuda)
            for _ in range(20):
                hx.weight_grad(dy, b, s, fmt, out=out, status=st)
            assert (out == 0).all() and int(st.item()) == 0
            out.fill_(3)
            assert (hx.weight_grad(dy, b, s, fmt, out=out, accumulate=True) == 3).all()


def test_rows_and_columns_of_the_product(cuda):
    """Each byte's place: one token at a time, one output feature, counted values."""
    T, n, k = 130, 300, 520
    x = torch.zeros(T, k, device=cuda)
    dy = torch.zeros(T, n, device=cuda, dtype=torch.bfloat16)
    for t in range(T):
        x[t] = torch.arange(k, device=cuda) % 13 - 6 + t % 3
        dy[t, (7 * t) % n] = 1 + t % 4
    b, s = hx.quantize_rows(x, hx.ROWS_E4M3)
    v = hx.dequantize_rows(b, s, dtype=torch.float32)
    assert torch.equal(hx.weight_grad(dy, b, s, dtype=torch.float32), (dy.double().T @ v.double()).float())


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_a_row_that_was_not_finite(cuda, fmt):
    dy, b, s = setup(200, 136, 72, "bf16", fmt, cuda)
    s[77] = float("nan")
    assert torch.isnan(hx.weight_grad(dy, b, s, FMT[fmt])).all()


def test_f16_rows_beyond_its_range(cuda):
    x = torch.tensor([[65504.0, -65504.0, 1e6, 3.0]], device=cuda)
    for fmt in (hx.ROWS_E4M3, hx.ROWS_INT8):
        b, s = hx.quantize_rows(x, fmt)
        dy = torch.full((1, 8), 0.5, dtype=torch.float16, device=cuda)
        dw = hx.weight_grad(dy, b, s, fmt, dtype=torch.float32)
        want = hx.dequantize_rows(b, s, fmt, dtype=torch.float32).clamp(-65504, 65504) * 0.5
        assert torch.isfinite(dw).all() and torch.allclose(dw, want.expand(8, 4), rtol=2.0 ** -20, atol=0)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_rows_of_every_level(cuda, dt, fmt):
    """Scales from far below f16's range to its top, some rows of each in every step of 64 tokens."""
    T, n, k = 150, 70, 96
    g = torch.Generator(device=cuda).manual_seed(2)
    x = torch.randn(T, k, generator=g, device=cuda) * torch.exp2(torch.arange(T, device=cuda) % 37 - 24.0)[:, None]
    dy = torch.randn(T, n, generator=g, device=cuda).to(DT[dt])
    b, s = hx.quantize_rows(x, FMT[fmt])
    check(hx.weight_grad(dy, b, s, FMT[fmt], dtype=torch.float32), dy, b, s, dt, fmt)
    for lo, hi in ((0, 13), (24, 37)):  # of one kind only: the smallest, the largest
        rows = ((torch.arange(T, device=cuda) % 37 >= lo) & (torch.arange(T, device=cuda) % 37 < hi)).nonzero()[:, 0]
        part = [t[rows].contiguous() for t in (dy, b, s)]
        check(hx.weight_grad(*part, FMT[fmt], dtype=torch.float32), *part, dt, fmt)


@pytest.mark.parametrize("size", [(3000, 256, 256), (600, 515, 70), (100, 3328, 3200)])
def test_repeated_captured_and_two_at_once(cuda, size):
    """The same bits every time: eager, replayed, and two graphs at once with workspaces of their own."""
    dy, b, s = setup(*size, "bf16", "int8", cuda)
    want = hx.weight_grad(dy, b, s, hx.ROWS_INT8)
    graphs, held = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g in graphs:
        with torch.cuda.graph(g):
            held.append(hx.weight_grad(dy, b, s, hx.ROWS_INT8))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(h, want) for h in held) and torch.equal(hx.weight_grad(dy, b, s, hx.ROWS_INT8), want)


def test_launches_back_to_back(cuda):
    """Pairs of CTAs of several shapes one right after another, each where another one's has just ended: the same bits."""
    cases = []
    for T, n, k in ((65, 1664, 1664), (200, 1664, 1664), (3000, 771, 784), (64, 4096, 4096), (700, 2048, 2048)):
        dy, b, s = setup(T, n, k, "bf16", "e4m3", cuda, seed=T)
        cases.append((dy, b, s, hx.weight_grad(dy, b, s), torch.zeros(n, k, dtype=torch.bfloat16, device=cuda)))
    st = hx.new_status(cuda)
    for _ in range(30):
        for dy, b, s, _, out in cases:
            hx.weight_grad(dy, b, s, out=out, status=st)
    assert int(st.item()) == 0 and all(torch.equal(out, want) for *_, want, out in cases)


@pytest.mark.parametrize("size", [(1, 40, 72), (3, 130, 264), (70, 515, 261), (40, 1664, 1664)])
@pytest.mark.parametrize("level", [300.0, 1.0, 2.0 ** -4, 1e-3, 1e-4, 1e-5, 1e-7])
def test_int8_rows_in_f16_at_every_level(cuda, size, level):
    """X is held as two f16 values, the second 2^11 times as large: each value within 2^-23 of itself and 2^-36, after
    one rounding of scale times byte to 32 bits (2^-24). Joining the two sums rounds once more. Sums as above, but relative to
    terms of at least 2^-14 |dY|: the tensor core aligns a term by its factors' exponents, and that of a subnormal f16 is
    2^-14's. (Two tokens, X = 2^-24 in both, dY = 1 and 2^-6 (1 + 2^-10): the terms' sum has its last bit at 2^-40 = 2^-26 of
    2^-14, and the result lacks it; with 2^-5 in place of 2^-6 the last bit is at 2^-39, and the result has it. Relative to
    the larger term itself, 2^-24, 16 bits would have been kept.)"""
    T, n, k = size
    g = torch.Generator(device=cuda).manual_seed(T)
    dy = torch.randn(T, n, generator=g, device=cuda).half()
    b, s = hx.quantize_rows(level * (2 * torch.rand(T, k, generator=g, device=cuda) - 1), hx.ROWS_INT8)
    x, d = b.view(torch.int8).double() * s.double()[:, None], dy.double()
    want, mags = d.T @ x, d.abs().T @ x.abs().clamp(min=2.0 ** -14)
    tol = mags * ((T + 4) * 2.0 ** -23) + (d.abs().sum(0) * 2.0 ** -36)[:, None]
    dw = hx.weight_grad(dy, b, s, hx.ROWS_INT8, dtype=torch.float32)
    assert ((dw.double() - want).abs() <= tol).all()
    old = torch.randn(n, k, generator=g, device=cuda) * level
    dw = hx.weight_grad(dy, b, s, hx.ROWS_INT8, out=old.clone(), accumulate=True)
    assert ((dw.double() - want - old.double()).abs() <= tol + (want + old.double()).abs() * 2.0 ** -24).all()


def test_on_a_new_host_thread(cuda):
    """A thread's first CUDA call: nothing has made the device's context current there."""
    import threading

    dy, b, s = setup(256, 256, 256, "bf16", "e4m3", cuda)
    want, out, raised = hx.weight_grad(dy, b, s), torch.zeros(256, 256, dtype=torch.bfloat16, device=cuda), []

    def call():
        try:
            hx.weight_grad(dy, b, s, out=out)
        except Exception as e:
            raised.append(e)

    t = threading.Thread(target=call)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not raised and torch.equal(out, want)


def test_status_stays_clear(cuda):
    dy, b, s = setup(300, 200, 100, "bf16", "e4m3", cuda)
    st = hx.new_status(cuda)
    hx.weight_grad(dy, b, s, status=st)
    assert int(st.item()) == 0


def test_more_bytes_than_32_bits(cuda):
    """Tokens and columns whose product passes 2^32."""
    T, n, k = 1 << 16, 8, (1 << 16) + 64
    b = torch.zeros(T, k, dtype=torch.uint8, device=cuda)
    s = torch.ones(T, device=cuda)
    dy = torch.zeros(T, n, dtype=torch.bfloat16, device=cuda)
    b[T - 1, k - 5:] = 0x38  # 1.0
    b[T - 2] = 0x40  # 2.0
    dy[T - 1, 3], dy[T - 2, 5] = 3, 0.25
    dw = hx.weight_grad(dy, b, s)
    want = torch.zeros(n, k, dtype=torch.bfloat16, device=cuda)
    want[3, k - 5:] = 3
    want[5] = 0.5
    assert torch.equal(dw, want)


def test_binding_refusals(cuda):
    dy, b, s = setup(8, 16, 24, "bf16", "e4m3", cuda)
    for call, err in ((lambda: hx.weight_grad(dy.float(), b, s), hx.HxError),
                      (lambda: hx.weight_grad(dy, b[:7], s), ValueError),
                      (lambda: hx.weight_grad(dy, b, s[:7]), ValueError),
                      (lambda: hx.weight_grad(dy, b.t().contiguous().t(), s), ValueError),
                      (lambda: hx.weight_grad(dy.t(), b, s), ValueError),
                      (lambda: hx.weight_grad(dy, b, s, accumulate=True), ValueError),
                      (lambda: hx.weight_grad(dy, b, s, dtype=torch.float16), hx.HxError),
                      (lambda: hx.weight_grad(dy, b, s, out=torch.empty(24, 16, device=cuda)), ValueError),
                      (lambda: hx.weight_grad(dy, b, s, 7), hx.HxError)):
        with pytest.raises(err):
            call()

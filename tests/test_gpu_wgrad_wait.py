"""The weight gradient's bounded waits (failure detection without a GPU fault). A block of the launch whose part of X
never counts as ready (`withhold` of hx_weight_grad_bounded) makes the waits for it run out: HX_ERR_TIMEOUT is raised, its
cluster's part of the result is NaN (never sums that are not whole, nor what was there before), the rest is what it is
without, and the context stays usable."""
import pytest

torch = pytest.importorskip("torch")
from lossless_entropy_coding_fixed_b200 import hx  # noqa: E402

pytestmark = pytest.mark.gpu

FMT = {"e4m3": hx.ROWS_E4M3, "int8": hx.ROWS_INT8}
WAIT = 2_000_000  # ns


@pytest.fixture(scope="module")
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def setup(T, n, k, fmt, cuda):
    g = torch.Generator(device=cuda).manual_seed(T + n)
    dy = (0.05 * torch.randn(T, n, generator=g, device=cuda)).bfloat16()
    return (dy, *hx.quantize_rows(torch.randn(T, k, generator=g, device=cuda), FMT[fmt]))


CASES = [  # tokens, out, in, format, blocks of a cluster: steps fewer and more than the stages, in every kind of tile
    (60, 300, 260, "e4m3", 1), (200, 515, 300, "int8", 1), (1000, 3500, 1500, "e4m3", 2), (640, 1036, 261, "e4m3", 4),
    (3000, 3, 6, "e4m3", 8), (2000, 772, 1316, "e4m3", 4), (2000, 650, 897, "int8", 8), (100, 1664, 1664, "e4m3", 2),
    (130, 4096, 4096, "e4m3", 2), (2000, 4096, 4096, "int8", 2)]


@pytest.mark.parametrize("which", ["first", "second", "last"])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_withheld_block_leaves_nan(cuda, case, accumulate, which):
    T, n, k, fmt, cluster = case
    dy, b, s = setup(T, n, k, fmt, cuda)
    block = {"first": 0, "second": 1, "last": cluster - 1}[which]
    for dt in (torch.bfloat16, torch.float32):
        old = torch.randn(n, k, device=cuda).to(dt)
        want = hx.weight_grad(dy, b, s, FMT[fmt], out=old.clone(), accumulate=accumulate)
        got, st = hx.weight_grad_bounded(dy, b, s, old.clone(), WAIT, block, FMT[fmt], accumulate=accumulate)
        assert int(st.item()) == hx.HX_ERR_TIMEOUT
        lost = torch.isnan(got)
        assert torch.equal(torch.where(lost, want, got), want)
        # one cluster's tile and no more: a rectangle at the first row and column (the second block can be a tile of its own)
        rows, cols = lost.any(1).nonzero()[:, 0], lost.any(0).nonzero()[:, 0]
        hi, lo = [int(v.max()) + 1 for v in (rows, cols)], [int(v.min()) for v in (rows, cols)]
        assert lost[lo[0]:hi[0], lo[1]:hi[1]].all() and int(lost.sum()) == (hi[0] - lo[0]) * (hi[1] - lo[1])
        assert hi[0] - lo[0] <= 512 and hi[1] - lo[1] <= 256
        if block < cluster:
            assert lo == [0, 0] and hi[0] >= min(n, 128) and hi[1] >= min(k, 128)
        # and the context still works
        again = hx.weight_grad(dy, b, s, FMT[fmt], out=old.clone(), accumulate=accumulate)
        assert torch.equal(again, want)


def test_no_withheld_block(cuda):
    for case in CASES:
        dy, b, s = setup(*case[:4], cuda)
        want = hx.weight_grad(dy, b, s, FMT[case[3]])
        got, st = hx.weight_grad_bounded(dy, b, s, torch.empty_like(want), 10 ** 9, 1 << 40, FMT[case[3]])
        assert int(st.item()) == 0 and torch.equal(got, want)


def test_without_a_status_word_the_result_tells(cuda):
    dy, b, s = setup(130, 200, 100, "e4m3", cuda)
    out = torch.zeros(200, 100, device=cuda)
    rc = hx.lib().hx_weight_grad_bounded(0, hx.BF16, dy.data_ptr(), 200, b.data_ptr(), s.data_ptr(), 130, 200, 100, hx.F32,
                                         out.data_ptr(), 100, 0, None, 0, None, WAIT, 0,
                                         torch.cuda.current_stream().cuda_stream)
    assert rc == hx.HX_ERR_ARG  # rows of 100 bytes need a workspace
    ws = torch.empty(130 * 112, dtype=torch.uint8, device=cuda)
    rc = hx.lib().hx_weight_grad_bounded(0, hx.BF16, dy.data_ptr(), 200, b.data_ptr(), s.data_ptr(), 130, 200, 100, hx.F32,
                                         out.data_ptr(), 100, 0, ws.data_ptr(), ws.numel(), None, WAIT, 0,
                                         torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and torch.isnan(out).any()

"""The 8-bit-row operators together, their rows kept entropy coded between the passes: one block's forward and
backward pass (head norm and rotation, gated feed-forward layer, weight gradients), gradients against 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from lossless_entropy_coding_fixed_b200 import hx  # noqa: E402
from lossless_entropy_coding_fixed_b200.checkpoint import CheckpointStore  # noqa: E402

from . import _rows as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def tables_for(samples, cuda, kind=hx.KIND_HUFFMAN):
    counts = np.zeros(256, np.uint64)
    for b in samples:
        counts += np.bincount(b.cpu().numpy().reshape(-1), minlength=256).astype(np.uint64)
    build = {hx.KIND_HUFFMAN: hx.build_codebook, hx.KIND_QLC: hx.qlc_build, hx.KIND_SHANNONIC: hx.shannonic_build}
    return build[kind](counts).upload(cuda)


@pytest.mark.parametrize("kind", [hx.KIND_HUFFMAN, hx.KIND_QLC, hx.KIND_SHANNONIC])
@pytest.mark.parametrize("fmt", [hx.ROWS_E4M3, hx.ROWS_INT8])
def test_store_gives_back_every_byte(cuda, kind, fmt):
    g = torch.Generator(device=cuda).manual_seed(4)
    rows = [hx.quantize_rows(0.5 * torch.randn(r, c, generator=g, device=cuda).bfloat16(), fmt)
            for r, c in ((0, 8), (1, 1), (300, 700), (64, 4096), (777, 1365), (1024, 4096))]
    hist = torch.zeros(256, dtype=torch.int32, device=cuda)
    store = CheckpointStore(tables_for([b for b, _ in rows], cuda, kind), kind, hist=hist)
    keys = [store.put(b, s) for b, s in rows[:4]]
    unsealed = store.nbytes()
    store.seal()
    assert store.nbytes() < unsealed
    keys += [store.put(b, s) for b, s in rows[4:]]
    raw = sum(b.numel() for b, _ in rows)
    late = store.take(keys.pop())  # not sealed
    assert torch.equal(late[0], rows[-1][0]) and late[1] is rows[-1][1]
    store.seal()
    store.seal()
    assert store.nbytes() < sum(b.numel() + 4 * s.numel() for b, s in rows[:5])
    for key, (b, s) in reversed(list(zip(keys, rows))):
        got, sc = store.take(key)
        assert torch.equal(got, b) and sc is s
    store.check()
    assert len(store) == 0 and int(hist.sum()) == raw
    with pytest.raises(KeyError):
        store.take(keys[0])


def test_store_reports_a_byte_without_a_code(cuda):
    counts = np.zeros(256, np.uint64)
    counts[:10] = 5
    store = CheckpointStore(hx.build_codebook(counts, seen_only=True).upload(cuda))
    s = torch.ones(4, device=cuda)
    good = store.put(torch.full((4, 100), 3, dtype=torch.uint8, device=cuda), s)
    store.put(torch.full((4, 100), 30, dtype=torch.uint8, device=cuda), s)
    with pytest.raises(hx.HxError) as e:
        store.seal()
    assert e.value.code == hx.HX_ERR_UNCODABLE and len(store) == 1
    assert (store.take(good)[0] == 3).all()
    store.check()
    bad = store.put(torch.full((4, 100), 30, dtype=torch.uint8, device=cuda), s)
    store.take(bad)  # before anything was read back
    with pytest.raises(hx.HxError) as e:
        store.check()
    assert e.value.code & hx.HX_ERR_UNCODABLE
    store.check()  # told once
    with pytest.raises(TypeError):
        store.put(s, s)


@pytest.mark.parametrize("fmt,name", [(hx.ROWS_E4M3, "e4m3"), (hx.ROWS_INT8, "int8")])
def test_a_block_forward_and_backward(cuda, fmt, name):
    T, D, F, nq, nk, hd = 333, 256, 520, 4, 2, 64
    g = torch.Generator(device=cuda).manual_seed(11)
    rnd = lambda *s: torch.randn(*s, generator=g, device=cuda)  # noqa: E731
    bf = torch.bfloat16
    x = rnd(T, D).to(bf)
    wqk, wgu, wd = (rnd(*s).mul_(s[1] ** -0.5).to(bf) for s in (((nq + nk) * hd, D), (2 * F, D), (D, F)))
    wq, wk = 1 + 0.1 * rnd(hd), 1 + 0.1 * rnd(hd)
    ang = torch.arange(T, device=cuda, dtype=torch.float64)[:, None] * 100.0 ** (-torch.arange(0, hd, 2, device=cuda) / hd)
    cos, sin, pos = ang.cos().float(), ang.sin().float(), torch.arange(T, device=cuda)

    # a codebook from an earlier batch
    early = rnd(T, D).to(bf)
    store = CheckpointStore(tables_for([hx.quantize_rows(early, fmt)[0], hx.quantize_rows(early @ wgu.T, fmt)[0]], cuda))

    # forward: nothing but coded rows is kept of x, the projections and the activation
    b, s = hx.quantize_rows(x, fmt)
    kx = store.put(b, s)
    qk = (x @ wqk.T).view(T, nq + nk, hd)
    y, b, s = hx.head_norm_rope_forward(qk, nq, wq, wk, cos, sin, pos, fmt=fmt)
    kqk = store.put(b, s)
    h, b, s = hx.gated_forward(x @ wgu.T, fmt)
    kgu = store.put(b, s)
    out = h @ wd.T
    store.seal()
    del b, s, h, qk

    # backward
    dy, dout = 0.1 * rnd(T, nq + nk, hd).to(bf), 0.1 * rnd(T, D).to(bf)
    bgu, sgu = store.take(kgu)
    dh = dout @ wd
    dgu, h2 = hx.gated_backward(dh, bgu, sgu, fmt, need_h=True)
    bh, sh = hx.quantize_rows(h2, fmt)
    dwd = hx.weight_grad(dout, bh, sh, fmt)
    bqk, sqk = store.take(kqk)
    dqk, dwq, dwk = hx.head_norm_rope_backward(dy, bqk, sqk, nq, wq, wk, cos, sin, pos, fmt=fmt)
    bx, sx = store.take(kx)
    dwgu = hx.weight_grad(dgu, bx, sx, fmt)
    dwqk = torch.zeros(wqk.shape, device=cuda)
    hx.weight_grad(dqk.view(T, -1), bx, sx, fmt, out=dwqk, accumulate=True)

    # 64 bits, from the definitions, at the rows as they were saved and at the gradients as they were handed on
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    vx, vgu, vqk, vh = (ref.values(a.cpu().numpy(), f64(c), name) for a, c in ((bx, sx), (bgu, sgu), (bqk, sqk), (bh, sh)))
    near = lambda got, want: np.linalg.norm(f64(got) - want) <= 2.0 ** -8 * np.linalg.norm(want)  # noqa: E731
    dg, du = ref.gated_grad(vgu[:, 0], vgu[:, 1], f64(dh))
    assert near(dgu, np.concatenate([dg, du], 1)) and near(h2, ref.gated(vgu[:, 0], vgu[:, 1]))
    rx, rq, rk = ref.head_norm_rope_grad(f64(dy), vqk, nq, f64(wq), f64(wk), f64(cos), f64(sin), 1e-6, False)
    assert near(dqk, rx) and near(dwq, rq) and near(dwk, rk)
    assert near(dwd, f64(dout).T @ vh)
    assert near(dwgu, f64(dgu).T @ vx) and near(dwqk, f64(dqk).reshape(T, -1).T @ vx)

    # and against the block without any rows: the saved values are within half a step of theirs (e4m3 2^-4; INT8 half
    # of 1/127 of a row's largest), which the gradients inherit
    xt = x.double().requires_grad_(False)
    leaves = [w.double().requires_grad_(True) for w in (wqk, wgu, wd, wq, wk)]
    lqk, lgu, ld, lq, lk = leaves
    q = (xt @ lqk.T).view(T, nq + nk, hd)
    n = q / torch.sqrt(q.square().mean(-1, keepdim=True) + 1e-6)
    n = torch.cat((n[:, :nq] * lq, n[:, nq:] * lk), 1)
    a, c = n[..., :hd // 2], n[..., hd // 2:]
    cc, ss = cos.double()[:, None], sin.double()[:, None]
    full = torch.cat((a * cc - c * ss, c * cc + a * ss), -1)
    gu = xt @ lgu.T
    o = (torch.nn.functional.silu(gu[:, :F]) * gu[:, F:]) @ ld.T
    ((full * dy.double()).sum() + (o * dout.double()).sum()).backward()
    for got, w in zip((dwqk, dwgu, dwd, dwq, dwk), leaves):
        assert float((got.double() - w.grad).norm() / w.grad.norm()) < 2.0 ** -4
    full, o = full.detach(), o.detach()
    assert float((y.double() - full).norm() / full.norm()) < 2.0 ** -6
    assert float((out.double() - o).norm() / o.norm()) < 2.0 ** -6

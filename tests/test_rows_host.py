"""8-bit rows without a GPU: the definitions the GPU tests compare with (against the INT8 weight law, and
gradients against differences), and the refusals of the C calls, which come before any CUDA work."""
import ctypes

import numpy as np
import pytest

import datagen
from lossless_entropy_coding_fixed_b200 import hx

from . import _rows as ref


def test_int8_definition_is_the_weight_law():
    m = datagen._draw("student_t4", np.random.default_rng(3), 64 * 257, 0.02).reshape(64, 257)
    m[5] = 0
    b, s = ref.quantize(m.astype(np.float64), "int8")
    assert (b.reshape(-1) == datagen.int8_rowwise_bytes(m)).all()
    assert s[5] == 1


def test_e4m3_definition_scale():
    x = np.array([[448.0, 1], [448.0001, 1], [0.4375, 0], [np.nan, 1], [np.inf, 1], [0, 0], [1e-44, 0], [3e38, 0]])
    s = ref.scale(x, "e4m3")
    assert s[0] == 1 and s[1] == 2 and s[2] == 2.0 ** -10 and s[5] == 1
    assert np.isnan(s[3]) and np.isnan(s[4])
    assert s[6] == 2.0 ** -126 and s[7] == 2.0 ** 119


def test_gated_gradient_against_differences():
    rng = np.random.default_rng(0)
    g, u, dh = rng.normal(0, 2, (3, 50))
    dg, du = ref.gated_grad(g, u, dh)
    e = 1e-6
    assert np.allclose((ref.gated(g + e, u) - ref.gated(g - e, u)) / (2 * e) * dh, dg, rtol=0, atol=1e-8)
    assert np.allclose((ref.gated(g, u + e) - ref.gated(g, u - e)) / (2 * e) * dh, du, rtol=0, atol=1e-8)


@pytest.mark.parametrize("inter", [False, True])
def test_head_norm_rope_gradient_against_differences(inter):
    rng = np.random.default_rng(1)
    T, H, nq, D, R = 3, 3, 2, 10, 6
    x, dy = rng.normal(0, 1, (2, T, H, D))
    wq, wk = rng.normal(1, 0.2, (2, D))
    ang = rng.uniform(0, 6, (T, R // 2))
    cos, sin = np.cos(ang), np.sin(ang)

    def loss(x, wq, wk):
        return (ref.head_norm_rope(x, nq, wq, wk, cos, sin, 1e-6, inter) * dy).sum()

    dx, dwq, dwk = ref.head_norm_rope_grad(dy, x, nq, wq, wk, cos, sin, 1e-6, inter)
    e = 1e-6
    for idx in [(0, 0, 0), (1, 2, 9), (2, 1, 5), (0, 2, 3)]:
        d = np.zeros_like(x)
        d[idx] = e
        assert abs((loss(x + d, wq, wk) - loss(x - d, wq, wk)) / (2 * e) - dx[idx]) < 1e-7
    for i in (0, 4, 9):
        d = np.zeros(D)
        d[i] = e
        assert abs((loss(x, wq + d, wk) - loss(x, wq - d, wk)) / (2 * e) - dwq[i]) < 1e-7
        assert abs((loss(x, wq, wk + d) - loss(x, wq, wk - d)) / (2 * e) - dwk[i]) < 1e-7


A = 4096  # stands for an aligned device address: nothing is read before the checks


def test_rows_refusals():
    L, bad = hx.lib(), hx.HX_ERR_ARG
    q = L.hx_quantize_rows
    assert q(2, 0, A, 4, 8, 8, A, A, None) == bad  # no format 2
    assert q(0, 3, A, 4, 8, 8, A, A, None) == bad  # no element type 3
    assert q(0, 0, A, 4, 0, 8, A, A, None) == bad  # rows of nothing
    assert q(0, 0, A, 4, 8, 7, A, A, None) == bad  # rows that overlap
    assert q(0, 0, None, 4, 8, 8, A, A, None) == bad
    assert q(0, 0, A, 4, 8, 8, None, A, None) == bad
    assert q(0, 0, A, 4, 8, 8, A, None, None) == bad
    assert q(0, 0, A + 2, 4, 8, 8, A, A, None) == bad  # f32 on 2 bytes
    assert q(0, 2, A + 1, 4, 8, 8, A, A, None) == bad
    assert q(0, 0, A, 4, 8, 8, A, A + 2, None) == bad
    assert q(0, 0, A, 1 << 31, 8, 8, A, A, None) == bad
    assert q(0, 0, A, 4, 1 << 30, 1 << 30, A, A, None) == bad
    assert q(0, 0, A, 1 << 30, 1 << 20, 1 << 20, A, A, None) == bad
    assert q(0, 0, None, 0, 8, 8, None, None, None) == 0  # no rows: nothing to do
    d = L.hx_dequantize_rows
    assert d(0, 5, A, A, 4, 8, A, 8, None) == bad
    assert d(0, 0, A, A, 4, 8, A, 7, None) == bad
    assert d(0, 0, None, A, 4, 8, A, 8, None) == bad
    assert d(0, 0, A, A, 4, 8, A + 2, 8, None) == bad
    assert d(0, 0, A, A, 0, 8, None, 8, None) == 0
    f = L.hx_gated_forward
    assert f(0, 2, A, 4, 8, 15, A, A, A, None) == bad  # gate and up do not fit the stride
    assert f(0, 2, A, 4, 8, 16, A, A, None, None) == bad  # bytes without scales
    assert f(0, 2, A, 4, 8, 16, A, None, A, None) == bad
    assert f(0, 2, A, 4, 8, 16, None, A, A, None) == bad
    assert f(0, 2, A, 0, 8, 16, A, A, A, None) == 0
    b = L.hx_gated_backward
    assert b(0, 2, A, 7, A, A, 4, 8, A, None, None) == bad
    assert b(0, 2, A, 8, None, A, 4, 8, A, None, None) == bad
    assert b(0, 2, A, 8, A, None, 4, 8, A, None, None) == bad
    assert b(0, 2, A, 8, A, A, 4, 8, None, None, None) == bad
    assert b(0, 2, A, 8, A, A, 4, 8, A, A + 1, None) == bad
    assert b(0, 2, A, 8, A, A, 0, 8, A, None, None) == 0


def _norm(**kw):
    p = dict(format=0, dtype=2, weight_dtype=0, position_bits=64, tokens=4, q_heads=4, k_heads=2, dim=64, rot_dim=64,
             interleaved=0, eps=1e-6, places=16, d_wq=A, d_wk=A, d_cos=A, d_sin=A, d_positions=A)
    p.update(kw)
    return ctypes.byref(hx._HeadNormRope(**p))


@pytest.mark.parametrize("kw", [
    dict(format=2), dict(dtype=3), dict(weight_dtype=1), dict(position_bits=16), dict(q_heads=0, k_heads=0),
    dict(dim=63), dict(dim=0), dict(dim=514), dict(rot_dim=66), dict(rot_dim=3), dict(eps=-1.0), dict(eps=float("nan")),
    dict(places=0), dict(d_wq=None), dict(d_wk=None), dict(d_cos=None), dict(d_sin=None), dict(d_positions=None),
    dict(d_cos=A + 2), dict(d_wq=A + 2), dict(d_positions=A + 4), dict(tokens=1 << 31), dict(q_heads=1 << 21)])
def test_head_norm_rope_refusals(kw):
    L, bad = hx.lib(), hx.HX_ERR_ARG
    n = L.hx_head_norm_rope_workspace(64)
    assert L.hx_head_norm_rope_forward(_norm(**kw), A, 384, 64, A, 384, 64, A, A, None, None) == bad
    assert L.hx_head_norm_rope_backward(_norm(**kw), A, 384, 64, A, A, A, 384, 64, A, A, A, n, None, None) == bad


def test_head_norm_rope_fields():
    """The binding's packed arguments have the layout of the C structure."""
    v = (0, 2, 0, 64, 4, 4, 2, 64, 32, 1, 0.5, 16, A, A + 8, A + 16, A + 24, A + 32)
    p = hx._HeadNormRope.from_buffer_copy(hx._NORM.pack(*v))
    assert ctypes.sizeof(p) == hx._NORM.size
    assert tuple(getattr(p, n) for n, _ in p._fields_) == v


def test_head_norm_rope_call_refusals():
    L, bad = hx.lib(), hx.HX_ERR_ARG
    f, b = L.hx_head_norm_rope_forward, L.hx_head_norm_rope_backward
    n = L.hx_head_norm_rope_workspace(64)
    assert n > 0
    assert f(None, A, 384, 64, A, 384, 64, A, A, None, None) == bad
    assert f(_norm(), None, 384, 64, A, 384, 64, A, A, None, None) == bad
    assert f(_norm(), A, 384, 64, None, 384, 64, A, A, None, None) == bad
    assert f(_norm(), A, 384, 64, A, 384, 64, A, None, None, None) == bad  # bytes without scales
    assert f(_norm(), A + 1, 384, 64, A, 384, 64, A, A, None, None) == bad
    assert f(_norm(tokens=0), None, 384, 64, None, 384, 64, None, None, None, None) == 0
    assert b(_norm(), A, 384, 64, None, A, A, 384, 64, A, A, A, n, None, None) == bad
    assert b(_norm(), A, 384, 64, A, A, A, 384, 64, None, A, A, n, None, None) == bad
    assert b(_norm(), A, 384, 64, A, A, A, 384, 64, A, None, A, n, None, None) == bad
    assert b(_norm(), A, 384, 64, A, A, A, 384, 64, A, A, None, n, None, None) == bad
    assert b(_norm(), A, 384, 64, A, A, A, 384, 64, A, A, A, n - 1, None, None) == bad


def test_weight_grad_refusals():
    L, bad = hx.lib(), hx.HX_ERR_ARG
    w = L.hx_weight_grad

    def call(fmt=0, dt=2, dy=A, ld=64, b=A, s=A, t=128, n=64, k=32, wt=2, dw=A, ldw=32, acc=0, ws=A, wsb=1 << 30, st=None):
        return w(fmt, dt, dy, ld, b, s, t, n, k, wt, dw, ldw, acc, ws, wsb, st, None)

    for kw in (dict(fmt=2), dict(dt=0), dict(dt=3), dict(wt=1), dict(dy=None), dict(b=None), dict(s=None), dict(dw=None),
               dict(ld=63), dict(ldw=31), dict(n=0), dict(k=0), dict(t=1 << 31), dict(n=(1 << 23) + 1, ld=1 << 24),
               dict(k=(1 << 22) + 1, ldw=1 << 23), dict(dy=A + 1), dict(dw=A + 1), dict(s=A + 2), dict(st=A + 2)):
        assert call(**kw) == bad, kw
    need = L.hx_weight_grad_workspace
    assert need(A, 64, A, 128, 64, 32) == 0  # rows that TMA takes as they are
    odd = need(A, 65, A, 128, 64, 32)
    assert odd >= 128 * 64 * 2 and need(A + 2, 64, A, 128, 64, 32) == odd
    assert need(A, 64, A + 1, 128, 64, 32) >= 128 * 32 and need(A, 64, A, 128, 64, 33) >= 128 * 33
    assert call(ld=65, ws=None) == bad
    assert call(ld=65, wsb=odd - 1) == bad
    assert call(ld=65, ws=A + 4) == bad
    assert call(t=0, acc=1, dy=None, b=None, s=None) == 0  # nothing to add
    assert need(None, 64, None, 0, 64, 32) == 0


def test_binding_refuses_tensors_that_are_not_on_a_gpu():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 8)
    b, s = torch.zeros(4, 8, dtype=torch.uint8), torch.zeros(4)
    for call in (lambda: hx.quantize_rows(x), lambda: hx.dequantize_rows(b, s), lambda: hx.gated_forward(x),
                 lambda: hx.gated_backward(x, b, s), lambda: hx.weight_grad(x, b, s),
                 lambda: hx.head_norm_rope_forward(x.view(1, 4, 8), 2, s, s, x, x, s)):
        with pytest.raises(TypeError):
            call()


def test_weight_grad_bounded_refuses_what_the_call_refuses():
    w, bad = hx.lib().hx_weight_grad_bounded, hx.HX_ERR_ARG
    tail = (10 ** 6, 0, None)
    assert w(2, 2, A, 64, A, A, 128, 64, 32, 2, A, 32, 0, A, 1 << 30, None, *tail) == bad
    assert w(0, 2, A, 65, A, A, 128, 64, 32, 2, A, 32, 0, None, 0, None, *tail) == bad
    assert w(0, 2, A, 64, A, A, 128, 64, 32, 2, A, 31, 0, A, 1 << 30, None, *tail) == bad
    assert w(0, 2, None, 64, None, None, 0, 64, 32, 2, A, 32, 1, None, 0, None, *tail) == 0

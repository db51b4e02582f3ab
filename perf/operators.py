"""The 8-bit activation checkpoint operators, their plain forms and the cases they are measured on.

Four operators work on "8-bit rows": a matrix of bytes (e4m3 or INT8), one 32-bit scale per row, the
bytes being what the entropy coder codes.

  rows    save: quantise the rows of a matrix; load: bytes and scales back to values
  gated   silu(gate) * up of a gated feed-forward layer that saves gate and up as 8-bit rows, and its
          backward pass, which reads them
  qk      per-head RMS norm of queries and keys with the position rotation in the same pass, the
          inputs saved as 8-bit rows, and its backward pass, which reads them
  wgrad   the weight gradient of a linear layer, dY^T X, from the 8-bit rows of its input X

Scales. e4m3: the smallest power of two s, within 2^-126 .. 2^119, with absmax / s <= 448, so that a
byte's value times its scale is exact. INT8: s = absmax / 127 within 2^-126 .. 2^121, the symmetric
per-row law of the INT8 weight matrices. A row of zeros has the scale 1; a row with a NaN or an
infinity has the scale NaN and bytes of 0.

`run` computes the operators from elementary torch operations in 32 bits, or (own = True) calls the
library. `exact` computes them in 64 bits, apart from both.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


# ------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # an INT8 weight matrix, quantised per row from the trainer's 32-bit copy
        {"name": "save_int8_weights", "op": "save", "fmt": "int8", "dtype": "f32", "rows": 8192, "cols": 8192, "pad": 0},
        # a short ragged batch of activations (a column count that is odd), a slice of a wider buffer
        {"name": "save_e4m3_ragged", "op": "save", "fmt": "e4m3", "dtype": "bf16", "rows": 777, "cols": 1365, "pad": 11},
        # 64 MiB of saved activations brought back for a recomputation
        {"name": "load_e4m3", "op": "load", "fmt": "e4m3", "dtype": "bf16", "rows": 8192, "cols": 8192, "pad": 0},
        # a training step's feed-forward activation, saved
        {"name": "gated_forward", "op": "gated_fwd", "fmt": "e4m3", "dtype": "bf16", "rows": 8192, "cols": 8192, "save": True},
        # the same for one token being served: nothing is saved
        {"name": "gated_token", "op": "gated_fwd", "fmt": "e4m3", "dtype": "bf16", "rows": 1, "cols": 8192, "save": False},
        # its backward pass, with the activation itself recomputed for the next weight gradient
        {"name": "gated_backward", "op": "gated_bwd", "fmt": "e4m3", "dtype": "bf16", "rows": 8192, "cols": 8192},
        # queries and keys of a training step, read out of the packed projection
        {"name": "qk_forward", "op": "qk_fwd", "fmt": "e4m3", "dtype": "bf16", "tokens": 8192, "q": 32, "k": 8, "dim": 128, "rot": 128, "inter": False, "save": True},
        # one token being served
        {"name": "qk_token", "op": "qk_fwd", "fmt": "e4m3", "dtype": "bf16", "tokens": 1, "q": 32, "k": 8, "dim": 128, "rot": 128, "inter": False, "save": False},
        # the backward pass of the training step
        {"name": "qk_backward", "op": "qk_bwd", "fmt": "e4m3", "dtype": "bf16", "tokens": 8192, "q": 32, "k": 8, "dim": 128, "rot": 128, "inter": False},
        # the weight gradient of a square projection over one step's tokens
        {"name": "wgrad_large", "op": "wgrad", "fmt": "e4m3", "dtype": "bf16", "tokens": 8192, "out": 8192, "in": 8192},
        # a narrow projection over a short batch, INT8 rows
        {"name": "wgrad_narrow", "op": "wgrad", "fmt": "int8", "dtype": "bf16", "tokens": 4096, "out": 1024, "in": 1024},
        # odd sizes throughout
        {"name": "wgrad_odd", "op": "wgrad", "fmt": "e4m3", "dtype": "f16", "tokens": 1001, "out": 515, "in": 1365},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["save", "load", "gated_fwd", "gated_bwd", "qk_fwd", "qk_bwd", "wgrad", "wgrad"])
    c = {"op": op, "fmt": rng.choice(["e4m3", "int8"])}
    if op == "wgrad":
        c["dtype"] = rng.choice(["bf16", "bf16", "f16"])
        most = 1 << 37
        c["tokens"] = _log(rng, 1, 16384)
        c["out"] = _log(rng, 1, 8192)
        c["in"] = _log(rng, 1, max(1, min(8192, most // (c["tokens"] * c["out"]))))
        if rng.random() < 0.6:  # most projections have round widths
            c["out"], c["in"] = (max(64, v // 64 * 64) for v in (c["out"], c["in"]))
        return c
    c["dtype"] = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("qk_fwd", "qk_bwd"):
        c["dim"] = rng.choice([32, 64, 80, 96, 128, 128, 192, 256, 2 * rng.randint(2, 100)])
        c["rot"] = c["dim"] if rng.random() < 0.6 else 2 * rng.randint(1, c["dim"] // 2)
        c["k"] = rng.choice([1, 2, 4, 8])
        c["q"] = c["k"] * rng.choice([1, 2, 3, 4, 8])
        c["tokens"] = _log(rng, 1, min(16384, (1 << 25) // (c["dim"] * (c["q"] + c["k"]))))
        c["inter"] = rng.random() < 0.4
        if op == "qk_fwd":
            c["save"] = rng.random() < 0.7
        return c
    c["cols"] = _log(rng, 1, 32768)
    if rng.random() < 0.5:
        c["cols"] = max(8, c["cols"] // 8 * 8)
    c["rows"] = _log(rng, 1, min(65536, (1 << 25) // c["cols"]))
    if op in ("save", "load"):
        c["pad"] = rng.choice([0, 0, 1, 8, rng.randint(1, 64)])
    elif op == "gated_fwd":
        c["save"] = rng.random() < 0.7
    return c


# ------------------------------------------------------------------------------------ the inputs
def _activations(gen, rows, cols, dtype):
    """What a layer hands on: nine Laplace values to one of a wide normal, a level of its own for
    each row, and now and then a row of zeros (a padded token)."""
    dev = "cuda"
    u = torch.rand(rows, cols, generator=gen, device=dev).sub_(0.5)
    x = -0.3 * u.sign() * torch.log1p(-2 * u.abs().clamp_(max=0.4999999))
    wide = torch.rand(rows, cols, generator=gen, device=dev) < 0.1
    x = torch.where(wide, 3 * torch.randn(rows, cols, generator=gen, device=dev), x)
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=gen, device=dev))
    if rows > 8:
        x[torch.rand(rows, generator=gen, device=dev) < 0.02] = 0
    return x.to(dtype)


def _padded(x, pad):
    """x as the left columns of a buffer that is `pad` columns wider."""
    if not pad:
        return x
    b = torch.zeros(x.shape[0], x.shape[1] + pad, dtype=x.dtype, device=x.device)
    b[:, :x.shape[1]] = x
    return b[:, :x.shape[1]]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s, op = dict(case), case["op"]
    dt = DTYPES[case["dtype"]]
    if op == "save":
        s["x"] = _padded(_activations(gen, case["rows"], case["cols"], dt), case["pad"])
    elif op == "load":
        s["bytes"], s["scale"] = _save(_activations(gen, case["rows"], case["cols"], dt), case["fmt"])
        s["out"] = _padded(torch.zeros(case["rows"], case["cols"], dtype=dt, device="cuda"), case["pad"])
    elif op == "gated_fwd":
        s["x"] = _activations(gen, case["rows"], 2 * case["cols"], dt)
    elif op == "gated_bwd":
        x = _activations(gen, 2 * case["rows"], case["cols"], dt)
        b, s["scale"] = _save(x, case["fmt"])
        s["bytes"], s["scale"] = b.view(case["rows"], 2, case["cols"]), s["scale"].view(case["rows"], 2)
        s["dh"] = (0.02 * torch.randn(case["rows"], case["cols"], generator=gen, device="cuda")).to(dt)
    elif op in ("qk_fwd", "qk_bwd"):
        t, h, d = case["tokens"], case["q"] + case["k"], case["dim"]
        s["wq"], s["wk"] = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda").to(torch.float32) for _ in range(2))
        places = 2 * t + 64
        # a packed batch: positions start anew with each sequence
        s["pos"] = (torch.arange(t, device="cuda") + int(torch.randint(0, t + 64, (1,), generator=gen, device="cuda"))) % places
        rate = 10000.0 ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64) / case["rot"])
        angle = torch.arange(places, device="cuda", dtype=torch.float64)[:, None] * rate
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        x = _activations(gen, t * h, d, dt)
        if op == "qk_fwd":  # the projection's output holds the values' heads behind the keys'
            packed = torch.zeros(t, h + case["k"], d, dtype=dt, device="cuda")
            packed[:, :h] = x.view(t, h, d)
            s["x"] = packed[:, :h]
        else:
            b, sc = _save(x, case["fmt"])
            s["bytes"], s["scale"] = b.view(t, h, d), sc.view(t, h)
            s["dy"] = (0.02 * torch.randn(t, h, d, generator=gen, device="cuda")).to(dt)
    else:
        s["dy"] = (0.02 * torch.randn(case["tokens"], case["out"], generator=gen, device="cuda")).to(dt)
        s["bytes"], s["scale"] = _save(_activations(gen, case["tokens"], case["in"], dt), case["fmt"])
    return s


# --------------------------------------------------------------------------------- the plain form
def _save(x, fmt):
    """Bytes (uint8) and scales of the rows of x."""
    x = x.float()
    top = x.abs().amax(-1)
    fine = torch.isfinite(x).all(-1)
    if fmt == "e4m3":
        # 448 = 7/8 * 2^9, so a fraction in [1/2, 1) above 7/8 needs the next power
        m, e = torch.frexp(top)
        scale = ((e - 9 + (m > 0.875).int()).clamp(-126, 119) + 127 << 23).view(torch.float32)
    else:
        scale = (top / torch.full_like(top, 127)).clamp(2.0 ** -126, 2.0 ** 121)
    scale = torch.where(top == 0, torch.ones_like(scale), scale)
    safe = torch.where(fine, scale, torch.ones_like(scale))[..., None]
    v = torch.where(fine[..., None], x, torch.zeros_like(x)) / safe
    if fmt == "e4m3":
        b = v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        b = v.round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
    return b, torch.where(fine, scale, torch.full_like(scale, math.nan))


def _load(b, scale, fmt):
    return b.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8).float() * scale[..., None]


def _values(b, fmt):
    """The bytes as the numbers they stand for, in units of their row's scale."""
    return b.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8)


def _pairs(v, rot, inter):
    """The two elements of each rotated pair."""
    if inter:
        return v[..., 0:rot:2], v[..., 1:rot:2]
    return v[..., :rot // 2], v[..., rot // 2:rot]


def _joined(a, b, rest, inter):
    r = torch.stack((a, b), -1).flatten(-2) if inter else torch.cat((a, b), -1)
    return torch.cat((r, rest), -1)


def _plain(s):
    op, fmt = s["op"], s["fmt"]
    dt = DTYPES[s["dtype"]]
    if op == "save":
        b, scale = _save(s["x"], fmt)
        return _values(b, fmt), scale
    if op == "load":
        top = torch.finfo(dt).max
        s["out"].copy_(_load(s["bytes"], s["scale"], fmt).clamp(-top, top).to(dt))
        return s["out"]
    if op == "gated_fwd":
        n = s["cols"]
        x = s["x"].float()
        g, u = x[:, :n], x[:, n:]
        h = (g * torch.sigmoid(g) * u).to(dt)
        if not s["save"]:
            return h
        b, scale = _save(s["x"].view(-1, 2, n), fmt)
        return h, _values(b, fmt), scale
    if op == "gated_bwd":
        x = _load(s["bytes"], s["scale"], fmt)
        g, u, dh = x[:, 0], x[:, 1], s["dh"].float()
        p = torch.sigmoid(g)
        dg = dh * u * p * (1 + g * (1 - p))
        du = dh * g * p
        return torch.cat((dg, du), -1).to(dt), (g * p * u).to(dt)
    if op == "wgrad":
        return (s["dy"].float().T @ _load(s["bytes"], s["scale"], fmt)).to(dt)
    rot, inter, nq = s["rot"], s["inter"], s["q"]
    x = s["x"].float() if op == "qk_fwd" else _load(s["bytes"], s["scale"], fmt)
    w = torch.cat((s["wq"].expand(nq, -1), s["wk"].expand(s["k"], -1)))
    cos, sin = s["cos"][s["pos"]][:, None], s["sin"][s["pos"]][:, None]
    rstd = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
    if op == "qk_fwd":
        n = x * rstd * w
        a, b = _pairs(n, rot, inter)
        y = _joined(a * cos - b * sin, b * cos + a * sin, n[..., rot:], inter).to(dt)
        if not s["save"]:
            return y
        b, scale = _save(s["x"], fmt)
        return y, _values(b, fmt), scale
    dy = s["dy"].float()
    a, b = _pairs(dy, rot, inter)
    dn = _joined(a * cos + b * sin, b * cos - a * sin, dy[..., rot:], inter)
    xh = x * rstd
    dxh = dn * w
    dx = rstd * (dxh - xh * (dxh * xh).mean(-1, keepdim=True))
    dw = dn * xh
    return dx.to(dt), dw[:, :nq].sum((0, 1)), dw[:, nq:].sum((0, 1))


# ------------------------------------------------------------------------------ the library's calls
def _library(s):
    from lossless_entropy_coding_fixed_b200 import hx
    op = s["op"]
    fmt = hx.ROWS_E4M3 if s["fmt"] == "e4m3" else hx.ROWS_INT8
    if op == "save":
        b, scale = hx.quantize_rows(s["x"], fmt)
        return _values(b, s["fmt"]), scale
    if op == "load":
        return hx.dequantize_rows(s["bytes"], s["scale"], fmt, out=s["out"])
    if op == "gated_fwd":
        h, b, scale = hx.gated_forward(s["x"], fmt, save=s["save"])
        return (h, _values(b, s["fmt"]), scale) if s["save"] else h
    if op == "gated_bwd":
        return hx.gated_backward(s["dh"], s["bytes"], s["scale"], fmt, need_h=True)
    if op == "wgrad":
        return hx.weight_grad(s["dy"], s["bytes"], s["scale"], fmt)
    if op == "qk_fwd":
        y, b, scale = hx.head_norm_rope_forward(s["x"], s["q"], s["wq"], s["wk"], s["cos"], s["sin"], s["pos"], eps=EPS,
                                                interleaved=s["inter"], fmt=fmt, save=s["save"])
        return (y, _values(b, s["fmt"]), scale) if s["save"] else y
    return hx.head_norm_rope_backward(s["dy"], s["bytes"], s["scale"], s["q"], s["wq"], s["wk"], s["cos"], s["sin"], s["pos"],
                                      eps=EPS, interleaved=s["inter"], fmt=fmt)


def run(state):
    if own:
        return _library(state)
    return _plain(state)


# -------------------------------------------------------------------------------------- the work
def work(case):
    op = case["op"]
    e = {"f32": 4, "f16": 2, "bf16": 2}[case["dtype"]]
    if op == "wgrad":
        t, n, k = case["tokens"], case["out"], case["in"]
        return {"bytes": t * n * e + t * k + 4 * t + n * k * e, "flops": 2 * t * n * k}
    if op in ("qk_fwd", "qk_bwd"):
        t, h, d = case["tokens"], case["q"] + case["k"], case["dim"]
        extra = 8 * t + 4 * t * case["rot"] + 8 * d
        saved = t * h * (d + 4) if op == "qk_bwd" or case["save"] else 0
        return {"bytes": 2 * t * h * d * e + saved + extra + (8 * d if op == "qk_bwd" else 0),
                "flops": t * h * d * (8 if op == "qk_fwd" else 16)}
    r, n = case["rows"], case["cols"]
    if op in ("save", "load"):
        return {"bytes": r * (n * (e + 1) + 4), "flops": 2 * r * n}
    if op == "gated_fwd":
        return {"bytes": r * (3 * n * e + (2 * n + 8 if case["save"] else 0)), "flops": 8 * r * n}
    return {"bytes": r * (4 * n * e + 2 * n + 8), "flops": 16 * r * n}


# ------------------------------------------------------------------- the definition, in 64 bits
def _exact_scale(x, fmt):
    """Each row's scale, from the definition."""
    top = x.abs().amax(-1)
    if fmt == "e4m3":
        k = torch.ceil(torch.log2(top / 448)).clamp(-126, 119)
        k = torch.where(top > 448 * torch.exp2(k), k + 1, k)
        k = torch.where(top <= 448 * torch.exp2(k - 1), k - 1, k).clamp(-126, 119)
        s = torch.exp2(k)
    else:
        s = (top / 127).clamp(2.0 ** -126, 2.0 ** 121)
    s[top == 0] = 1
    s[~torch.isfinite(top)] = math.nan
    return s


def _exact_e4m3(v):
    """Values to the nearest of e4m3 (3 fraction bits, smallest normal 2^-6), ties to even."""
    m = v.abs().clamp(max=448)
    step = torch.exp2(torch.floor(torch.log2(m.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(v) * (torch.round(m / step) * step).clamp(max=448)


def _exact_saved(x, fmt):
    s = _exact_scale(x, fmt)
    return (_exact_e4m3(x / s[..., None]) if fmt == "e4m3" else None), s


def exact(case, seed):
    s = prepare(case, seed)
    op, fmt = case["op"], case["fmt"]
    if "bytes" in s:
        b = s["bytes"].to(torch.int64)
        if fmt == "e4m3":
            e, m = (b >> 3) & 15, (b & 7).double()
            v = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e.double() - 7))
            v = torch.where(b >= 128, -v, v)
        else:
            v = torch.where(b >= 128, b - 256, b).double()
        x = v * s["scale"].double().unsqueeze(-1)
    else:
        x = s["x"].double()
    if op == "save":
        return _exact_saved(x, fmt)
    if op == "load":
        return x
    if op == "wgrad":
        return torch.einsum("to,ti->oi", s["dy"].double(), x)
    if op in ("gated_fwd", "gated_bwd"):
        x = x.reshape(case["rows"], 2, case["cols"])
        g, u = x[:, 0], x[:, 1]
        silu = g / (1 + torch.exp(-g))
        if op == "gated_fwd":
            return (silu * u, *_exact_saved(x, fmt)) if case["save"] else silu * u
        dh = s["dh"].double()
        slope = (1 + torch.exp(-g) * (1 + g)) / (1 + torch.exp(-g)).square()
        return torch.cat((dh * u * slope, dh * silu), -1), silu * u
    nq, rot, d = case["q"], case["rot"], case["dim"]
    i = torch.arange(rot // 2, device=x.device)
    first, second = (2 * i, 2 * i + 1) if case["inter"] else (i, i + rot // 2)
    cos, sin = s["cos"].double()[s["pos"]], s["sin"].double()[s["pos"]]
    norm = torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS)
    w = torch.ones_like(x)
    w[:, :nq] *= s["wq"].double()
    w[:, nq:] *= s["wk"].double()

    def turned(v, sign):
        z = torch.complex(v[..., first], v[..., second]) * torch.complex(cos, sign * sin)[:, None]
        r = v.clone()
        r[..., first], r[..., second] = z.real, z.imag
        return r

    if op == "qk_fwd":
        y = turned(x / norm * w, 1)
        return (y, *_exact_saved(x, fmt)) if case["save"] else y
    dn = turned(s["dy"].double(), -1)
    grad = dn * w
    dx = grad / norm - x * (grad * x).sum(-1, keepdim=True) / (d * norm ** 3)
    dw = (dn * x / norm).sum(0)
    return dx, dw[:nq].sum(0), dw[nq:].sum(0)

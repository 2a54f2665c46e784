"""The 8-bit formats and the layer built on them, in 64 bits on the CPU, with
bounds on what a correct fp32 computation may differ by.

Intervals are (centre, radius) pairs of float64 tensors: a quantity that is
computed in fp32 lies within radius of centre, and rounding (to codes, or to a
16-bit type) is monotone, so the rounded ends enclose the rounded value.
"""
import math

import torch

B = 128
U = 2.0**-24  # half a step of fp32
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
FLOOR = 448 * 2.0**-126


def nb(n):
    return -(-n // B)


def e4m3(v):
    """The nearest e4m3 value (ties to even) of |v| <= 448, from the format's definition."""
    m = v.abs()
    e = torch.floor(torch.log2(m.clamp_min(2.0**-30)))
    e = torch.where(m < torch.exp2(e), e - 1, e).clamp(-6, 8)
    step = torch.exp2(e - 3)
    return torch.sign(v) * torch.round(m / step) * step


def _blocked(x, rows):
    """[M][R][C] -> [M][R blocks of `rows`][rows][C blocks][128], padded with zeros."""
    M, R, C = x.shape
    nr = -(-R // rows)
    p = torch.nn.functional.pad(x, (0, nb(C) * B - C, 0, nr * rows - R))
    return p.view(M, nr, rows, nb(C), B)


def quantize(x, rows):
    """Code values [M][R][C] and scales [M][R blocks][C blocks] of x in 64 bits (rows = 1 or 128)."""
    M, R, C = x.shape
    p = _blocked(x.double(), rows)
    m = p.abs().amax(dim=(2, 4)).clamp_min(FLOOR)
    q = e4m3(p * 448 / m[:, :, None, :, None])
    q = q.view(M, -1, nb(C) * B)[:, :R, :C]
    return q, m / 448


def code_values(codes):
    return codes.view(torch.float8_e4m3fn).float().double()


def row_values(codes, scales):
    """Rows [R][K] of codes with scales [blocks][R]."""
    return code_values(codes) * scales.double().t().repeat_interleave(B, dim=1)[:, :codes.shape[1]]


def matrix_values(codes, scales):
    """Matrices [M][N][K] of codes with scales [M][N blocks][K blocks]."""
    s = scales.double().repeat_interleave(B, dim=1)[:, :codes.shape[1]]
    return code_values(codes) * s.repeat_interleave(B, dim=2)[:, :, :codes.shape[2]]


def product_radius(K):
    """Relative to the sum of the magnitudes: 128 additions in a block (a whole
    step each, whichever way the matrix cores round), the blocks' running sum,
    and the product of two scales."""
    return (B + nb(K) + 2) * 2 * U


def product(a, w):
    """a [R][K] times w [N][K]^T with its fp32 radius."""
    return a @ w.t(), product_radius(a.shape[1]) * (a.abs() @ w.abs().t())


def dropped(a, w):
    """What the 8-bit matrix instruction may leave out of a w^T: of the products of 8 neighbouring
    elements, aligned to the largest, each but that one loses less than 2^-13 of the largest's power of two."""
    out = torch.zeros((a.shape[0], w.shape[0]), dtype=torch.float64)
    for k in range(0, a.shape[1], 8):
        p = (a[:, None, k:k + 8] * w[None, :, k:k + 8]).abs()
        out += 7 * 2.0**-13 * p.amax(dim=2)
    return out


def rounded(v, act):
    """An interval after rounding to a 16-bit type."""
    c, r = v
    f = lambda t: t.to(TORCH[act]).double()  # noqa: E731
    lo, hi, mid = f(c - r), f(c + r), f(c)
    return mid, torch.maximum(hi - mid, mid - lo)


def gated(g, u, geglu, act):
    """The gated unit of two intervals; act: the type of its per-operation rounding, or None.  The fp32
    gate is within (8 + 2 |g|) steps of 2 U: the exponential's argument rounds once, and exp2, the
    reciprocal and the products are a few units each; its slope is below 1.13."""
    rd = (lambda v: rounded(v, act)) if act else (lambda v: v)
    times = lambda p, q: (p[0] * q[0], p[0].abs() * q[1] + q[0].abs() * p[1] + p[1] * q[1]  # noqa: E731
                          + 2 * U * (p[0] * q[0]).abs())
    (gc, gr), u = rd(g), rd(u)
    units = (8 + 2 * gc.abs()) * 2 * U
    if geglu:
        z = math.sqrt(2 / math.pi) * (gc + 0.044715 * gc**3)
        a = 0.5 * gc * (1 + torch.tanh(z))
        # the cubic's rounding enters the exponent too
        return rd(times(rd((a, 1.13 * gr + a.abs() * (units + 8 * z.abs() * U) + 1e-37)), u))
    s = torch.sigmoid(gc)
    if not act:
        a = gc * s
        return times((a, 1.13 * gr + a.abs() * units + 1e-37), u)
    s = rd((s, 0.25 * gr + s * units + 1e-37))
    return rd(times(rd(times((gc, gr), s)), u))


def quantized_rows(v, halves):
    """The values that row codes of an interval [R][C] stand for, as an interval.  halves: the values are of
    a 16-bit type, and so are the interval's ends: 448 x is then exact in fp32, and the quotient of two such
    values is a border between codes or further from it than fp32 rounds, so nothing is added for it."""
    c, r = v
    R, C = c.shape
    blk = lambda t: _blocked(t[None], 1)[0][:, 0]  # noqa: E731   [R][blocks][128]
    pc, pr = blk(c), blk(r)
    mag = pc.abs()
    m = mag.amax(dim=2).clamp_min(FLOOR)
    lo_m = (mag - pr).amax(dim=2).clamp_min(FLOOR)
    hi_m = (mag + pr).amax(dim=2).clamp_min(FLOOR)
    val = lambda x, mm: e4m3((x * 448 / mm[:, :, None]).clamp(-448, 448)) * (mm / 448)[:, :, None]  # noqa: E731
    mid = val(pc, m)
    # the quotient of a value and a maximum that both moved, a few roundings on top
    ends = []
    for x in (pc - pr, pc + pr):
        for mm in (lo_m, hi_m):
            for f in (1,) if halves else (1 - 4 * U, 1 + 4 * U):
                ends.append(e4m3((x * 448 / mm[:, :, None] * f).clamp(-448, 448)))
    ends = torch.stack(ends)
    hi = ends.amax(dim=0) * (m / 448)[:, :, None]
    lo = ends.amin(dim=0) * (m / 448)[:, :, None]
    rad = torch.maximum(hi - mid, mid - lo)
    rad = rad + (mid.abs() + rad) * ((hi_m - lo_m) / lo_m + 4 * U)[:, :, None]  # the scale moves with m, and rounds
    flat = lambda t: t.reshape(R, -1)[:, :C]  # noqa: E731
    return flat(mid), flat(rad)


def product_of(v, w):
    """An interval of rows times w^T."""
    c, r = v
    return c @ w.t(), product_radius(c.shape[1]) * ((c.abs() + r) @ w.abs().t()) + r @ w.abs().t()

"""The 8-bit products on the GPU against the formulas in 64 bits: quantisation
value by value, the grouped product within a bound that counts its roundings,
the layer within one that follows them through the second quantisation."""
import numpy as np
import pytest
import torch

import fp8_ref as ref
from sparse_mixture_experts_amd import moe

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"f32": moe.MOE_DT_F32, "bf16": moe.MOE_DT_BF16, "f16": moe.MOE_DT_F16}
NAN, INF = float("nan"), float("inf")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def quantize(x, act, block_rows):
    """x [M][R][C] (CPU) through the library: codes (uint8) and scales on the CPU."""
    M, R, C = x.shape
    codes = torch.full((M, R, C), 0xAA, dtype=torch.uint8, device=DEV)
    shape = (ref.nb(C), M * R) if block_rows == 1 else (M, ref.nb(R), ref.nb(C))
    scales = torch.full(shape, NAN, device=DEV)
    moe.moe_fp8_quantize(M, R, C, x.to(DEV), DT[act], block_rows, codes, scales)
    torch.cuda.synchronize()
    return codes.cpu(), scales.cpu()


def make_weights(g, M, N, K):
    w = torch.randn((M, N, K), generator=g) * K**-0.5
    q, s = ref.quantize(w, B)
    codes = q.float().to(torch.float8_e4m3fn).view(torch.uint8).contiguous()
    return codes, s.float().contiguous()


B = ref.B

QUANT = [  # M, R, C
    (1, 1, 16), (1, 1, 2048), (1, 3, 128), (1, 33, 144), (2, 31, 112), (1, 129, 272), (3, 130, 400), (1, 257, 1040),
]


@pytest.mark.parametrize("act", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("M,R,C", QUANT)
def test_quantize(M, R, C, block_rows, act):
    g = gen(M * 1000 + R + C)
    # magnitudes over many binades, a block of zeros
    x = torch.randn((M, R, C), generator=g) * torch.exp2(torch.randint(-9, 4, (M, R, C), generator=g).float())
    x[0, 0, :128] = 0
    x = x.to(ref.TORCH[act])
    codes, scales = quantize(x, act, block_rows)
    q, s = ref.quantize(x, block_rows)
    s = s.reshape(M * R, -1).t() if block_rows == 1 else s
    assert torch.equal(scales, s.float())  # one division, correctly rounded
    got = ref.code_values(codes)
    if act == "f32":
        # 448 x and the quotient are rounded to fp32 first: only a value within
        # those two half steps of a border between codes may go the other way
        m = ref._blocked(x.double(), block_rows).abs().amax(dim=(2, 4)).clamp_min(ref.FLOOR)
        full = m.repeat_interleave(block_rows, dim=1)[:, :R].repeat_interleave(B, dim=2)[:, :, :C]
        t = x.double() * 448 / full
        lo, hi = ref.e4m3(t * (1 - 2 * ref.U)), ref.e4m3(t * (1 + 2 * ref.U))
        assert torch.all((got == q) | (got == lo) | (got == hi))
    else:
        assert torch.equal(got, q)


@pytest.mark.parametrize("act", ["bf16", "f16", "f32"])
def test_quantize_every_border(act):
    """Every code, every value half way between two, and their neighbours, under several maxima."""
    codes = torch.arange(0, 0x7F, dtype=torch.uint8)
    v = ref.code_values(codes)
    half = (v[1:] + v[:-1]) / 2
    pts = torch.cat([v, half, half * (1 + 2.0**-9), half * (1 - 2.0**-9), -v, -half])
    rows = []
    for e in (0, 3, -9):
        for i in range(0, len(pts), 127):  # 127 points and the block's maximum
            row = torch.full((128,), 448.0, dtype=torch.float64)
            part = pts[i:i + 127]
            row[1:1 + len(part)] = part
            rows.append(row * 2.0**e)
    x = torch.stack(rows)[None].to(ref.TORCH[act])
    got, scales = quantize(x, act, 1)
    q, s = ref.quantize(x, 1)
    assert torch.equal(ref.code_values(got), q)
    assert torch.equal(scales, s[0].t().float())


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_special_values(block_rows):
    x = torch.randn((1, 4, 256), generator=gen(3))
    x[0, 0, 5] = NAN
    x[0, 1, 200] = INF
    x[0, 2, :128] = 1e-40          # subnormal: the scale's floor
    x[0, 3, 128:] = 3.0e38         # the largest binade
    codes, scales = quantize(x, "f32", 1)
    got = codes[0].view(torch.float8_e4m3fn).float()
    assert torch.isnan(got[0, 5]) and torch.isfinite(got[0, :5]).all() and torch.isfinite(got[0, 6:]).all()
    assert scales[1, 1] == INF and torch.isnan(got[1, 200])
    assert (got[1, 128:200] == 0).all() and (got[1, 201:] == 0).all()
    assert scales[0, 2] == 2.0**-126 and (got[2, :128] == 2.0**-7).all()  # 1e-40 / 2^-126 = 0.0085
    assert (got[3, 128:] == 448).all()
    # a block of 128 rows meets them all at once
    codes, scales = quantize(x, "f32", 128)
    assert scales[0, 0, 1] == INF


def test_quantize_nothing():
    x = torch.empty((0, 4, 32), device=DEV)
    codes, scales = torch.empty(16, dtype=torch.uint8, device=DEV), torch.full((4,), 7.0, device=DEV)
    moe.moe_fp8_quantize(0, 4, 32, codes, 0, 1, codes, scales)
    moe.moe_fp8_quantize(3, 0, 32, codes, 0, 128, codes, scales)
    torch.cuda.synchronize()
    assert (scales == 7).all()


@pytest.mark.parametrize("M,N,K", [(1, 16, 16), (2, 144, 272), (3, 128, 400), (1, 400, 16)])
def test_transpose(M, N, K):
    g = gen(N + K)
    w = torch.randint(0, 256, (M, N, K), generator=g, dtype=torch.uint8)
    s = torch.rand((M, ref.nb(N), ref.nb(K)), generator=g)
    wt = torch.zeros((M, K, N), dtype=torch.uint8, device=DEV)
    st = torch.zeros((M, ref.nb(K), ref.nb(N)), device=DEV)
    moe.moe_fp8_transpose(M, N, K, w.to(DEV), s.to(DEV), wt, st)
    torch.cuda.synchronize()
    assert torch.equal(wt.cpu(), w.transpose(1, 2).contiguous())
    assert torch.equal(st.cpu(), s.transpose(1, 2).contiguous())


def groups(g, rows, E, kind):
    """Offsets of E experts over `rows` rows."""
    if kind == "one":  # all rows at one expert
        return torch.tensor([0] * (E // 2 + 1) + [rows] * (E - E // 2), dtype=torch.int32)
    if kind == "tail":  # rows behind the last expert's
        return torch.linspace(0, max(rows - 5, 0), E + 1).to(torch.int32)
    cut = torch.randint(0, rows + 1, (E - 1,), generator=g).sort()[0]
    return torch.cat([torch.tensor([0]), cut, torch.tensor([rows])]).to(torch.int32)


# rows, N, K, E, offsets, gathered, out
PRODUCT = [
    # few workgroups or few rows per expert: the decode kernel
    (1, 16, 16, 1, None, False, "f32"),
    (1, 2048, 2048, 1, None, False, "bf16"),
    (8, 1536, 2048, 128, "random", True, "bf16"),
    (17, 48, 144, 3, "random", True, "f16"),
    (33, 272, 528, 5, "tail", False, "f32"),
    (100, 80, 1040, 7, "one", True, "f32"),
    (64, 528, 400, 4, "random", False, "bf16"),      # two waves along the reduction
    (200, 272, 272, 4, "random", True, "f32"),
    (300, 784, 1168, 3, "random", True, "f32"),
    (37, 64, 4096, 600, "random", False, "f32"),     # more experts than rows, long reduction
    # 64 rows a tile
    (2100, 784, 1168, 3, "random", True, "f32"),     # column and reduction tails
    (2100, 784, 1168, 3, "tail", True, "bf16"),
    (2000, 1040, 528, 50, "random", False, "f16"),
    (5000, 1040, 16, 7, "one", True, "f32"),
    # 128 rows a tile
    (4100, 2832, 400, 3, "random", True, "bf16"),
    (4200, 2832, 128, 1, None, False, "f16"),
    (4300, 2832, 144, 20, "tail", False, "bf16"),
    # 256 rows a tile
    (8229, 4112, 272, 1, None, False, "bf16"),
    (9000, 4096, 256, 2, "tail", True, "f16"),
]


def product_case(rows, N, K, E, kind, gathered, seed):
    g = gen(seed)
    a_rows = max(3, rows // 2) if gathered else rows + 2
    x = torch.randn((1, a_rows, K), generator=g)
    q, s = ref.quantize(x, 1)
    a = q[0].float().to(torch.float8_e4m3fn).view(torch.uint8).contiguous()
    sa = s[0].t().float().contiguous()
    w, sw = make_weights(g, E, N, K)
    off = groups(g, rows, E, kind) if kind else None
    row_map = torch.randint(0, a_rows, (rows,), generator=g).to(torch.int32) if gathered else None
    return a, sa, w, sw, off, row_map


def run_product(case, rows, N, K, E, out):
    a, sa, w, sw, off, row_map = (None if t is None else t.to(DEV) for t in case)
    y = torch.full((rows, N), 77.0, dtype=ref.TORCH[out], device=DEV)
    moe.moe_fp8_matmul(rows, N, K, E, a.shape[0], a, sa, row_map, off, w, sw, y, DT[out])
    torch.cuda.synchronize()
    return y.cpu()


def check_product(case, y, rows, N, K, E, out):
    a, sa, w, sw, off, row_map = case
    rv, wv = ref.row_values(a, sa), ref.matrix_values(w, sw)
    rv = rv[row_map.long()] if row_map is not None else rv[:rows]
    off = off.tolist() if off is not None else [0, rows]
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            at = torch.arange(lo, hi)
            if rows > 1000:  # a sample: the ends, the rows around each tile's border, some others
                m = at - lo
                at = at[(m < 2) | (at >= hi - 2) | (m % 256 >= 255) | (m % 64 == 0) & (m < 700) | (m % 97 == 5)]
            c, r = ref.product(rv[at], wv[e])
            if out != "f32":
                r = r + ref.dropped(rv[at], wv[e])
            bound = r + torch.finfo(ref.TORCH[out]).eps / 2 * (c.abs() + r)
            bound = bound + (2.0**-25 if out == "f16" else 1e-38)  # half a step of fp16's subnormals
            assert torch.all((y[at].double() - c).abs() <= bound), f"expert {e}"
            assert torch.isfinite(y[lo:hi]).all()
    assert (y[off[E]:] == 77).all()  # rows of no expert


@pytest.mark.parametrize("rows,N,K,E,kind,gathered,out", PRODUCT)
def test_product(rows, N, K, E, kind, gathered, out):
    print(f"[case] product {rows} {N} {K} {E} {kind}", flush=True)
    case = product_case(rows, N, K, E, kind, gathered, rows + N + K)
    y = run_product(case, rows, N, K, E, out)
    check_product(case, y, rows, N, K, E, out)
    assert torch.equal(y.view(torch.uint8), run_product(case, rows, N, K, E, out).view(torch.uint8))


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("E,N,K", [(60, 2320, 272), (36, 3088, 144), (20, 3600, 400)])  # 32, 48 and 64 rows a small tile
def test_product_unequal_experts(E, N, K, out):
    """Experts on both sides of every tile's border side by side, some without rows."""
    counts = [95, 0, 96, 1, 97, 300, 17, 128, 129, 64, 0, 255, 2, 33]
    counts += [1] * (E - len(counts))
    off = torch.tensor([0] + counts).cumsum(0).to(torch.int32)
    rows = int(off[-1]) + 5  # the last five belong to no expert
    case = list(product_case(rows, N, K, E, "random", True, E))
    case[4] = off
    y = run_product(case, rows, N, K, E, out)
    check_product(case, y, rows, N, K, E, out)
    assert torch.equal(y.view(torch.uint8), run_product(case, rows, N, K, E, out).view(torch.uint8))


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("rows,N", [(20, 64), (700, 64), (5000, 1040), (9000, 2064), (17000, 4112)])
def test_product_bad_tables(rows, N, out):
    """A map entry outside the rows gives zeros; wild offsets stay inside the output (every kernel)."""
    K, E = 272, 4
    case = list(product_case(rows, N, K, E, "random", True, rows))
    row_map = case[5]
    bad = torch.arange(0, rows, 7)
    row_map[bad] = torch.tensor([-1, 1 << 30, case[0].shape[0]], dtype=torch.int32).repeat(rows)[:len(bad)]
    y = run_product(case, rows, N, K, E, out)
    assert (y[bad] == 0).all()
    case[4] = torch.tensor([-5, 3, rows + 9, 1 << 30, -7], dtype=torch.int32)
    y = run_product(case, rows, N, K, E, out)  # ranges [0, 3), [3, rows), [rows, rows), [rows, rows)
    case[4] = torch.tensor([0, 3, rows, rows, rows], dtype=torch.int32)
    assert torch.equal(y, run_product(case, rows, N, K, E, out))


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("rows,N", [(20, 64), (130, 64), (700, 64), (5000, 1040), (9000, 2064), (17000, 4112)])
def test_product_rows_outside_stay_zero_beside_nans(rows, N, out):
    """A row of zeros stays one where the weights or their scales hold NaNs and infinities."""
    K, E = 272, 4
    case = list(product_case(rows, N, K, E, "random", True, rows))
    case[5][::5] = -1
    case[2][:, 3, 7] = 0x7F
    case[3][:, -1, 1] = INF
    y = run_product(case, rows, N, K, E, out)
    assert (y[::5] == 0).all()
    assert torch.isnan(y[1::5][:, 3]).all()


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("rows,N,E", [(6, 48, 1), (150, 48, 2), (5000, 1040, 2), (9000, 2064, 2), (17000, 4112, 1)])
def test_product_padding_is_not_read(rows, N, E, out):
    """NaN codes outside a row's reduction (the next row's, a neighbour expert's) do not reach it."""
    K = 144  # 16 codes past one block
    case = product_case(rows, N, K, E, "random" if E > 1 else None, False, 5)
    a, w = case[0], case[2]
    y0 = run_product(case, rows, N, K, E, out)
    w[:, 7, :] = 0x7F
    a[rows // 2, :] = 0x7F
    y1 = run_product(case, rows, N, K, E, out)
    keep_n = torch.arange(N) != 7
    keep_r = torch.arange(rows) != rows // 2
    assert torch.equal(y1[keep_r][:, keep_n], y0[keep_r][:, keep_n])
    assert torch.isnan(y1[rows // 2]).all() and torch.isnan(y1[:, 7]).all()


@pytest.mark.parametrize("rows", [5, 90, 260])
def test_product_gradient(rows):
    """dL/da of the product is the product with the transposed weights, checked against the formula
    and, since the product is linear in a, against differences of two products."""
    N, K, E = 144, 272, 3
    g = gen(rows)
    case = product_case(rows, N, K, E, "random", False, rows)
    w, sw, off = case[2].to(DEV), case[3].to(DEV), case[4].to(DEV)
    dy = torch.randn((1, rows, N), generator=g)
    dq, ds = (t.to(DEV) for t in quantize(dy, "f32", 1))
    wt = torch.empty((E, K, N), dtype=torch.uint8, device=DEV)
    st = torch.empty((E, ref.nb(K), ref.nb(N)), device=DEV)
    moe.moe_fp8_transpose(E, N, K, w, sw, wt, st)
    da = torch.empty((rows, K), device=DEV)
    moe.moe_fp8_matmul(rows, K, N, E, rows, dq[0], ds, None, off, wt, st, da, moe.MOE_DT_F32)
    torch.cuda.synchronize()
    da = da.cpu().double()
    dv, wv = ref.row_values(dq[0].cpu(), ds.cpu()), ref.matrix_values(case[2], case[3])
    o = off.tolist()
    # one code of a row moves: y moves by w, the loss <dy, y> by da times the move
    a2 = case[0].clone()
    j = 130
    a2[:, j] = 0x38  # the code of 1
    y1 = run_product(case, rows, N, K, E, "f32").double()
    y2 = run_product((a2,) + case[1:], rows, N, K, E, "f32").double()
    move = ref.row_values(a2, case[1])[:rows, j] - ref.row_values(case[0], case[1])[:rows, j]
    for e in range(E):
        lo, hi = o[e], o[e + 1]
        if hi == lo:
            continue
        c, r = ref.product(dv[lo:hi], wv[e].t())
        assert torch.all((da[lo:hi] - c).abs() <= r + ref.U * (c.abs() + r))
        diff = (dv[lo:hi] * (y2[lo:hi] - y1[lo:hi])).sum(dim=1)
        rows_v = ref.row_values(case[0], case[1])[lo:hi].abs() + ref.row_values(a2, case[1])[lo:hi].abs()
        tol = 2 * (ref.product_radius(K) + ref.U) * (dv[lo:hi].abs() * (rows_v @ wv[e].abs().t())).sum(dim=1)
        tol = tol + r[:, j] * move[lo:hi].abs()
        assert torch.all((diff - da[lo:hi, j] * move[lo:hi]).abs() <= tol)


# T, D, F, E, k, S, act, fused, glu, round
LAYERS = [
    (1, 64, 64, 4, 2, 0, "bf16", False, "swiglu", False),
    (1, 2048, 768, 16, 8, 0, "bf16", True, "swiglu", True),
    (5, 272, 144, 8, 3, 1, "f16", False, "geglu", False),
    (16, 64, 128, 8, 2, 0, "f32", True, "swiglu", False),
    (40, 144, 400, 6, 2, 2, "bf16", True, "geglu", True),     # up rows start inside a scale block
    (70, 528, 272, 3, 2, 1, "f16", True, "swiglu", True),     # 64-row tiles
    (300, 256, 144, 3, 2, 0, "bf16", False, "swiglu", False), # 128-row tiles
    (400, 144, 336, 2, 2, 1, "f32", True, "geglu", False),
]


def layer(T, D, F, E, k, S, act, fused, glu, rnd, seed):
    g = gen(seed)
    M = E + S
    desc = moe.make_desc(D, F, E, k, S, act=act, wfmt="fp8", gate_up_fused=fused, glu_round=rnd, activation=glu)
    gu, down = make_weights(g, M, 2 * F, D), make_weights(g, M, D, F)
    if not fused:
        gate, up = make_weights(g, M, F, D), make_weights(g, M, F, D)
    parts = {"gate_up": gu} if fused else {"gate": gate, "up": up}
    parts["down"] = down
    w_router = (torch.randn((D, E), generator=g) * D**-0.5).to(ref.TORCH[act])
    bias = torch.randn(E, generator=g)
    x = torch.randn((T, D), generator=g).to(ref.TORCH[act])
    table = moe.DeviceWeights(w_router.to(DEV), bias.to(DEV),
                              {n: {"w": c.to(DEV), "scales": s.to(DEV)} for n, (c, s) in parts.items()})
    return desc, parts, table, x


def expert_matrices(parts, fused, F):
    down = ref.matrix_values(*parts["down"])
    if fused:
        gu = ref.matrix_values(*parts["gate_up"])
        return gu[:, :F], gu[:, F:], down
    return ref.matrix_values(*parts["gate"]), ref.matrix_values(*parts["up"]), down


def expert_rows(x, e, mats, glu, rnd):
    """An expert's outputs for rows x in 64 bits, with their radius."""
    gate, up, down = mats
    v = ref.quantized_rows((x.double(), torch.zeros_like(x, dtype=torch.float64)), x.dtype != torch.float32)
    h = ref.gated(ref.product_of(v, gate[e]), ref.product_of(v, up[e]), glu == "geglu", rnd)
    return ref.product_of(ref.quantized_rows(h, rnd is not None), down[e])


@pytest.mark.parametrize("T,D,F,E,k,S,act,fused,glu,rnd", LAYERS)
def test_layer(T, D, F, E, k, S, act, fused, glu, rnd):
    """moe_forward, and the same steps called one by one, of an fp8 layer."""
    print(f"[case] fp8 layer {T} {D} {F} {E}", flush=True)
    desc, parts, table, x = layer(T, D, F, E, k, S, act, fused, glu, rnd, T + D)
    N = T * k
    ws = torch.empty(moe.moe_workspace_size(desc, T), dtype=torch.uint8, device=DEV)
    y = torch.empty((T, D), device=DEV)
    idx = torch.empty((T, k), dtype=torch.int32, device=DEV)
    wt = torch.empty((T, k), device=DEV)
    xd = x.to(DEV)
    moe.moe_forward(desc, T, xd, table, y, moe.MOE_DT_F32, idx, wt, ws)
    ints = lambda n: torch.empty(n, dtype=torch.int32, device=DEV)  # noqa: E731
    order, inv, row_map, off, tiles = ints(N), ints(N), ints(N), ints(E + 1), ints(E + 1)
    rows = torch.empty((N + S * T, D), device=DEV)
    y2 = torch.empty_like(y)
    ws2 = torch.full_like(ws, 0xFF)  # stale workspace bytes (NaN patterns)
    moe.moe_dispatch(desc, T, idx, 64, order, inv, row_map, off, tiles, ws2)
    moe.moe_expert_ffn(desc, T, xd, row_map, off, table, rows, ws2)
    moe.moe_combine(desc, T, rows, inv, wt, y2, moe.MOE_DT_F32)
    torch.cuda.synchronize()
    assert torch.equal(y, y2)

    mats = expert_matrices(parts, fused, F)
    rnd_act = act if rnd else None
    c, r = torch.zeros((T, D), dtype=torch.float64), torch.zeros((T, D), dtype=torch.float64)
    total = torch.zeros_like(c)
    idx, wt, rows = idx.cpu(), wt.cpu().double(), rows.cpu().double()
    inv = inv.cpu().view(T, k)
    for e in range(E + S):
        if e < E:
            t, j = torch.nonzero(idx == e, as_tuple=True)
            at, cw = inv[t, j].long(), wt[t, j][:, None]
        else:
            t = torch.arange(T)
            at, cw = N + (e - E) * T + t, torch.ones((T, 1), dtype=torch.float64)
        if not len(t):
            continue
        yc, yr = expert_rows(x[t], e, mats, glu, rnd_act)
        assert torch.all((rows[at] - yc).abs() <= yr + ref.U * (yc.abs() + yr)), f"expert {e}"
        c.index_add_(0, t, cw * yc)
        r.index_add_(0, t, cw * yr)
        total.index_add_(0, t, cw * (yc.abs() + yr))
    # the combine: k + S products and sums in fp32
    assert torch.all((y.cpu().double() - c).abs() <= r + (k + S + 1) * 2 * ref.U * total)
    # the bound is no empty one: it stays below the layer's own scale (every rounding at its worst, all of
    # one sign: a tenth of h near a border between two bf16 values in the longest rounded case)
    assert r.median() < (1 if rnd else 0.05) * c.abs().mean()


def test_layer_forms_agree():
    """The timed, the allocation-free and a captured, replayed forward give moe_forward's bits."""
    T, D, F, E, k, S = 40, 144, 400, 6, 2, 2
    desc, _, table, x = layer(T, D, F, E, k, S, "bf16", True, "swiglu", False, 9)
    xd = x.to(DEV)
    ws = torch.empty(moe.moe_workspace_size(desc, T), dtype=torch.uint8, device=DEV)
    out = lambda: torch.full((T, D), NAN, device=DEV)  # noqa: E731
    y = out()
    moe.moe_forward(desc, T, xd, table, y, moe.MOE_DT_F32, None, None, ws)
    n = out()
    moe.moe_forward_noalloc(desc, T, xd, table, n, moe.MOE_DT_F32, None, None)
    torch.cuda.synchronize()
    assert torch.equal(y, n)
    cap, graph, z = torch.cuda.Stream(), torch.cuda.CUDAGraph(), out()
    ws3 = torch.empty_like(ws)
    with torch.cuda.graph(graph, stream=cap):
        moe.moe_forward(desc, T, xd, table, z, moe.MOE_DT_F32, None, None, ws3, cap)
    for _ in range(3):
        z.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, z)
        moe.moe_forward(desc, T, xd, table, n, moe.MOE_DT_F32, None, None, ws)
        torch.cuda.synchronize()
        assert torch.equal(y, n)


@pytest.mark.parametrize("T,D,F,E,k,S,act,fused,glu,renorm", [
    (3, 64, 64, 4, 2, 1, "f32", True, "swiglu", True),
    (20, 144, 80, 5, 3, 0, "bf16", False, "geglu", False),
])
def test_layer_backward(T, D, F, E, k, S, act, fused, glu, renorm):
    """dx against autograd of the layer's formula on the weights' values (activations unrounded), in 64 bits."""
    desc, parts, table, x = layer(T, D, F, E, k, S, act, fused, glu, False, 11)
    desc.renormalize = int(renorm)
    dy = torch.randn((T, D), generator=gen(12))
    ws = torch.empty(moe.moe_backward_workspace_size(desc, T), dtype=torch.uint8, device=DEV)
    dx = torch.full((T, D), NAN, device=DEV)
    moe.moe_backward(desc, T, x.to(DEV), table, dy.to(DEV), dx, ws)
    idx = torch.empty((T, k), dtype=torch.int32, device=DEV)
    wt = torch.empty((T, k), device=DEV)
    ws2 = torch.empty(moe.moe_workspace_size(desc, T), dtype=torch.uint8, device=DEV)
    moe.moe_route(desc, T, x.to(DEV), table.w_router, table.router_bias, idx, wt, ws2)
    torch.cuda.synchronize()
    idx = idx.cpu().long()
    gate, up, down = expert_matrices(parts, fused, F)
    xv = x.double().requires_grad_(True)
    logits = xv @ table.w_router.cpu().double() + table.router_bias.cpu().double()
    p = torch.softmax(logits, dim=1).gather(1, idx)
    p = p / p.sum(dim=1, keepdim=True) if renorm else p
    act_f = (lambda v: 0.5 * v * (1 + torch.tanh(0.7978845608028654 * (v + 0.044715 * v**3)))) if glu == "geglu" \
        else (lambda v: v * torch.sigmoid(v))
    ffn = lambda rows, e: (act_f(rows @ gate[e].t()) * (rows @ up[e].t())) @ down[e].t()  # noqa: E731
    y = torch.zeros((T, D), dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            y[t] = y[t] + p[t, j] * ffn(xv[t:t + 1], int(idx[t, j]))[0]
        for s in range(S):
            y[t] = y[t] + ffn(xv[t:t + 1], E + s)[0]
    (want,) = torch.autograd.grad(y, xv, dy.double())
    # fp32 chains of at most D + 2 F + E products in a row, relative to the largest gradient
    err = (dx.cpu().double() - want).abs().max() / want.abs().max()
    assert err <= (D + 2 * F + E) * 2 * ref.U


def test_other_stream_and_concurrent_workspaces():
    """Two layers in flight on two streams, each with its own workspace."""
    T, D, F, E, k = 200, 256, 272, 3, 2
    desc, _, table, x = layer(T, D, F, E, k, 0, "bf16", False, "swiglu", False, 21)
    xs = [x.to(DEV), (x * 1.5).to(DEV)]
    ws = [torch.empty(moe.moe_workspace_size(desc, T), dtype=torch.uint8, device=DEV) for _ in range(2)]
    want, got = [], [torch.empty((T, D), device=DEV) for _ in range(2)]
    for i in range(2):
        y = torch.empty((T, D), device=DEV)
        moe.moe_forward(desc, T, xs[i], table, y, moe.MOE_DT_F32, None, None, ws[i])
        torch.cuda.synchronize()
        want.append(y)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for i in range(2):
            moe.moe_forward(desc, T, xs[i], table, got[i], moe.MOE_DT_F32, None, None, ws[i], streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(want[i], got[i])


def test_work_of_many_experts_and_rows():
    """1024 experts with one to three rows each: the table search over the whole wave."""
    E, N, K = 1024, 32, 64
    g = gen(8)
    counts = torch.randint(0, 4, (E,), generator=g)
    off = torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)]).to(torch.int32)
    rows = int(off[-1])
    case = list(product_case(rows, N, K, E, "random", False, 8))
    case[4] = off
    y = run_product(case, rows, N, K, E, "f32")
    check_product(case, y, rows, N, K, E, "f32")
    assert np.isfinite(y.numpy()).all()


def test_weights_past_32_bits():
    """The last of 520 matrices, 4 GiB into the codes: quantised, transposed and multiplied to the same
    bits as the first one, which holds the same values (every kernel of the grouped product)."""
    E, N, K = 520, 4096, 2048
    x = torch.randn((E, N, K), device=DEV, dtype=torch.bfloat16)
    x[0] = x[E - 1]
    w = torch.empty((E, N, K), dtype=torch.uint8, device=DEV)
    sw = torch.empty((E, ref.nb(N), ref.nb(K)), device=DEV)
    moe.moe_fp8_quantize(E, N, K, x, DT["bf16"], 128, w, sw)
    c, s = quantize(x[E - 1:].cpu(), "bf16", 128)
    assert torch.equal(w[E - 1].cpu(), c[0]) and torch.equal(sw[E - 1].cpu(), s[0])
    del x
    wt, st = torch.empty((E, K, N), dtype=torch.uint8, device=DEV), torch.empty((E, ref.nb(K), ref.nb(N)), device=DEV)
    moe.moe_fp8_transpose(E, N, K, w, sw, wt, st)
    assert torch.equal(wt[E - 1], w[E - 1].t()) and torch.equal(st[E - 1], sw[E - 1].t())
    del wt
    a_rows = 97
    a, sa = quantize(torch.randn((1, a_rows, K), generator=gen(2)).bfloat16(), "bf16", 1)
    rv, wv = ref.row_values(a[0], sa)[:16], ref.matrix_values(w[E - 1:].cpu(), sw[E - 1:].cpu())[0]
    a, sa = a[0].to(DEV), sa.to(DEV)
    for rows, out in ((100, "f32"), (9000, "f32"), (18000, "bf16"), (24000, "bf16"), (52000, "bf16")):
        print(f"[case] {rows} rows {out}", flush=True)
        row_map = (torch.arange(rows) % a_rows).to(torch.int32).to(DEV)
        y = [torch.empty((rows, N), dtype=ref.TORCH[out], device=DEV) for _ in range(2)]
        for i, e in enumerate((0, E - 1)):
            off = torch.full((E + 1,), rows, dtype=torch.int32)
            off[:e + 1] = 0
            moe.moe_fp8_matmul(rows, N, K, E, a_rows, a, sa, row_map, off.to(DEV), w, sw, y[i], DT[out])
        assert torch.equal(y[0], y[1])
        c, r = ref.product(rv, wv)
        if out != "f32":
            r = r + ref.dropped(rv, wv)
        bound = r + torch.finfo(ref.TORCH[out]).eps / 2 * (c.abs() + r) + 1e-38
        assert torch.all((y[1][:16].cpu().double() - c).abs() <= bound)


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_results_past_32_bits(out):
    """530000 x 4112 results: the last rows, past 2^31 of them, repeat the first ones' bits."""
    rows, N, K, a_rows = 530000, 4112, 144, 1000
    a, sa, w, sw = (t.to(DEV) for t in product_case(a_rows - 2, N, K, 1, None, False, 3)[:4])
    row_map = (torch.arange(rows) % a_rows).to(torch.int32).to(DEV)
    y = torch.empty((rows, N), dtype=ref.TORCH[out], device=DEV)
    moe.moe_fp8_matmul(rows, N, K, 1, a_rows, a, sa, row_map, None, w, sw, y, DT[out])
    assert torch.equal(y[529000:], y[:1000])
    x = y[528900:].float()  # and rows whose elements lie past 2^31, quantised
    del y
    big = torch.zeros((rows, N), dtype=torch.bfloat16, device=DEV)
    big[528900:] = x.bfloat16()
    codes = torch.empty((rows, N), dtype=torch.uint8, device=DEV)
    scales = torch.empty((ref.nb(N), rows), device=DEV)
    moe.moe_fp8_quantize(1, rows, N, big, DT["bf16"], 1, codes, scales)
    c, s = quantize(big[528900:][None].cpu(), "bf16", 1)
    assert torch.equal(codes[528900:].cpu(), c[0]) and torch.equal(scales[:, 528900:].cpu(), s)

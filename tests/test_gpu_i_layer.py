"""The 4-bit expert layer on the GPU against the float64 oracle: quantization bit for bit, products, the
gate/up activation, routing with gate weights, combination.

Tolerances. A stored rounding is off by half a step of the type (bf16 2^-8 relative, fp32 2^-24). The
products' sums are float32 on the tensor cores: 64 columns are added to the accumulator at a time with at
most one truncation of 2^-23 of the larger operand each, so K columns give at most (K / 64 + 64) 2^-23 of
the sum of the terms' magnitudes |x| |w|^T.
"""
import ctypes

import numpy as np
import pytest
import torch

import oracle.layer_oracle as O
from helpers import to64
from post_quantization_expert_b200 import clha as L

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FMT = {"e8m0_32": L.FP4_E8M0_32, "e4m3_16": L.FP4_E4M3_16}
FMTS = sorted(FMT)
BF16, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def buffers(fmt, rows, d):
    """Code and scale buffers holding a pattern, so that what is not written shows."""
    return (torch.full((rows, d // 2), 0xA5, dtype=torch.uint8, device=DEV),
            torch.full((L.clha_fp4_scale_bytes(FMT[fmt], rows, d),), 0xA5, dtype=torch.uint8, device=DEV))


def quantize(ctx, x, fmt, g=None):
    rows, d = x.shape
    codes, scales = buffers(fmt, rows, d)
    L.clha_fp4_quantize(ctx, x, rows, d, FMT[fmt], codes, scales, tensor_scale=g)
    return codes, scales


def route(n, E, k, seed):
    """ids, seg, perm (torch, host) as clha_gather lays them out, some experts without tokens."""
    r = np.random.default_rng(seed)
    p = r.random((n, E)) * np.where(np.arange(E) % 5 == 3, 1e-3, 1.0)[None]
    ids = np.argsort(-p, 1, kind="stable")[:, :k].astype(np.int32)
    counts = np.bincount(ids.ravel(), minlength=E)
    starts = np.concatenate([[0], np.cumsum((counts + 127) // 128 * 128)])
    P = n * k + 128 * E
    perm = np.full(P, -1, np.int32)
    for e in range(E):
        perm[starts[e]:starts[e] + counts[e]] = np.nonzero((ids == e).any(1))[0]
    return ids, np.concatenate([starts, counts]).astype(np.int64), perm


# ------------------------------------------------------------------ quantization
def check_quantized(codes, scales, x64, fmt, g=1.0, rows=None):
    want_c, want_s = O.fp4_quantize(x64, fmt, g)
    np.testing.assert_array_equal(scales.cpu().numpy(), O.tile_scales(want_s))
    got = codes.cpu().numpy()
    np.testing.assert_array_equal(got, O.pack_codes4(want_c))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("rows,d", [(1, 128), (33, 384), (129, 256), (500, 1152)])
def test_quantize_bit_exact(ctx, fmt, dtype, scaled, rows, d):
    x = (torch.randn((rows, d), generator=gen(rows + d)) * torch.logspace(-3, 3, d)[None]).to(dtype)
    x[0, :64] = 0
    g = (x.float().abs().max() / 2688).view(1) if scaled else None
    codes, scales = quantize(ctx, x.to(DEV), fmt, None if g is None else g.to(DEV))
    check_quantized(codes, scales, to64(x), fmt, 1.0 if g is None else float(g))
    L.clha_check(ctx)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("g", [None, 1.0, 0.37, 3.1e-5, 2.0 ** -130, 2.9e38])
def test_quantize_borders(ctx, fmt, g):
    """Every border between codes, and the values one float32 step to either side of it, under scales whose
    quotients do not come out even; tiny, huge and subnormal numbers; signed zeros."""
    r = np.random.default_rng(7)
    levels = np.concatenate([O.E2M1, (O.E2M1[1:] + O.E2M1[:-1]) / 2])
    unit = 1.0 if g is None else np.float64(np.float32(g))
    rows = []
    for i in range(64):
        s = 2.0 ** r.integers(-3, 3) * (1.0 if fmt == "e8m0_32" else 1 + r.integers(0, 8) / 8)
        row = r.choice(levels, 256) * r.choice([-1, 1], 256) * s * unit
        row[::16] = 6 * s * unit                       # pins the block's scale to s
        with np.errstate(over="ignore"):
            row = row.astype(np.float32)
        step = r.integers(-1, 2, 256)
        row = np.where(step < 0, np.nextafter(row, np.float32(0)), np.where(step > 0, np.nextafter(row, np.float32(np.inf) * np.sign(row + 1e-45)), row))
        rows.append(np.where(np.isfinite(row), row, 0))
    x = np.array(rows, np.float32)
    if g is None or g == 1.0:
        x[3] = np.float32(1e-45) * r.integers(-5, 6, 256)
        x[4] = np.float32(3.4e38) * r.choice([-1, 1], 256)
        x[5] = -0.0
        x[6] = np.float32(2.0 ** -126) * r.random(256)
    codes, scales = quantize(ctx, torch.from_numpy(x).to(DEV), fmt, None if g is None else torch.tensor([g], device=DEV))
    check_quantized(codes, scales, x.astype(np.float64), fmt, unit)
    L.clha_check(ctx)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize_every_exponent(ctx, fmt, dtype):
    """A row for each exponent of the type, subnormal ones among them, with values down to far below the largest."""
    r = np.random.default_rng(3)
    e = np.arange(-149 if dtype == F32 else -133, 128)
    x = np.ldexp(1 + r.random((len(e), 256)), e[:, None] - r.integers(0, 9, (len(e), 256))) * r.choice([-1, 1], (len(e), 256))
    x = torch.from_numpy(np.clip(x, -3.3e38, 3.3e38)).to(dtype)
    codes, scales = quantize(ctx, x.to(DEV), fmt)
    check_quantized(codes, scales, to64(x), fmt)
    L.clha_check(ctx)


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_routed_rows(ctx, fmt):
    """Rows through a permutation, segments with padding and empty experts, rows behind the last segment."""
    n, E, k, d = 300, 10, 3, 384
    ids, seg, perm = route(n, E, k, 1)
    P, end = len(perm), int(seg[E])
    assert end < P
    x = torch.randn((n, d), generator=gen(2)).to(BF16)
    codes, scales = buffers(fmt, P, d)
    L.clha_fp4_quantize(ctx, x.to(DEV), n, d, FMT[fmt], codes, scales, perm=torch.from_numpy(perm).to(DEV), rows=P,
                        seg=torch.from_numpy(seg).to(DEV), E=E)
    x64 = np.where((perm >= 0)[:, None], to64(x)[np.maximum(perm, 0)], 0.0)
    want_c, want_s = O.fp4_quantize(x64[:end], fmt)
    np.testing.assert_array_equal(codes[:end].cpu().numpy(), O.pack_codes4(want_c))
    np.testing.assert_array_equal(scales.cpu().numpy()[:end * d // O.BLOCK[fmt]], O.tile_scales(want_s))
    assert (codes[end:] == 0xA5).all() and (scales[end * d // O.BLOCK[fmt]:] == 0xA5).all()
    L.clha_check(ctx)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,E,k,d,dtype", [(9000, 24, 3, 4096, BF16), (3300, 300, 4, 2048, F32), (7000, 64, 2, 1024, F32)])
def test_quantize_routed_rows_of_a_large_x(ctx, fmt, n, E, k, d, dtype):
    """X of several tens of megabytes: the row tiles are taken in another order, with the same result."""
    ids, seg, perm = route(n, E, k, 5)
    P, end = len(perm), int(seg[E])
    x = torch.randn((n, d), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).to(dtype)
    codes, scales = buffers(fmt, P, d)
    L.clha_fp4_quantize(ctx, x, n, d, FMT[fmt], codes, scales, perm=torch.from_numpy(perm).to(DEV), rows=P,
                        seg=torch.from_numpy(seg).to(DEV), E=E)
    p = torch.from_numpy(perm[:end]).to(DEV)
    xp = torch.where((p >= 0)[:, None], x[p.clamp_min(0).long()], torch.zeros((), dtype=dtype, device=DEV))
    want_c, want_s = quantize(ctx, xp, fmt)                # rows as they lie, held to the oracle above
    assert torch.equal(codes[:end], want_c) and torch.equal(scales[:want_s.numel()], want_s)
    assert (codes[end:] == 0xA5).all() and (scales[want_s.numel():] == 0xA5).all()
    L.clha_check(ctx)


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_only_the_first_routed_rows(ctx, fmt):
    """Fewer rows than the segments hold, of an X that is large enough for another order of the tiles."""
    n, E, k, d = 9000, 24, 3, 4096
    ids, seg, perm = route(n, E, k, 5)
    rows = 128 * 100 + 37
    assert n < rows < int(seg[E])
    x = torch.randn((n, d), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).to(BF16)
    codes, scales = buffers(fmt, rows + 200, d)
    L.clha_fp4_quantize(ctx, x, n, d, FMT[fmt], codes, scales, perm=torch.from_numpy(perm).to(DEV), rows=rows,
                        seg=torch.from_numpy(seg).to(DEV), E=E)
    p = torch.from_numpy(perm[:rows]).to(DEV)
    xp = torch.where((p >= 0)[:, None], x[p.clamp_min(0).long()], torch.zeros((), dtype=BF16, device=DEV))
    want_c, want_s = quantize(ctx, xp, fmt)
    assert torch.equal(codes[:rows], want_c) and torch.equal(scales[:want_s.numel()], want_s)
    assert (codes[rows:] == 0xA5).all() and (scales[want_s.numel():] == 0xA5).all()
    L.clha_check(ctx)


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_batch_of_scales_and_dequantize(ctx, fmt):
    """Three matrices with a scale each: clha_fp4_tensor_scale, the codes under them, and their values."""
    B, rows, d = 3, 130, 256
    x = torch.randn((B, rows, d), generator=gen(3)) * torch.tensor([1e-4, 1.0, 300.0])[:, None, None]
    x[1] = 0
    xd = x.to(DEV)
    g = torch.empty(B, device=DEV)
    L.clha_fp4_tensor_scale(ctx, xd, B, rows, d, FMT[fmt], g)
    top = x.abs().amax((1, 2)).numpy()
    want_g = np.where(top > 0, top / np.float32(6.0 if fmt == "e8m0_32" else 2688.0), np.float32(1))
    np.testing.assert_array_equal(g.cpu().numpy(), want_g)
    codes, scales = buffers(fmt, B * rows, d)
    L.clha_fp4_quantize(ctx, xd.view(-1, d), B * rows, d, FMT[fmt], codes, scales, tensor_scale=g)
    per_row = np.repeat(want_g.astype(np.float64), rows)
    want_c, want_s = O.fp4_quantize(to64(x.view(-1, d)), fmt, per_row)
    np.testing.assert_array_equal(codes.cpu().numpy(), O.pack_codes4(want_c))
    np.testing.assert_array_equal(scales.cpu().numpy(), O.tile_scales(want_s))
    want = O.fp4_values(want_c, want_s, fmt, per_row)
    for dtype in (F32, BF16):
        v = torch.full((B * rows, d), 7.0, dtype=dtype, device=DEV)
        L.clha_fp4_dequantize(ctx, codes, scales, B * rows, d, FMT[fmt], v, tensor_scale=g)
        if dtype == F32:
            np.testing.assert_array_equal(v.cpu().numpy(), want.astype(np.float32))
        else:   # one rounding to bf16: nearest even of the exact value, by way of float64 bits
            assert torch.equal(v.cpu(), round_bf16(want))
    L.clha_check(ctx)


def round_bf16(x64):
    """Float64 -> bf16, nearest even, in one rounding."""
    m, e = np.frexp(x64)
    return torch.from_numpy(np.ldexp(np.rint(m * 256), e - 8)).to(BF16)


@pytest.mark.parametrize("fmt", FMTS)
def test_non_finite_blocks_are_reported(ctx, fmt):
    x = torch.randn((140, 256), generator=gen(4))
    x[131, 70] = float("nan")
    x[2, 5] = float("inf")
    codes, scales = quantize(ctx, x.to(DEV), fmt)
    with pytest.raises(L.ClhaError) as ei:
        L.clha_check(ctx)
    assert ei.value.status == L.ERR_NONFINITE
    v = torch.empty((140, 256), device=DEV)
    L.clha_fp4_dequantize(ctx, codes, scales, 140, 256, FMT[fmt], v)
    bad = torch.zeros((140, 256), dtype=torch.bool)
    B = O.BLOCK[fmt]
    bad[131, 70 // B * B:(70 // B + 1) * B] = True
    bad[2, :B] = True
    assert torch.equal(v.isnan().cpu(), bad)
    L.clha_check(ctx)


# ------------------------------------------------------------------ products
def operand(ctx, x, fmt, g=None):
    """(codes, scales, exact values) of x [R, d] (host); g float32 [B]: a scale for each equal share of the rows."""
    gd = None if g is None else g.to(DEV)
    codes, scales = quantize(ctx, x.to(DEV), fmt, gd)
    per_row = 1.0 if g is None else np.repeat(to64(g), x.shape[0] // len(g))
    c, s = O.fp4_quantize(to64(x), fmt, per_row)
    return codes, scales, O.fp4_values(c, s, fmt, per_row)


def check_product(got, want, mags, K, out):
    err = np.abs(to64(got) - want)
    tol = (K / 64 + 64) * 2.0 ** -23 * mags + np.abs(want) * (2.0 ** -8 if out == BF16 else 2.0 ** -24)
    assert (err <= tol + 1e-30).all(), (float((err - tol).max()), float(err.max()))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("n,K,N", [(1, 128, 128), (1, 2048, 256), (7, 384, 384), (128, 256, 128), (129, 640, 256),
                                   (300, 1152, 640), (64, 8192, 128),
                                   # many tiles: pairs of SMs, the last row tile and the last column block halves
                                   (2600, 640, 2176), (4999, 1152, 1024),
                                   # a long K over few tiles: clusters of 8 and 4 share it, three row tiles
                                   (300, 8192, 128), (70, 4224, 384), (32, 3968, 1024), (33, 2176, 128)])
def test_matmul(ctx, fmt, out, n, K, N):
    x = torch.randn((n, K), generator=gen(n + K)).to(BF16)
    w = (0.02 * torch.randn((N, K), generator=gen(N))).to(BF16)
    xq, xs, x64 = operand(ctx, x, fmt)
    wq, ws, w64 = operand(ctx, w, fmt)
    y = torch.full((n, N), 5.0, dtype=out, device=DEV)
    L.clha_fp4_matmul(ctx, FMT[fmt], xq, xs, n, K, wq, ws, N, y)
    check_product(y, x64 @ w64.T, np.abs(x64) @ np.abs(w64.T), K, out)
    L.clha_check(ctx)


def stacked(w, E):
    return w.view(E * w.shape[1], w.shape[2])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("n,E,k,K,N", [(300, 10, 3, 384, 256), (5, 16, 2, 512, 128), (1, 4, 1, 128, 384),
                                       (1500, 4, 2, 256, 640),
                                       # many tiles: pairs of SMs, segments with an odd number of 128-row tiles
                                       (3001, 10, 3, 384, 640), (2000, 64, 6, 256, 384),
                                       # few rows an expert: with K shared by clusters, and without
                                       (5, 16, 2, 2048, 128), (40, 64, 6, 2048, 128), (1, 8, 8, 1920, 384),
                                       (100, 16, 2, 1024, 1280),
                                       # the most experts
                                       (1100, 1024, 130, 128, 128)])
def test_expert_products(ctx, fmt, scaled, n, E, k, K, N):
    """Both products over segments: padding rows zero, rows behind the last segment untouched, experts without
    tokens, a scale for each expert."""
    ids, seg, perm = route(n, E, k, n)
    P, end = len(perm), int(seg[E])
    x = torch.randn((n, K), generator=gen(n)).to(BF16)
    xp = torch.where(torch.from_numpy(perm >= 0)[:, None], x[torch.from_numpy(np.maximum(perm, 0)).long()], torch.zeros((), dtype=BF16))
    xp[end:] = 3.0                                     # behind the last segment: must not matter
    w, u = ((s * torch.randn((E, N, K), generator=gen(i))).to(BF16) for i, s in ((11, 0.05), (12, 0.2)))
    gs = [t.float().abs().amax((1, 2)) / 2688 if scaled else None for t in (w, u)]
    gx = x.float().abs().max().view(1) / 2688 if scaled else None
    xq, xs, x64 = operand(ctx, xp, fmt, gx)
    wq, ws, w64 = operand(ctx, stacked(w, E), fmt, gs[0])
    uq, us, u64 = operand(ctx, stacked(u, E), fmt, gs[1])
    w64, u64 = w64.reshape(E, N, K), u64.reshape(E, N, K)
    dev = lambda t: None if t is None else t.to(DEV)
    segd = torch.from_numpy(seg).to(DEV)
    tokens = np.zeros(P, bool)
    for e in range(E):
        tokens[seg[e]:seg[e] + seg[E + 1 + e]] = True
    for out in (F32, BF16):
        y = torch.full((P, N), 5.0, dtype=out, device=DEV)
        L.clha_fp4_matmul(ctx, FMT[fmt], xq, xs, P, K, wq, ws, N, y, x_scale=dev(gx), w_scale=dev(gs[0]), seg=segd, E=E)
        want = O.expert_products(x64, w64, seg)
        check_product(y[:end], want[:end], O.expert_products(np.abs(x64), np.abs(w64), seg)[:end], K, out)
        assert (y[end:] == 5.0).all() and (y[:end][~torch.from_numpy(tokens[:end])] == 0).all()
    h = torch.full((P, N), 5.0, dtype=BF16, device=DEV)
    L.clha_fp4_expert_act(ctx, FMT[fmt], xq, xs, P, K, wq, ws, uq, us, N, h, x_scale=dev(gx), g_scale=dev(gs[0]),
                          u_scale=dev(gs[1]), seg=segd, E=E)
    check_act(h[:end], x64[:end], w64, u64, seg, K)
    assert (h[end:] == 5.0).all() and (h[:end][~torch.from_numpy(tokens[:end])] == 0).all()
    L.clha_check(ctx)


def check_act(h, x64, w64, u64, seg, K):
    """The two sums are off by at most t_g, t_u (as in check_product); silu has a slope below 1.1, its float32
    exponential and division a relative error below 2^-20 for |g| < 88, and h is rounded once to bf16."""
    step = (K / 64 + 64) * 2.0 ** -23
    g, u = O.expert_products(x64, w64, seg), O.expert_products(x64, u64, seg)
    tg, tu = (step * O.expert_products(np.abs(x64), np.abs(m), seg) for m in (w64, u64))
    want = O.silu(g) * u
    tol = 1.1 * tg * (np.abs(u) + tu) + np.abs(O.silu(g)) * tu + np.abs(want) * 2.0 ** -20 + 1e-30
    err = np.abs(to64(h) - want)
    assert (err <= tol + (np.abs(want) + tol) * 2.0 ** -8).all(), float((err - tol).max())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,K,N", [(1, 2048, 128), (3, 4096, 256), (130, 128, 384), (257, 640, 128), (2570, 384, 1024),
                                   (130, 4224, 128)])
def test_dense_act(ctx, fmt, n, K, N):
    x = torch.randn((n, K), generator=gen(n)).to(BF16)
    w, u = ((0.05 * torch.randn((N, K), generator=gen(i))).to(BF16) for i in (21, 22))
    (xq, xs, x64), (wq, ws, w64), (uq, us, u64) = (operand(ctx, t, fmt) for t in (x, w, u))
    h = torch.full((n, N), 5.0, dtype=BF16, device=DEV)
    L.clha_fp4_expert_act(ctx, FMT[fmt], xq, xs, n, K, wq, ws, uq, us, N, h)
    check_act(h, x64, w64[None], u64[None], None, K)
    L.clha_check(ctx)


def test_large_activations_do_not_overflow(ctx):
    """Gate sums of +-thousands: silu is 0 or g, never NaN."""
    K, N = 256, 128
    x = torch.full((2, K), 6.0, dtype=BF16)
    w = torch.full((N, K), 6.0, dtype=BF16)
    w[::2] = -6.0
    (xq, xs, x64), (wq, ws, w64) = operand(ctx, x, "e8m0_32"), operand(ctx, w, "e8m0_32")
    h = torch.empty((2, N), dtype=BF16, device=DEV)
    L.clha_fp4_expert_act(ctx, L.FP4_E8M0_32, xq, xs, 2, K, wq, ws, wq, ws, N, h)
    want = torch.from_numpy(O.silu(x64 @ w64.T) * (x64 @ w64.T)).to(BF16)
    assert torch.equal(h.cpu().abs(), want.abs())


def test_nan_scale_reaches_only_its_row(ctx):
    """A block with the formats' NaN scale makes its row of the product NaN and no other."""
    for fmt in FMTS:
        x = torch.randn((130, 256), generator=gen(5))
        x[7, 3] = float("nan")
        w = torch.randn((128, 256), generator=gen(6))
        xq, xs = quantize(ctx, x.to(DEV), fmt)
        with pytest.raises(L.ClhaError):
            L.clha_check(ctx)
        wq, ws = quantize(ctx, w.to(DEV), fmt)
        y = torch.empty((130, 128), device=DEV)
        L.clha_fp4_matmul(ctx, FMT[fmt], xq, xs, 130, 256, wq, ws, 128, y)
        bad = y.isnan().any(1).cpu()
        assert bad[7] and bad.sum() == 1 and y[7].isnan().all()


# ------------------------------------------------------------------ routing
def check_route(ctx, l, k, bias=None, **kw):
    n, E = l.shape
    ids = torch.full((n, k), -7, dtype=torch.int32, device=DEV)
    w = torch.full((n, k), -7.0, device=DEV)
    counts = torch.full((E,), -7, dtype=torch.int32, device=DEV)
    names = {"score": {"softmax": L.SCORE_SOFTMAX, "sigmoid": L.SCORE_SIGMOID},
             "group_rank": {"max": L.GROUP_MAX, "top2": L.GROUP_TOP2}}
    L.clha_route_gated(ctx, l.to(DEV), n, E, k, ids, w, counts, bias=None if bias is None else bias.to(DEV),
                       **{a: names[a][b] if a in names else b for a, b in kw.items()})
    want_ids, want_w, want_counts = O.route_gated(to64(l), k, bias=None if bias is None else to64(bias), **kw)
    np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
    np.testing.assert_array_equal(counts.cpu().numpy(), want_counts)
    # float32: the argument of exp is off by |l - max| 2^-24 (here below 40), exp by 2 steps, a sum of E <= 1024
    # terms by E / 32 + 5, the divisions by 1 each; twice over with the weights' own sum
    tol = 2 * (40 + 4 + 37 + 4) * 2.0 ** -24
    assert (np.abs(to64(w) - want_w) <= tol * np.abs(want_w) + 1e-37).all()
    L.clha_check(ctx)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("n,E,k,groups,top,rank", [
    (1, 1, 1, 1, 1, "max"), (3, 7, 7, 1, 1, "max"), (16, 64, 6, 1, 1, "max"), (17, 64, 6, 8, 3, "top2"),
    (200, 256, 8, 8, 4, "top2"), (33, 40, 4, 5, 2, "max"), (50, 96, 10, 48, 9, "top2"), (40, 12, 3, 12, 5, "top2"),
    (9, 1024, 32, 1, 1, "max"), (9, 1000, 40, 40, 7, "top2"), (70, 300, 5, 3, 1, "max"),
    # groups that cut through a lane's experts, groups of one and of two experts, more groups than lanes for the experts
    (300, 100, 7, 4, 2, "top2"), (61, 16, 4, 8, 3, "top2"), (61, 30, 4, 30, 6, "max"), (130, 328, 9, 8, 5, "top2"),
    (45, 20, 2, 2, 1, "max"), (45, 510, 8, 30, 11, "top2"), (20, 512, 8, 2, 1, "top2"), (20, 384, 8, 4, 3, "max")])
def test_route_gated(ctx, score, dtype, biased, n, E, k, groups, top, rank):
    l = torch.randn((n, E), generator=gen(n * E)).to(dtype)
    bias = 0.2 * torch.randn(E, generator=gen(E)) if biased else None
    for renorm, scale in ((True, 1.0), (False, 2.5)):
        check_route(ctx, l, k, bias, score=score, n_groups=groups, top_groups=top, group_rank=rank, renormalise=renorm,
                    scale=scale)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top,rank", [(1, 1, "max"), (4, 2, "max"), (4, 2, "top2")])
def test_route_near_ties(ctx, score, groups, top, rank):
    """Choices a float32 step apart or equal: the bias undoes the scores up to its rounding, token 0 exactly."""
    E, k = 64, 6
    l = torch.randn((1, E), generator=gen(9))
    s = torch.softmax(l.double(), 1) if score == "softmax" else torch.sigmoid(l.double())
    bias = (0.6 - s[0]).float()
    l = torch.cat((l, l.nextafter(torch.zeros(())), l + torch.randn((30, E), generator=gen(10)) * 1e-7))
    check_route(ctx, l, k, bias, score=score, n_groups=groups, top_groups=top, group_rank=rank)
    same = torch.zeros((20, E))                                  # every choice equal: the lowest experts
    check_route(ctx, same, k, None, score=score, n_groups=groups, top_groups=top, group_rank=rank)
    check_route(ctx, same, k, torch.zeros(E), score=score, n_groups=groups, top_groups=top, group_rank=rank)
    for many in ((40, 128), (70, 1000)):                         # choices above a warp's lanes
        check_route(ctx, torch.zeros((5, many[1])), many[0], torch.zeros(many[1]), score=score)
        check_route(ctx, torch.randn((5, many[1]), generator=gen(12)).mul(4).round().div(4), many[0],
                    torch.zeros(many[1]), score=score, renormalise=groups == 1)
    coarse = torch.randn((64, E), generator=gen(11)).mul(2).round().div(2)   # many exact ties
    check_route(ctx, coarse, k, torch.zeros(E), score=score, n_groups=groups, top_groups=top, group_rank=rank)


def test_route_extreme_logits(ctx):
    """Scores that underflow float32 (and float64): the weights still sum to one."""
    E = 32
    l = torch.full((4, E), -200.0)
    l[1] = -1e4
    l[2] = 3e38
    l[3, :5] = torch.tensor([100.0, 90.0, 80.0, 70.0, 60.0])
    check_route(ctx, l[:3], 4, None, score="sigmoid")
    check_route(ctx, l[3:] + 240, 4, None, score="softmax")
    check_route(ctx, torch.full((2, E), -100.0), 4, 0.1 * torch.randn(E, generator=gen(1)), score="sigmoid")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top,rank", [(64, 1, 1, "max"), (64, 4, 2, "max"), (64, 4, 2, "top2"), (30, 5, 2, "top2"),
                                               (600, 6, 3, "top2"), (600, 1, 1, "max")])
def test_route_biases_of_the_lowest_value(ctx, score, E, groups, top, rank):
    """Experts shut out by a bias of float32's lowest value; fewer open ones than k; group sums past float32's range,
    whose order only the float64 values show."""
    k, low = 6, torch.finfo(F32).min
    l = torch.randn((90, E), generator=gen(E + groups))
    kw = dict(score=score, n_groups=groups, top_groups=top, group_rank=rank)
    bias = 0.2 * torch.randn(E, generator=gen(E))
    some = torch.rand(E, generator=gen(E + 1)) < 0.4
    check_route(ctx, l, k, torch.where(some, low, bias), **kw)
    check_route(ctx, l, k, torch.where(torch.arange(E) < E - 3, low, bias), **kw)
    by_group = torch.linspace(1.0, 0.6, groups).mul(low).repeat_interleave(E // groups)      # the last groups first
    check_route(ctx, l, k, by_group, **kw)
    check_route(ctx, l, k, -by_group, **kw)
    check_route(ctx, l, k, torch.full((E,), low), **kw)


def test_route_scale_over_a_small_sum(ctx):
    """A scale over a sum that leaves float32 where the weights do not."""
    l = torch.randn((20, 64), generator=gen(5)) - 60
    check_route(ctx, l, 4, None, score="sigmoid", scale=1e20)


def test_route_reports_non_finite(ctx):
    E, k = 40, 4
    for where, v in (("l", float("nan")), ("l", float("inf")), ("l", -float("inf")), ("b", float("nan"))):
        l, b = torch.randn((50, E), generator=gen(12)), torch.randn(E, generator=gen(13))
        (l[3] if where == "l" else b)[17] = v
        ids = torch.full((50, k), -7, dtype=torch.int32, device=DEV)
        w, counts = torch.empty((50, k), device=DEV), torch.empty(E, dtype=torch.int32, device=DEV)
        L.clha_route_gated(ctx, l.to(DEV), 50, E, k, ids, w, counts, score=L.SCORE_SIGMOID, bias=b.to(DEV))
        with pytest.raises(L.ClhaError) as ei:
            L.clha_check(ctx)
        assert ei.value.status == L.ERR_NONFINITE
        assert (ids >= 0).all() and (ids < E).all() and int(counts.sum()) == 50 * k
        assert all(len(set(r)) == k for r in ids.tolist())


# ------------------------------------------------------------------ combination
@pytest.mark.parametrize("zt", [F32, BF16])
@pytest.mark.parametrize("yt", [F32, BF16])
@pytest.mark.parametrize("n,E,k,d,weighted,added", [(1, 4, 2, 128, True, False), (5, 64, 6, 384, True, True),
                                                    (700, 8, 3, 2304, False, True), (300, 40, 40, 128, True, False)])
def test_combine(ctx, zt, yt, n, E, k, d, weighted, added):
    ids, seg, perm = route(n, E, k, n)
    P = len(perm)
    z = torch.randn((P, d), generator=gen(n)).to(zt)
    w = torch.rand((n, k), generator=gen(n + 1)) if weighted else None
    add = torch.randn((n, d), generator=gen(n + 2)).to(yt) if added else None
    dev = lambda t: None if t is None else (torch.from_numpy(t) if isinstance(t, np.ndarray) else t).to(DEV)
    y = torch.full((n, d), 5.0, dtype=yt, device=DEV)
    args = (dev(z), P, d, dev(ids), dev(w), n, k, E, dev(seg), dev(perm))
    L.clha_combine(ctx, *args, y, add=dev(add))
    w64 = None if w is None else to64(w)
    want = O.combine(to64(z), ids, w64, seg, perm, E, None if add is None else to64(add))
    mags = O.combine(np.abs(to64(z)), ids, w64, seg, perm, E, None if add is None else np.abs(to64(add)))
    tol = (k + 1) * 2.0 ** -24 * mags      # one rounding for each fused multiply-add
    err = np.abs(to64(y) - want)
    assert (err <= tol + (np.abs(want) + tol) * (2.0 ** -8 if yt == BF16 else 0)).all()
    if added:                              # an addend of the other type; one that is the output itself
        other = F32 if yt == BF16 else BF16
        y3 = torch.full((n, d), 5.0, dtype=yt, device=DEV)
        L.clha_combine(ctx, *args, y3, add=dev(add.to(other)))
        want3 = O.combine(to64(z), ids, w64, seg, perm, E, to64(add.to(other)))
        assert (np.abs(to64(y3) - want3) <= tol * 1.01 + (np.abs(want3) + tol) * (2.0 ** -8 if yt == BF16 else 0)).all()
        y2 = dev(add).clone()
        L.clha_combine(ctx, *args, y2, add=y2)
        assert torch.equal(y2, y)
    L.clha_check(ctx)


def test_combine_with_an_expert_twice(ctx):
    """A token that names one expert in two slots has two equal rows there; each slot counts."""
    n, E, d = 40, 3, 256
    ids = np.stack([np.arange(n) % E, np.where(np.arange(n) % 2, np.arange(n) % E, (np.arange(n) + 1) % E)], 1).astype(np.int32)
    x = torch.randn((n, d), generator=gen(1)).to(DEV)
    P = L.clha_packed_rows(n, 2, E)
    seg, perm = torch.empty(2 * E + 1, dtype=torch.int64, device=DEV), torch.empty(P, dtype=torch.int32, device=DEV)
    z = torch.empty((P, d), device=DEV)
    L.clha_gather(ctx, x, n, d, torch.from_numpy(ids).to(DEV), 2, E, z, P, seg, perm)
    y = torch.empty((n, d), device=DEV)
    L.clha_combine(ctx, z, P, d, torch.from_numpy(ids).to(DEV), None, n, 2, E, seg, perm, y)
    assert torch.equal(y, 2 * x)
    L.clha_check(ctx)


def test_combine_reports_a_missing_token(ctx):
    ids, seg, perm = route(20, 4, 2, 3)
    z = torch.ones((len(perm), 128), device=DEV)
    bad = torch.from_numpy(ids.copy())
    bad[4, 1] = 9                          # no such expert
    perm = perm.copy()
    e = int(ids[6, 0])
    at = seg[e] + int(np.nonzero(perm[seg[e]:seg[e] + seg[5 + e]] == 6)[0][0])
    perm[at] = 7 if perm[at + 1] != 7 else 6
    y = torch.empty((20, 128), device=DEV)
    L.clha_combine(ctx, z, len(perm), 128, bad.to(DEV), None, 20, 2, 4, torch.from_numpy(seg).to(DEV),
                   torch.from_numpy(perm).to(DEV), y)
    with pytest.raises(L.ClhaError) as ei:
        L.clha_check(ctx)
    assert ei.value.status == L.ERR_INVALID_ARG
    assert (y[4] == 1).all() and (y[0] == 2).all()


# ------------------------------------------------------------------ refusals with a context (nothing is queued)
def test_refusals(ctx):
    n, d, E, k = 4, 256, 4, 2
    f = L.FP4_E4M3_16
    x, y = torch.randn((n, d), device=DEV), torch.empty((n, 128), device=DEV)
    q, s = buffers("e4m3_16", n, d)
    wq, ws = buffers("e4m3_16", E * 128, d)
    ids, w, counts = (torch.zeros((n, k), dtype=torch.int32, device=DEV), torch.empty((n, k), device=DEV),
                      torch.empty(E, dtype=torch.int32, device=DEV))
    seg, perm = torch.zeros(2 * E + 1, dtype=torch.int64, device=DEV), torch.zeros(n, dtype=torch.int32, device=DEV)
    one = torch.ones(3, device=DEV)
    lg = torch.randn((n, E), device=DEV)
    odd = torch.empty(n * d + 1, device=DEV)[1:].view(n, d)
    route = lambda **kw: L.clha_route_gated(ctx, lg, n, kw.pop("E", E), kw.pop("k", k), ids, w, counts, **kw)
    A, U = L.ERR_INVALID_ARG, L.ERR_UNSUPPORTED_SHAPE
    cases = [
        (A, lambda: route(score=2)), (A, lambda: route(group_rank=2)), (A, lambda: route(n_groups=3)),
        (A, lambda: route(n_groups=2, top_groups=3)), (A, lambda: route(n_groups=0)), (A, lambda: route(E=0)),
        (A, lambda: route(k=0)), (A, lambda: route(n_groups=4, top_groups=1)), (A, lambda: route(scale=float("nan"))),
        (A, lambda: route(scale=float("inf"))),
        (A, lambda: L.clha_route_gated(ctx, lg, -1, E, k, ids, w, counts)),
        (A, lambda: L.clha_fp4_quantize(ctx, x, n, d, 5, q, s)),
        (U, lambda: L.clha_fp4_quantize(ctx, x, n, 192, f, q, s)),
        (A, lambda: L.clha_fp4_quantize(ctx, x, n, d, f, q, s, rows=3)),
        (A, lambda: L.clha_fp4_quantize(ctx, x, n, d, f, q, s, tensor_scale=one)),
        (A, lambda: L.clha_fp4_quantize(ctx, odd, n, d, f, q, s)),
        (A, lambda: L.clha_fp4_quantize(ctx, x, n, d, f, q, None)),
        (U, lambda: L.clha_fp4_dequantize(ctx, q, s, n, 64, f, x)),
        (A, lambda: L.clha_fp4_dequantize(ctx, q, s, n, d, f, odd)),
        (U, lambda: L.clha_fp4_tensor_scale(ctx, x, 1, n, 100, f, one)),
        (A, lambda: L.clha_fp4_tensor_scale(ctx, x, 0, n, d, f, one)),
        (A, lambda: L.clha_fp4_matmul(ctx, 9, q, s, n, d, wq, ws, 128, y)),
        (U, lambda: L.clha_fp4_matmul(ctx, f, q, s, n, d, wq, ws, 64, y)),
        (U, lambda: L.clha_fp4_matmul(ctx, f, q, s, n, 64, wq, ws, 128, y)),
        (A, lambda: L.clha_fp4_matmul(ctx, f, q, s, n, d, wq, ws, 128, y, E=2)),
        (A, lambda: L.clha_fp4_matmul(ctx, f, q, None, n, d, wq, ws, 128, y)),
        (A, lambda: L.clha_fp4_expert_act(ctx, f, q, s, n, d, wq, ws, None, None, 128, y.to(BF16))),
        (A, lambda: L.clha_combine(ctx, x, n, d, ids, None, n, k, 1, seg, perm, x)),   # k > E
        (U, lambda: L.clha_combine(ctx, x, n, 64, ids, None, n, k, E, seg, perm, x)),
        (A, lambda: L.clha_combine(ctx, odd, n, d, ids, None, n, k, E, seg, perm, x)),
    ]
    launched = L.clha_kernel_launches(ctx)
    for i, (status, call) in enumerate(cases):
        with pytest.raises(L.ClhaError) as ei:
            call()
        assert ei.value.status == status, (i, ei.value)
    params = L._route_params(E, k, L.SCORE_SOFTMAX, 1, 1, L.GROUP_MAX, True, 1.0)     # more tokens than a count holds
    assert L.load().clha_route_gated(ctx.handle, lg.data_ptr(), L.F32, 2 ** 31, ctypes.byref(params), None, ids.data_ptr(),
                                     w.data_ptr(), counts.data_ptr()) == A
    with pytest.raises(ValueError):        # a non-contiguous tensor
        L.clha_fp4_quantize(ctx, torch.randn((d, n), device=DEV).T, n, d, f, q, s)
    with pytest.raises(TypeError):         # half-precision inputs are not taken
        L.clha_fp4_quantize(ctx, x.half(), n, d, f, q, s)
    assert L.clha_kernel_launches(ctx) == launched
    L.clha_check(ctx)


def test_no_rows(ctx):
    """Zero tokens: counts are cleared, nothing else is touched."""
    e = torch.empty(0, device=DEV)
    u = torch.empty(0, dtype=torch.uint8, device=DEV)
    counts = torch.full((4,), 9, dtype=torch.int32, device=DEV)
    L.clha_route_gated(ctx, e, 0, 4, 2, e.int(), e, counts)
    assert (counts == 0).all()
    L.clha_fp4_quantize(ctx, e, 0, 128, L.FP4_E8M0_32, u, u)
    L.clha_fp4_dequantize(ctx, u, u, 0, 128, L.FP4_E8M0_32, e)
    w = torch.zeros((128, 64), dtype=torch.uint8, device=DEV)
    s = torch.zeros(512, dtype=torch.uint8, device=DEV)
    L.clha_fp4_matmul(ctx, L.FP4_E8M0_32, u, u, 0, 128, w, s, 128, e)
    L.clha_fp4_expert_act(ctx, L.FP4_E8M0_32, u, u, 0, 128, w, s, w, s, 128, e.to(BF16))
    seg, perm = torch.zeros(9, dtype=torch.int64, device=DEV), torch.full((512,), -1, dtype=torch.int32, device=DEV)
    L.clha_combine(ctx, torch.zeros((512, 128), device=DEV), 512, 128, e.int(), e, 0, 2, 4, seg, perm, e)
    # segments without any token: an empty product
    xq, xs = buffers("e8m0_32", 512, 128)
    y = torch.full((512, 128), 5.0, device=DEV)
    L.clha_fp4_quantize(ctx, e, 0, 128, L.FP4_E8M0_32, xq, xs, perm=perm, rows=512, seg=seg, E=4)
    L.clha_fp4_matmul(ctx, L.FP4_E8M0_32, xq, xs, 512, 128, w.repeat(4, 1), s.repeat(4), 128, y, seg=seg, E=4)
    assert (xq == 0xA5).all() and (y == 5.0).all()
    L.clha_check(ctx)


# ------------------------------------------------------------------ the layer
def layer_case(n, E, k, dm, dff, ns, sdff, seed=0):
    from post_quantization_expert_b200.pipeline import MoEWeights
    g = gen(seed)
    r = lambda *s: (0.05 * torch.randn(s, generator=g)).to(BF16)
    w = MoEWeights(r(2 * E, dff, dm), r(E, dm, dff), r(2 * ns, sdff, dm) if ns else None, r(ns, dm, sdff) if ns else None)
    return w, torch.randn((n, dm), generator=g).to(BF16), torch.randn((n, E), generator=g)


def to_dev(w):
    from post_quantization_expert_b200.pipeline import MoEWeights
    return MoEWeights(*(None if t is None else t.to(DEV) for t in (w.Wgu, w.Wd, w.Sgu, w.Sd)))


def quantized_weight(W, fmt):
    """Exact values of the layer's 4-bit weights [E, N, K]."""
    E, N, K = W.shape
    g = np.ones(E)
    if fmt == "e4m3_16":
        g = (W.float().abs().amax((1, 2)).numpy() / np.float32(2688.0)).astype(np.float64)
    rows = to64(W).reshape(E * N, K)
    per = np.repeat(g, N)
    return O.fp4_values(*O.fp4_quantize(rows, fmt, per), fmt, per).reshape(E, N, K)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,E,k,dm,dff,ns,sdff,gx,gh", [
    (1, 8, 2, 256, 128, 0, 0, None, None), (37, 16, 2, 384, 256, 2, 128, None, 1.7e-3),
    (700, 8, 3, 256, 384, 1, 256, 0.013, None)])
def test_layer(ctx, fmt, n, E, k, dm, dff, ns, sdff, gx, gh):
    """The calls together, each stage against the oracle on the stage's own inputs as the GPU left them (so that
    a 4-bit code on a border, decided by float32 sums, is not carried on)."""
    from post_quantization_expert_b200.pipeline import Fp4Layer
    w, X, lg = layer_case(n, E, k, dm, dff, ns, sdff)
    scales = {a: None if g is None else torch.tensor([g], device=DEV) for a, g in (("x_scale", gx), ("h_scale", gh))}
    gx, gh = (1.0 if g is None else float(np.float32(g)) for g in (gx, gh))
    layer = Fp4Layer(ctx, to_dev(w), k, max_tokens=n + 5, fmt=FMT[fmt], score=L.SCORE_SIGMOID, scale=1.5, **scales)
    Y = torch.full((n, dm), 5.0, device=DEV)
    assert layer.forward(X.to(DEV), lg.to(DEV), Y) is Y
    L.clha_check(ctx)
    ids, wts, counts = O.route_gated(to64(lg), k, score="sigmoid", scale=1.5)
    np.testing.assert_array_equal(layer.ids[:n].cpu().numpy(), ids)
    np.testing.assert_array_equal(layer.counts.cpu().numpy(), counts)
    seg, perm = layer.seg.cpu().numpy(), layer.perm.cpu().numpy()
    end = int(seg[E])
    x64 = np.where((perm[:end] >= 0)[:, None], to64(X)[np.maximum(perm[:end], 0)], 0.0)
    W = [quantized_weight(t, fmt) for t in (w.Wg, w.Wu, w.Wd)]
    check_act(layer.h[:end], O.fp4_values(*O.fp4_quantize(x64, fmt, gx), fmt, gx), W[0], W[1], seg, dm)
    h64 = O.fp4_values(*O.fp4_quantize(to64(layer.h[:end]), fmt, gh), fmt, gh)
    check_product(layer.z[:end], O.expert_products(h64, W[2], seg), O.expert_products(np.abs(h64), np.abs(W[2]), seg), dff,
                  F32)
    add = mags = None
    if ns:
        S = [quantized_weight(t.reshape(1, ns * sdff, dm), fmt) for t in (w.Sg, w.Su)]
        S.append(quantized_weight(w.Sd.permute(1, 0, 2).reshape(1, dm, ns * sdff).contiguous(), fmt))
        check_act(layer.sh[:n], O.fp4_values(*O.fp4_quantize(to64(X), fmt, gx), fmt, gx), S[0], S[1], None, dm)
        hs = O.fp4_values(*O.fp4_quantize(to64(layer.sh[:n]), fmt, gh), fmt, gh)
        add, mags = hs @ S[2][0].T, np.abs(hs) @ np.abs(S[2][0]).T
    z64 = to64(layer.z)
    got_w = to64(layer.weights[:n])
    want = O.combine(z64, ids, got_w, seg, perm, E, add)
    tol = (k + 1) * 2.0 ** -24 * O.combine(np.abs(z64), ids, got_w, seg, perm, E, None if add is None else np.abs(add))
    if ns:
        tol = tol + (ns * sdff / 64 + 64) * 2.0 ** -23 * mags
    assert (np.abs(to64(Y) - want) <= tol + 1e-30).all()
    with pytest.raises(ValueError):
        layer.forward(X.to(DEV).repeat(2 * (n + 6) // n + 1, 1), lg.to(DEV), Y)
    one = torch.full((1, dm), 5.0, device=DEV)      # fewer tokens after more: the buffers hold the earlier call's rows
    layer.forward(X[:1].to(DEV).contiguous(), lg[:1].to(DEV).contiguous(), one)
    fresh = Fp4Layer(ctx, to_dev(w), k, max_tokens=1, fmt=FMT[fmt], score=L.SCORE_SIGMOID, scale=1.5, **scales)
    assert torch.equal(one, fresh.forward(X[:1].to(DEV).contiguous(), lg[:1].to(DEV).contiguous(), torch.empty_like(one)))
    empty = torch.empty((0, dm), device=DEV)
    layer.forward(empty, torch.empty((0, E), device=DEV), empty)
    assert (layer.counts == 0).all()
    L.clha_check(ctx)


def test_layer_captured_and_on_other_streams(ctx):
    """A captured graph replayed on new inputs gives the eager bits; so do two contexts on streams of their own,
    queued at once, and a second graph of the same layer."""
    from post_quantization_expert_b200.pipeline import Fp4Layer
    n, E, k, dm, dff = 70, 8, 2, 256, 256
    w, X, lg = layer_case(n, E, k, dm, dff, 1, 128)
    wd = to_dev(w)
    Xs = [X.to(DEV), (2 * X).to(DEV)]
    lgs = [lg.to(DEV), (-lg).to(DEV)]
    layer = Fp4Layer(ctx, wd, k, n, fmt=L.FP4_E4M3_16)
    want = [layer.forward(x, l, torch.empty((n, dm), dtype=BF16, device=DEV)) for x, l in zip(Xs, lgs)]
    torch.cuda.synchronize()
    # captures take a stream of their own, with a context on it
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    c1, c2 = L.Context(0, s1), L.Context(0, s2)
    s1.wait_stream(torch.cuda.current_stream())
    s2.wait_stream(torch.cuda.current_stream())
    l1, l2 = Fp4Layer(c1, wd, k, n), Fp4Layer(c2, wd, k, n)
    for _ in range(3):
        with torch.cuda.stream(s1):
            y1 = l1.forward(Xs[0], lgs[0], torch.empty((n, dm), dtype=BF16, device=DEV))
        with torch.cuda.stream(s2):
            y2 = l2.forward(Xs[1], lgs[1], torch.empty((n, dm), dtype=BF16, device=DEV))
    torch.cuda.synchronize()
    assert torch.equal(y1, want[0]) and torch.equal(y2, want[1])
    xin, lin, yout = Xs[0].clone(), lgs[0].clone(), torch.zeros((n, dm), dtype=BF16, device=DEV)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s1):
            l1.forward(xin, lin, yout)
        graphs.append(g)
    for i in (0, 1, 0):
        with torch.cuda.stream(s1):
            xin.copy_(Xs[i])
            lin.copy_(lgs[i])
            graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(yout, want[i]), i
    for c in (c1, c2, ctx):
        L.clha_check(c)
    del graphs, g
    c1.close()
    c2.close()


def test_layer_built_on_another_stream(ctx):
    """Weights that the current stream has yet to write, quantized on the context's own stream."""
    from post_quantization_expert_b200.pipeline import Fp4Layer
    n, E, k, dm, dff = 40, 8, 2, 256, 256
    w, X, lg = layer_case(n, E, k, dm, dff, 2, 128)
    wd, x, l = to_dev(w), X.to(DEV), lg.to(DEV)
    want = Fp4Layer(ctx, wd, k, n).forward(x, l, torch.empty((n, dm), device=DEV))
    late, busy = to_dev(w), torch.zeros((8192, 8192), dtype=BF16, device=DEV)
    fields = [t for t in vars(late).values() if torch.is_tensor(t)]
    kept = [t.clone() for t in fields]
    for t in fields:
        t.zero_()
    torch.cuda.synchronize()
    own = L.Context(0, torch.cuda.Stream())
    for _ in range(20):                    # a few milliseconds
        busy = busy @ busy
    for t, v in zip(fields, kept):
        t.copy_(v)
    layer = Fp4Layer(own, late, k, n)
    dropped = [torch.full((k_, 1 << 16), -1.0, dtype=BF16, device=DEV) for k_ in (1, 2, 3, 4)]   # reuses what was freed
    with torch.cuda.stream(own.stream):
        got = layer.forward(x, l, torch.empty((n, dm), device=DEV))
    torch.cuda.synchronize()
    assert torch.equal(got, want) and len(dropped) == 4
    L.clha_check(own)
    own.close()


def test_offsets_past_32_bits(ctx):
    """Codes, scales, values and outputs whose element offsets pass 2^31: the last rows against a small call."""
    rows, d, f = 131329, 16384, L.FP4_E8M0_32          # 2.15e9 elements
    x = torch.empty((rows, d), dtype=BF16, device=DEV)
    x[:-300] = 1.0
    x[-300:] = torch.randn((300, d), generator=gen(8)).to(BF16).to(DEV)
    codes = torch.empty((rows, d // 2), dtype=torch.uint8, device=DEV)
    scales = torch.empty(L.clha_fp4_scale_bytes(f, rows, d), dtype=torch.uint8, device=DEV)
    L.clha_fp4_quantize(ctx, x, rows, d, f, codes, scales)
    tail = x[-257:].contiguous()                       # 131072 = 1024 * 128: the same places in their tiles
    wc, wsc = quantize(ctx, tail, "e8m0_32")
    assert torch.equal(codes[-257:], wc) and torch.equal(scales[-wsc.numel():], wsc)
    L.clha_fp4_dequantize(ctx, codes, scales, rows, d, f, x)
    v = torch.empty((257, d), dtype=BF16, device=DEV)
    L.clha_fp4_dequantize(ctx, wc, wsc, 257, d, f, v)
    assert torch.equal(x[-257:], v)
    del x
    w = torch.randn((16384 + 128, 128), generator=gen(9))
    wq, ws = quantize(ctx, w.to(DEV), "e8m0_32")       # Y [rows, 16512]: 2.17e9 elements
    xq, xs = codes[:, :64].contiguous(), None
    xs = torch.full((L.clha_fp4_scale_bytes(f, rows, 128),), 127, dtype=torch.uint8, device=DEV)
    y = torch.empty((rows, 16512), dtype=BF16, device=DEV)
    L.clha_fp4_matmul(ctx, f, xq, xs, rows, 128, wq, ws, 16512, y)
    small = torch.empty((257, 16512), dtype=BF16, device=DEV)
    L.clha_fp4_matmul(ctx, f, xq[-257:].contiguous(), xs[-3 * 512:].contiguous(), 257, 128, wq, ws, 16512, small)
    assert torch.equal(y[-257:], small)
    L.clha_check(ctx)
    del codes, scales, y, small, xq
    torch.cuda.empty_cache()


@pytest.mark.parametrize("how", ["overwritten", "dropped"])
def test_layer_weights_are_the_callers_again(ctx, how):
    """Once a layer is built, its weights may be overwritten or dropped on the current stream, although the context's own
    stream has yet to read them."""
    from post_quantization_expert_b200.pipeline import Fp4Layer
    n, E, k, dm, dff = 40, 8, 2, 256, 256
    w, X, lg = layer_case(n, E, k, dm, dff, 2, 128)
    x, l = X.to(DEV), lg.to(DEV)
    want = Fp4Layer(ctx, to_dev(w), k, n).forward(x, l, torch.empty((n, dm), device=DEV))
    own = L.Context(0, torch.cuda.Stream())
    Fp4Layer(own, to_dev(w), k, n)         # (leaves its buffers in the stream's pool: the next one is built without a wait)
    mine = to_dev(w)
    torch.cuda.synchronize()
    with torch.cuda.stream(own.stream):    # some ten milliseconds
        busy = torch.zeros((8192, 8192), dtype=BF16, device=DEV)
        for _ in range(20):
            busy = busy @ busy
    layer = Fp4Layer(own, mine, k, n)
    if how == "overwritten":
        again = [t.fill_(7.0) for t in vars(mine).values()]
    else:
        sizes = [t.shape for t in vars(mine).values()]
        del mine
        again = [torch.full(s, 7.0, dtype=BF16, device=DEV) for s in sizes]
    with torch.cuda.stream(own.stream):
        got = layer.forward(x, l, torch.empty((n, dm), device=DEV))
    torch.cuda.synchronize()
    assert torch.equal(got, want) and all((t == 7.0).all() for t in again)
    L.clha_check(own)
    own.close()


@pytest.mark.parametrize("n,E,k", [(0, 4, 2), (1, 64, 6), (300, 10, 3), (1000, 300, 4)])
def test_gather_with_the_callers_scratch(ctx, n, E, k):
    """The same permutation, segments and rows as clha_gather, within the bytes that it asks for; fewer are refused."""
    ids = torch.from_numpy(route(n, E, k, n)[0]).to(DEV)
    X = torch.randn((n, 128), generator=gen(n)).to(DEV)
    P, need = L.clha_packed_rows(n, k, E), L.clha_gather_scratch_bytes(n, E)

    def run(call, *scratch):
        perm, seg = torch.zeros(P, dtype=torch.int32, device=DEV), torch.zeros(2 * E + 1, dtype=torch.int64, device=DEV)
        out = torch.full((P, 128), 5.0, device=DEV)
        call(ctx, X, n, 128, ids, k, E, out, P, seg, perm, *scratch)
        return perm, seg, out
    buf = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device=DEV)
    for a, b in zip(run(L.clha_gather), run(L.clha_gather_scratch, buf[:need])):
        assert torch.equal(a, b)
    assert (buf[need:] == 0xA5).all()
    for bad in (buf[:need - 1], buf[1:], None):
        with pytest.raises(L.ClhaError):
            run(L.clha_gather_scratch, bad)
    L.clha_check(ctx)


def test_layer_graph_outlives_the_workspace():
    """A forward captured before any eager call, replayed after calls that make the context's workspace grow and move."""
    from post_quantization_expert_b200.pipeline import Fp4Layer
    n, E, k, dm, dff = 600, 8, 2, 256, 256
    w, X, lg = layer_case(n, E, k, dm, dff, 1, 128)
    x, l = X.to(DEV), lg.to(DEV)
    s = torch.cuda.Stream()
    own = L.Context(0, s)
    layer = Fp4Layer(own, to_dev(w), k, n)
    few, some = torch.zeros((3, dm), device=DEV), torch.zeros((n, dm), device=DEV)
    torch.cuda.synchronize()
    small, large = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(small, stream=s):
        layer.forward(x[:3], l[:3], few)
    with torch.cuda.graph(large, stream=s):
        layer.forward(x, l, some)
    with torch.cuda.stream(s):
        want = layer.forward(x, l, torch.empty((n, dm), device=DEV))
        ids = torch.zeros((1 << 20, 1), dtype=torch.int32, device=DEV)
        P = L.clha_packed_rows(1 << 20, 1, 64)
        for _ in range(2):
            L.clha_gather(own, torch.empty((1 << 20, 128), device=DEV), 1 << 20, 128, ids, 1, 64, None, P,
                          torch.empty(129, dtype=torch.int64, device=DEV), torch.empty(P, dtype=torch.int32, device=DEV))
        for _ in range(3):
            large.replay()
            small.replay()
    torch.cuda.synchronize()
    assert torch.equal(some, want)
    with torch.cuda.stream(s):
        assert torch.equal(few, layer.forward(x[:3], l[:3], torch.empty_like(few)))
    L.clha_check(own)
    del small, large
    own.close()


def every_scale(ctx, fmt, g):
    """Every code under every finite scale byte, one row for each of the matrix scales g (host float32): the codes and
    tiled scales on the device, and their exact values."""
    top = 255 if fmt == "e8m0_32" else 127
    byte = np.tile(np.minimum(np.arange((top + 7) // 8 * 8), top - 1).astype(np.uint8), (len(g), 1))
    codes = np.tile(np.arange(16, dtype=np.uint8), (len(g), byte.shape[1] * O.BLOCK[fmt] // 16))
    want = O.fp4_values(codes, byte, fmt, to64(g))
    return torch.from_numpy(O.pack_codes4(codes)).to(DEV), torch.from_numpy(O.tile_scales(byte)).to(DEV), want


@pytest.mark.parametrize("fmt", FMTS)
def test_dequantize_every_scale(ctx, fmt):
    """float32 values of every code and finite scale, rounded once, also where q * s alone passes float32's range."""
    g = torch.tensor([1.0, 0.37, 2.0 ** -20, 1.0 - 2.0 ** -24, 1.0 + 2.0 ** -23, 3.3e-12, 1.3 * 2.0 ** -100, 2.0 ** -126, 1e-42,
                      1e30, 3e38])
    codes, scales, want = every_scale(ctx, fmt, g)
    with np.errstate(over="ignore"):
        want32 = want.astype(np.float32)
    got = torch.empty(want.shape, device=DEV)
    L.clha_fp4_dequantize(ctx, codes, scales, *want.shape, FMT[fmt], got, tensor_scale=g.to(DEV))
    np.testing.assert_array_equal(got.cpu().numpy(), want32)
    L.clha_check(ctx)


def nearest_bf16(x64):
    """Float64 -> bf16, nearest even, in one rounding, subnormal numbers included."""
    step = np.ldexp(1.0, np.maximum(np.frexp(x64)[1], -125) - 8)
    return torch.from_numpy(np.rint(x64 / step) * step).to(BF16)


@pytest.mark.parametrize("fmt", FMTS)
def test_dequantize_small_values_to_bf16(ctx, fmt):
    """Values above the middle between two bf16 numbers by less than float32 can hold there: v G = T 2^shift + r with T odd
    of 9 bits, v = 3 or 27 and 0 < r < v, times a power of two. Rounded once, they go up."""
    if fmt == "e4m3_16":
        v, unit, code, byte, shift = 27, -10, 3, O.E4M3.tolist().index(9 * 2.0 ** -9), 20     # q s = 1.5 * 9 * 2^-9
    else:
        v, unit, code, byte, shift = 3, -21, 3, 127 - 20, 17                                  # q s = 1.5 * 2^-20
    T = np.arange(257, 512, 2, dtype=np.int64) << shift
    G = T // v + 1
    G = G[(G < 2 ** 24) & (G * v > T)]
    for low in (-126, -130, -122, 0):                                                         # T 2^-shift 2^(low - 8) >= 2^low
        g = torch.from_numpy(np.ldexp(G.astype(np.float64), low - 8 - shift - unit)).float()
        codes = np.full((len(g), 128), code, np.uint8)
        bytes_ = np.full((len(g), 128 // O.BLOCK[fmt]), byte, np.uint8)
        want = nearest_bf16(O.fp4_values(codes, bytes_, fmt, to64(g)))
        got = torch.empty((len(g), 128), dtype=BF16, device=DEV)
        L.clha_fp4_dequantize(ctx, torch.from_numpy(O.pack_codes4(codes)).to(DEV), torch.from_numpy(O.tile_scales(bytes_)).to(DEV),
                              len(g), 128, FMT[fmt], got, tensor_scale=g.to(DEV))
        assert torch.equal(got.cpu(), want), low
    L.clha_check(ctx)


def act_between(h, g, u):
    """h against silu(g) u of exact sums g, u (float64), rounded once to bf16. The exponential's argument is rounded twice (its
    constant and the product), 1.5 2^-24 |g|; the exponential of its half is off by 2^-22 and counts twice, the reciprocal by
    2^-23, six more operations by 2^-24 each."""
    d = (1.5 * np.abs(g) + 16) * 2.0 ** -24
    want = O.silu(g) * u
    a, b = (round_bf16(want * (1 + s * d)) for s in (-1, 1))
    return bool(((h.cpu() >= torch.minimum(a, b)) & (h.cpu() <= torch.maximum(a, b))).all())


@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("n,K,N", [(20, 128, 128), (64, 128, 256), (3, 4096, 128), (4000, 128, 1024)])
def test_act_of_large_sums(ctx, sign, n, K, N):
    """Gate sums from +-1 to +-92 that are exact (one product of two values each), beside up sums large enough that silu's
    smallest values count."""
    x, w, u = torch.zeros((n, K)), torch.zeros((N, K)), torch.zeros((N, K))
    x[:, 0] = sign * torch.linspace(1, 9.6, n)
    x[:, 64] = 1.0
    w[:, 0] = torch.linspace(1, 9.6, N)
    u[:, 64] = torch.tensor([1.0, -3.0]).repeat(N // 2)
    (xq, xs, x64), (wq, ws, w64), (uq, us, u64) = (operand(ctx, t, "e4m3_16") for t in (x, w, u))
    h = torch.empty((n, N), dtype=BF16, device=DEV)
    big = torch.tensor([2.0 ** 100], device=DEV)
    L.clha_fp4_expert_act(ctx, L.FP4_E4M3_16, xq, xs, n, K, wq, ws, uq, us, N, h, u_scale=big)
    g = x64 @ w64.T
    assert np.abs(g).max() > 91 and act_between(h, g, x64 @ u64.T * 2.0 ** 100)
    L.clha_check(ctx)


@pytest.mark.parametrize("E", [30, 64, 256, 500, 600])
def test_route_small_sigmoid_scores(ctx, E):
    """Sigmoids at the lower end of float32, as weights times a scale that brings them back. The exponential and the
    division are off by 2^-22 each, or by two steps of 2^-149 where they are subnormal, the scaling by 2^-24."""
    k, scale = 8, 2.0 ** 100
    l, bias = -80 - 20 * torch.rand((40, E), generator=gen(E)), torch.linspace(0, 1, E)
    ids, w, counts = (torch.empty((40, k), dtype=torch.int32, device=DEV), torch.empty((40, k), device=DEV),
                      torch.empty(E, dtype=torch.int32, device=DEV))
    L.clha_route_gated(ctx, l.to(DEV), 40, E, k, ids, w, counts, score=L.SCORE_SIGMOID, renormalise=False, scale=scale,
                       bias=bias.to(DEV))
    want_ids, want, _ = O.route_gated(to64(l), k, score="sigmoid", renormalise=False, scale=scale, bias=to64(bias))
    got = to64(w)
    np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
    assert (np.abs(got - want) <= 2.0 ** -20 * want + 4 * 2.0 ** -149 * scale).all(), float((got / want).min())
    L.clha_check(ctx)


@pytest.mark.parametrize("x_scale,w_scale,top", [(1.3 * 2.0 ** -70, 1.7 * 2.0 ** -72, 40), (2.0 ** 100, 1.5 * 2.0 ** 40, -60),
                                                 (3e-39, 1.0, 10), (1e-20, 1e30, 3)])
def test_products_under_extreme_matrix_scales(ctx, x_scale, w_scale, top):
    """Matrix scales whose product leaves float32's (normal) range while the scaled sums do not: rows of zeros stay zero,
    and the sums keep their bits. Values around 2^top."""
    for n, K, N in ((20, 256, 128), (3, 4096, 128), (64, 256, 256), (4000, 256, 1024)):
        x, w = (torch.randn((r, K), generator=gen(r)) * 2.0 ** top for r in (n, N))
        x[2] = 0
        (xq, xs, x64), (wq, ws, w64) = operand(ctx, x, "e8m0_32"), operand(ctx, w, "e8m0_32")
        a, b = (torch.tensor([v], device=DEV) for v in (x_scale, w_scale))
        both = float(np.float64(np.float32(x_scale)) * np.float64(np.float32(w_scale)))
        for out in (F32, BF16):
            y = torch.empty((n, N), dtype=out, device=DEV)
            L.clha_fp4_matmul(ctx, L.FP4_E8M0_32, xq, xs, n, K, wq, ws, N, y, x_scale=a, w_scale=b)
            check_product(y, x64 @ w64.T * both, np.abs(x64) @ np.abs(w64).T * both, K, out)
            assert (y[2] == 0).all()
        h = torch.empty((n, N), dtype=BF16, device=DEV)
        L.clha_fp4_expert_act(ctx, L.FP4_E8M0_32, xq, xs, n, K, wq, ws, wq, ws, N, h, x_scale=a, g_scale=b, u_scale=b)
        check_act(h, x64 * both, w64[None], w64[None], None, K)
        assert (h[2] == 0).all()
    L.clha_check(ctx)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_a_scale_for_each_expert(ctx, fmt, dtype):
    """Weights of eight experts, each under its own matrix scale."""
    E, rows, d = 8, 520, 384
    x = (torch.randn((E, rows, d), generator=gen(31)) * torch.logspace(-3, 2, E)[:, None, None]).to(dtype)
    g = torch.empty(E, device=DEV)
    L.clha_fp4_tensor_scale(ctx, x.to(DEV), E, rows, d, FMT[fmt], g)
    codes, scales = quantize(ctx, x.view(-1, d).to(DEV), fmt, g)
    check_quantized(codes, scales, to64(x.view(-1, d)), fmt, np.repeat(to64(g), rows))
    L.clha_check(ctx)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("more", [0, 1, 5, 300])
def test_products_of_more_tiles_than_the_sizes_tell(ctx, fmt, more):
    """Each of 16 experts with 64 tokens in a call of their 2048 rows and `more`: the number of rows alone is that of far fewer
    row tiles (2049 rows could hold one token), so that K is shared by a cluster."""
    n, E, K, N = 64, 16, 4096, 128
    _, seg, perm = route(n, E, E, 0)
    rows, end = int(seg[E]) + more, int(seg[E])
    assert end == 128 * E
    x = torch.randn((rows, K), generator=gen(more)).to(BF16)
    w = 0.05 * torch.randn((E * N, K), generator=gen(32))
    (xq, xs, x64), (wq, ws, w64) = operand(ctx, x, fmt), operand(ctx, w, fmt)
    w64, segd = w64.reshape(E, N, K), torch.from_numpy(seg).to(DEV)
    y = torch.full((rows, N), 5.0, device=DEV)
    L.clha_fp4_matmul(ctx, FMT[fmt], xq, xs, rows, K, wq, ws, N, y, seg=segd, E=E)
    check_product(y[:end], O.expert_products(x64, w64, seg)[:end], O.expert_products(np.abs(x64), np.abs(w64), seg)[:end], K, F32)
    h = torch.full((rows, N), 5.0, dtype=BF16, device=DEV)
    L.clha_fp4_expert_act(ctx, FMT[fmt], xq, xs, rows, K, wq, ws, wq, ws, N, h, seg=segd, E=E)
    check_act(h[:end], x64[:end], w64, w64, seg, K)
    tokens = torch.from_numpy(perm[:end] >= 0)
    for out in (y, h):
        assert (out[end:] == 5.0).all() and (out[:end][~tokens] == 0).all()
    L.clha_check(ctx)


@pytest.mark.parametrize("n,N", [(20, 128), (64, 256), (4000, 1024)])
def test_products_of_extreme_block_scales(ctx, n, N):
    """Power-of-two block scales up to 2^127 that meet scales down to 2^-127: products of ordinary size."""
    K = 256
    up = torch.linspace(60, 125, K // 32).round().repeat_interleave(32)
    x, w = torch.randn((n, K), generator=gen(n)).clamp(-3, 3), torch.randn((N, K), generator=gen(N)).clamp(-3, 3)
    x, w = x * 2.0 ** up, w * 2.0 ** (-up)
    (xq, xs, x64), (wq, ws, w64) = operand(ctx, x, "e8m0_32"), operand(ctx, w, "e8m0_32")
    y = torch.empty((n, N), device=DEV)
    L.clha_fp4_matmul(ctx, L.FP4_E8M0_32, xq, xs, n, K, wq, ws, N, y)
    check_product(y, x64 @ w64.T, np.abs(x64) @ np.abs(w64).T, K, F32)
    L.clha_check(ctx)


@pytest.mark.parametrize("n,E,k", [(700, 64, 48), (700, 64, 49), (300, 256, 130), (257, 1024, 1024)])
def test_gather_of_many_choices(ctx, n, E, k):
    """More choices a token than fit a block's shared memory; one token names an expert twice, another one outside."""
    ids, _, _ = route(n, E, k, n)
    ids[5, 1], ids[n - 1, 0] = ids[5, 0], E
    counts = np.bincount(ids[ids < E], minlength=E)
    starts = np.concatenate([[0], np.cumsum((counts + 127) // 128 * 128)])
    P = L.clha_packed_rows(n, k, E)
    want = np.full(P, -1, np.int32)
    for e in range(E):                     # a token's row where its first choice of e comes in the count
        at = starts[e]
        for t, c in enumerate((ids == e).sum(1)):
            if c:
                want[at] = t
                at += c
    perm, seg = torch.zeros(P, dtype=torch.int32, device=DEV), torch.zeros(2 * E + 1, dtype=torch.int64, device=DEV)
    L.clha_gather(ctx, torch.zeros((n, 128), device=DEV), n, 128, torch.from_numpy(ids).to(DEV), k, E, None, P, seg, perm)
    np.testing.assert_array_equal(seg.cpu().numpy(), np.concatenate([starts, counts]))
    np.testing.assert_array_equal(perm.cpu().numpy(), want)
    with pytest.raises(L.ClhaError) as ei:
        L.clha_check(ctx)
    assert ei.value.status == L.ERR_INVALID_ARG

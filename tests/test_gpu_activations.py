"""GPU parity of the activation operators with the fp64 oracle.

Tolerances, from the arithmetic: rounding to bf16 is off by at most 2^-8 of the
value, an fp32 operation by 2^-24 (a tensor-core addition, which may truncate,
by 2^-23); a sum of n terms by n such steps of the sum of magnitudes."""
import ctypes

import numpy as np
import pytest
import torch

import matrix_orthogonalising_optimizer_step_b200 as mc
from oracle import activations as oa

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def draw(seed, *shape, std=1.0, dtype=BF):
    """Gaussian rows with channels of unequal size."""
    g = gen(seed)
    size = torch.exp(torch.randn(shape[-1], generator=g, device=DEV))
    return (torch.randn(*shape, generator=g, device=DEV) * size * std).to(dtype)


def n64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def ok():
    assert mc.device_status() == mc.MC_OK, mc.last_error()


def within(got, want, bound, tag=""):
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{tag}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - want) - bound)} beyond its bound"


def values(a):
    """The oracle's reading of an Act8."""
    D = a.shape[-1]
    return oa.act8_values(a.q.cpu().numpy(), a.scale.cpu().numpy(), D, a.fmt)


# ------------------------------------------------------------------ 8 bits
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,D", [(1, 1), (1, 4096), (3, 31), (5, 33), (7, 256), (4, 257), (130, 1000), (33, 1789), (2, 8), (1000, 72), (21, 98), (40, 1594), (3, 258)])
def test_pack_is_the_oracles_to_the_bit(T, D, fmt, dtype):
    x = draw(T * 10007 + D, T, D, std=3.0, dtype=dtype)
    a = mc.act8_pack(x, fmt)
    out = mc.act8_unpack(a)
    out32 = mc.act8_unpack(a, dtype=F32)
    ok()
    want, scale = oa.act8(n64(x), fmt)
    nb = -(-D // 32)
    assert np.array_equal(a.scale.cpu().numpy()[:, :nb], scale)
    assert np.array_equal(values(a), want)
    assert np.array_equal(n64(out), want) and np.array_equal(n64(out32), want)
    assert out.shape == x.shape and out.dtype == BF


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_pack_at_the_ends_of_the_range(fmt):
    top = oa.TOP[fmt]
    rows = []
    for base in (2.0 ** -126, 1.0, top, top * 2.0 ** -120, top * 2.0 ** -121, top * 2.0 ** 110, 3.0e38, 1e-45, 0.0):
        for toward in (None, np.finfo(np.float32).max, 0.0):       # at the border, and on either side of it
            v = np.float32(base) if toward is None else np.nextafter(np.float32(base), np.float32(toward))
            row = np.zeros(64, np.float32)
            row[5] = v
            row[6:32] = v * np.linspace(-1, 1, 26)
            rows.append(row)
    x = torch.from_numpy(np.stack(rows)).to(DEV)
    a = mc.act8_pack(x, fmt)
    want, scale = oa.act8(n64(x), fmt)
    assert np.array_equal(a.scale.cpu().numpy()[:, :2], scale)
    assert np.array_equal(values(a), want)
    assert np.array_equal(n64(mc.act8_unpack(a, dtype=F32)), np.where(np.abs(want) < 2.0 ** 128, want, np.copysign(np.inf, want)))
    ok()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("D", [8, 249, 512, 510, 511, 600, 1024, 1030, 1276, 1277, 1280, 2300, 2301, 2304, 5000])
def test_pack_of_one_to_many_runs_a_row(D, fmt):
    """Rows of 1 to 20 runs of 256 columns, whole and not, in all three column layouts."""
    x = draw(D, 150, D)
    a = mc.act8_pack(x, fmt)
    want, scale = oa.act8(n64(x), fmt)
    assert np.array_equal(a.scale.cpu().numpy()[:, :-(-D // 32)], scale)
    assert np.array_equal(values(a), want)
    assert np.array_equal(n64(mc.act8_unpack(a)), want) and np.array_equal(n64(mc.act8_unpack(a, dtype=F32)), want)
    ok()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("D", [96, 97, 98])
def test_a_nan_or_infinity_costs_its_block_alone(fmt, D):
    x = draw(5, 6, D)
    x[1, 3], x[2, 40], x[3, 95], x[4, 64] = float("nan"), float("inf"), float("-inf"), float("nan")
    a = mc.act8_pack(x, fmt)
    got = n64(mc.act8_unpack(a))
    want, _ = oa.act8(n64(x), fmt)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.isnan(got).sum() == 4 * 32
    assert np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])
    ok()


def test_pack_leaves_the_padding_and_takes_any_leading_shape():
    x = draw(6, 2, 3, 70)
    a = mc.act8_empty(x.shape, "int8")
    a.q.fill_(77)
    a.scale.fill_(78)
    assert mc.act8_pack(x, "e4m3", out=a) is a          # out's own format holds
    want, scale = oa.act8(n64(x).reshape(6, 70), "int8")
    assert np.array_equal(values(a), want)
    assert (a.q[:, 70:] == 77).all() and (a.scale[:, 3:] == 78).all()
    assert mc.act8_unpack(a).shape == x.shape
    for T in (0,):
        e = mc.act8_pack(torch.empty(T, 64, dtype=BF, device=DEV))
        assert mc.act8_unpack(e).shape == (0, 64)
    ok()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("D", [256, 250, 251])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_pack_of_any_bits(dtype, D, fmt):
    """Random bit patterns: every exponent, subnormals, infinities and NaN."""
    bits = torch.randint(-2 ** 31, 2 ** 31, (200, D), generator=gen(D), device=DEV, dtype=torch.int64).to(torch.int32)
    bits[100:] = (bits[100:] & 0x007FFFFF) | (torch.randint(100, 140, (100, 1), generator=gen(1), device=DEV).to(torch.int32) << 23)
    x = bits.view(F32) if dtype == F32 else (bits >> 16).to(torch.int16).view(BF)
    x = x.contiguous()
    a = mc.act8_pack(x, fmt)
    want, scale = oa.act8(n64(x), fmt)
    assert np.array_equal(a.scale.cpu().numpy()[:, :-(-D // 32)], scale)
    got = values(a)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])
    out = n64(mc.act8_unpack(a, dtype=F32))
    want = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want)
    assert np.array_equal(out[~np.isnan(want)], want[~np.isnan(want)]) and np.array_equal(np.isnan(out), np.isnan(want))
    ok()


@pytest.mark.parametrize("D", [64, 66, 67])
def test_residual_sum_of_any_bits(D):
    """h = x + residual rounds as the fp32 sum does, whatever the two bf16 numbers."""
    a, b = (torch.randint(-2 ** 15, 2 ** 15, (4000, D), generator=gen(s), device=DEV, dtype=torch.int32).to(torch.int16) for s in (1, 2))
    b[:2000] = (b[:2000] & 0x7F) | (a[:2000] & 0x7F80) ^ (b[:2000] & 0x0780)      # near exponents too
    x, r = a.contiguous().view(BF), b.contiguous().view(BF)
    h = mc.rms_norm(x, torch.ones(D, dtype=BF, device=DEV), residual=r).h
    want = (x.float() + r.float()).to(BF)
    nan = torch.isnan(want)
    assert torch.equal(nan, torch.isnan(h)) and torch.equal(h[~nan].view(torch.int16), want[~nan].view(torch.int16))


def test_every_code_unpacks():
    codes = torch.arange(256, dtype=torch.int32, device=DEV).to(torch.uint8).repeat(9, 1).contiguous()
    scale = torch.zeros(9, 16, dtype=torch.uint8, device=DEV)
    for i, s in enumerate((0, 1, 7, 126, 127, 128, 200, 254, 255)):
        scale[i] = s
    for fmt in ("e4m3", "int8"):
        a = mc.Act8(codes, scale, (9, 256), fmt)
        got, want = n64(mc.act8_unpack(a, dtype=F32)), values(a)
        want = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)]), fmt


# -------------------------------------------------------------------- norm
def check_norm(x, r, w, fmt, eps=1e-6):
    h, y, rstd = mc.rms_norm(x, w, residual=r, eps=eps, fmt=fmt)
    ok()
    h_want = x if r is None else (x.float() + r.float()).to(x.dtype)
    assert torch.equal(h, h_want)
    D = x.shape[-1]
    y_want, rstd_want = oa.rms_norm(n64(h_want).reshape(-1, D), n64(w), eps)
    # the sum of squares: at most 32 terms a thread, then trees of 5 + 32 steps; rstd and y a few operations more
    fp = 80 * 2.0 ** -24
    within(n64(rstd), rstd_want, fp * rstd_want, "rstd")
    if fmt is None:
        assert y.dtype == BF
        within(n64(y).reshape(-1, D), y_want, (2.0 ** -8 + 2 * fp) * np.abs(y_want) + 2.0 ** -134, "y")
        return
    got = values(y)
    nb = -(-D // 32)
    scale = np.repeat(np.ldexp(1.0, y.scale.cpu().numpy()[:, :nb].astype(np.int64) - 127), 32, axis=1)[:, :D]
    half = np.maximum(2.0 ** -4 * np.abs(y_want), 2.0 ** -10 * scale) if fmt == "e4m3" else 0.5 * scale
    within(got, y_want, half * (1 + 2 * fp) + 2 * fp * np.abs(y_want), "y8")
    want_scale = oa.act8(y_want, fmt)[1]
    differ = y.scale.cpu().numpy()[:, :nb] != want_scale
    if differ.any():       # only where the block's maximum lies at a border of two exponents
        pad = np.zeros((y_want.shape[0], nb * 32))
        pad[:, :D] = np.abs(y_want)
        amax = pad.reshape(-1, nb, 32).max(axis=2)[differ]
        ratio = amax / oa.TOP[fmt]
        assert np.all(np.abs(np.exp2(np.rint(np.log2(ratio))) / ratio - 1) <= 4 * fp)


@pytest.mark.parametrize("fmt", [None, "e4m3", "int8"])
@pytest.mark.parametrize("T,D", [(1, 4096), (1, 1), (3, 8), (5, 100), (2, 255), (9, 264), (700, 128), (3, 777), (2000, 520), (1300, 1024),
                                 (2, 8192), (700, 5000), (3, 8200), (2, 16384), (2, 32768), (1, 32767), (700, 1594), (2, 16390)])
def test_norm(T, D, fmt):
    x, r = draw(T + D, T, D), draw(T + D + 1, T, D)
    w = 1 + 0.2 * draw(3, D).float()
    check_norm(x, r if (T + D) % 2 else None, w.to(BF), fmt)


@pytest.mark.parametrize("fmt", [None, "int8"])
@pytest.mark.parametrize("T,D", [(1, 4096), (5, 99), (700, 136), (4, 8192), (3, 20000), (400, 510)])
def test_norm_in_fp32(T, D, fmt):
    x, r = draw(T + D, T, D, dtype=F32), draw(T + D + 1, T, D, dtype=F32)
    check_norm(x, r, 1 + 0.2 * draw(3, D, dtype=F32), fmt)
    check_norm(x, None, (1 + 0.2 * draw(3, D, dtype=F32)).to(BF), fmt)


def test_norm_of_zero_rows_and_bad_rows():
    x = draw(8, 6, 512)
    x[1] = 0
    x[2, 100] = float("nan")
    x[3, 200] = float("inf")
    w = torch.ones(512, dtype=BF, device=DEV)
    _, y, rstd = mc.rms_norm(x, w, fmt="e4m3")
    got = n64(mc.act8_unpack(y))
    clean = [0, 4, 5]
    want, _ = oa.rms_norm(n64(x)[clean], np.ones(512), 1e-6)
    assert np.allclose(got[clean], want, rtol=0.07, atol=0.02)      # e4m3's half step, 2^-4
    assert (got[1] == 0).all() and abs(float(rstd[1]) - 1000.0) < 0.01   # 1 / sqrt(eps)
    assert np.isnan(got[2]).all()
    assert np.isnan(got[3, 192:224]).all() and (np.delete(got[3], np.arange(192, 224)) == 0).all() and rstd[3] == 0
    empty = mc.rms_norm(torch.empty(0, 512, dtype=BF, device=DEV), w, fmt="int8")
    assert empty.y.shape == (0, 512) and empty.rstd.numel() == 0
    ok()


def test_norm_in_place_of_its_inputs():
    x, r, w = draw(9, 50, 640), draw(10, 50, 640), draw(11, 640)
    want = mc.rms_norm(x, w, residual=r, fmt="int8")
    for target in (0, 1):
        xs = [x.clone(), r.clone()]
        h, y, rstd = mc.rms_norm(xs[0], w, residual=xs[1], fmt="int8", h_out=xs[target])
        assert h is xs[target] and torch.equal(h, want.h) and torch.equal(rstd, want.rstd)
        assert torch.equal(mc.act8_unpack(y), mc.act8_unpack(want.y))
    with pytest.raises(ValueError):
        mc.rms_norm(x, w, h_out=r)
    ok()


def check_norm_backward(T, D, dtype, kept, with_dh, wdtype=BF):
    h, dy = draw(T + D, T, D, dtype=dtype), draw(T + D + 1, T, D, std=1e-2, dtype=dtype)
    dh = draw(T + D + 2, T, D, std=1e-2, dtype=dtype) if with_dh else None
    w = (1 + 0.2 * draw(3, D, dtype=F32)).to(wdtype)
    rstd = torch.rsqrt(h.float().square().mean(dim=1) + 1e-6)
    kept_h = mc.act8_pack(h, kept) if kept else h
    dx, dw = mc.rms_norm_backward(dy, kept_h, w, rstd, dh=dh)
    ok()
    h64 = values(kept_h) if kept else n64(h)
    r, dy64, w64 = n64(rstd)[:, None], n64(dy), n64(w)
    want_dx, want_dw = oa.rms_norm_backward(dy64, h64, w64, n64(rstd), None if dh is None else n64(dh))
    xhat = h64 * r
    mean = np.abs(dy64 * w64 * xhat).mean(axis=1, keepdims=True)
    size = r * (np.abs(dy64 * w64) + np.abs(xhat) * mean) + (0 if dh is None else np.abs(n64(dh)))
    # the row's dot product: 32 terms a thread, trees of 5 + 32; then a few operations
    within(n64(dx), want_dx, 80 * 2.0 ** -24 * size + (2.0 ** -8 * np.abs(want_dx) if dtype == BF else 0) + 2.0 ** -134, "dx")
    within(n64(dw), want_dw, (T + 64) * 2.0 ** -24 * np.abs(dy64 * xhat).sum(axis=0) + 2.0 ** -140, "dw")


@pytest.mark.parametrize("kept", [None, "e4m3", "int8"])
@pytest.mark.parametrize("T,D", [(1, 1), (1, 4096), (7, 100), (777, 1000), (1500, 128), (2500, 64), (40, 2056), (700, 4096), (30, 8192), (9, 4100), (5, 16384),
                                 (3, 32768), (2, 9001), (900, 1594), (3, 5002), (4, 10002)])
def test_norm_backward(T, D, kept):
    check_norm_backward(T, D, BF, kept, (T + D) % 2 == 0)


@pytest.mark.parametrize("kept", [None, "int8"])
@pytest.mark.parametrize("T,D", [(5, 99), (600, 264), (20, 4096), (9, 8192), (3, 12000), (300, 510)])
def test_norm_backward_in_fp32(T, D, kept):
    check_norm_backward(T, D, F32, kept, True, F32)


def test_norm_backward_in_place_and_without_rows():
    h, dy, dh, w = draw(1, 70, 512), draw(2, 70, 512), draw(3, 70, 512), draw(4, 512)
    rstd = mc.rms_norm(h, w).rstd
    want = mc.rms_norm_backward(dy, h, w, rstd, dh=dh)
    for target in (0, 1):
        t = [dy.clone(), dh.clone()]
        dx, dw = mc.rms_norm_backward(t[0], h, w, rstd, dh=t[1], dx_out=t[target])
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1]) and dx is t[target]
    dx, dw = mc.rms_norm_backward(dy[:0], h[:0], w, rstd[:0])
    assert dx.shape == (0, 512) and (dw == 0).all()
    ok()


# --------------------------------------------------------- weight gradients
def check_grad(got, dy64, x64, dtype, base=None):
    want, size = dy64.T @ x64, np.abs(dy64).T @ np.abs(x64)
    rows = max(dy64.shape[0], 1)
    bound = (rows + 64) * 2.0 ** -23 * size
    if base is not None:
        want = want + base
        bound = bound + 2.0 ** -23 * np.abs(want) + 2.0 ** -23 * size
    if dtype == BF:
        bound = bound + 2.0 ** -8 * np.abs(want)
    within(n64(got), want, bound + 2.0 ** -134, "grad")


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,M,N", [(1, 8, 16), (1, 1, 1), (63, 256, 256), (64, 64, 72), (65, 300, 40), (129, 7, 100), (200, 257, 513),
                                   (1000, 512, 256), (31, 1000, 33), (700, 130, 1001), (4096, 64, 64), (9000, 256, 128)])
def test_weight_grad(T, M, N, dtype, fmt):
    dy, x = draw(T + M, T, M, std=1e-2), mc.act8_pack(draw(T + N, T, N), fmt)
    g = mc.weight_grad(dy, x, dtype=dtype)
    ok()
    assert g.shape == (M, N) and g.dtype == dtype
    check_grad(g, n64(dy), values(x), dtype)


@pytest.mark.parametrize("T,M,N", [(70, 264, 128), (5000, 96, 40), (12000, 512, 256), (9000, 1280, 2056), (300, 33, 65)])
def test_weight_grad_accumulates(T, M, N):
    dy, x = draw(T, T, M, std=1e-2), mc.act8_pack(draw(T + 1, T, N), "int8")
    base = draw(T + 2, M, N, dtype=F32)
    g = base.clone()
    assert mc.weight_grad(dy, x, out=g, accumulate=True) is g
    ok()
    check_grad(g, n64(dy), values(x), F32, n64(base))
    again = base.clone()
    mc.weight_grad(dy, x, out=again, accumulate=True)
    assert torch.equal(g, again)                           # whatever ran beside it
    none = base.clone()
    mc.weight_grad(dy[:0], mc.act8_empty((0, N)), out=none, accumulate=True)
    assert torch.equal(none, base)
    assert (mc.weight_grad(dy[:0], mc.act8_empty((0, N))) == 0).all()
    ok()


def test_long_fp32_sums_keep_their_precision():
    """65,536 rows of one sign: each addition of a lone fp32 accumulator would be off
    the same way.  An accumulator's 4096 rows are 256 tensor-core steps of up to
    2^-23, and the 16 chunks are added with 2^-24 each: 2^-15 in all (the plain
    sum of 4096 steps would be allowed 2^-11)."""
    T, M, N = 65536, 256, 256
    dy = (torch.rand(T, M, generator=gen(1), device=DEV) + 0.5).to(BF)
    x = mc.act8_pack((torch.rand(T, N, generator=gen(2), device=DEV) + 0.5).to(BF), "int8")
    g = mc.weight_grad(dy, x, dtype=F32)
    want = dy.double().t() @ mc.act8_unpack(x).double()
    assert float(((g.double() - want).abs() / want).max()) <= 2.0 ** -15
    ok()


def test_nan_rows_reach_their_own_entries_alone():
    dy, x = draw(1, 100, 64), draw(2, 100, 96)
    dy[3, 10] = float("nan")
    x[7, 40] = float("inf")
    g = mc.weight_grad(dy, mc.act8_pack(x, "e4m3"), dtype=F32)
    bad = torch.isnan(g)
    want = torch.zeros_like(bad)
    want[10, :] = True
    want[:, 32:64] = True
    assert torch.equal(bad, want)


# ------------------------------------------------------------------ experts
def routing(seed, T, K, E, drop=0.05, dtype=torch.int64):
    g = gen(seed)
    score = torch.randn(E, generator=g, device=DEV) + torch.randn(T, E, generator=g, device=DEV)
    top, idx = torch.topk(score, K, dim=1)
    idx = torch.where(torch.rand(T, K, generator=g, device=DEV) < drop, torch.full_like(idx, -1), idx)
    return idx.to(dtype), torch.softmax(top, dim=1)


def check_sort(idx, E):
    plan = mc.expert_sort(idx, E)
    ok()
    offsets, source, position = oa.expert_sort(idx.cpu().numpy(), E)
    assert np.array_equal(plan.offsets.cpu().numpy(), offsets)
    assert np.array_equal(plan.source.cpu().numpy(), source)
    assert np.array_equal(plan.position.cpu().numpy(), position)
    return plan


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("T,K,E", [(1, 1, 1), (1, 8, 64), (5, 2, 3), (256, 8, 64), (257, 8, 60), (1024, 2, 1024), (3000, 4, 128), (20000, 8, 16),
                                   (70000, 3, 40)])
def test_sort(T, K, E, dtype):
    check_sort(routing(T, T, K, E, dtype=dtype)[0], E)


def test_sort_of_unlike_loads():
    one = torch.full((3000, 2), 5, dtype=torch.int64, device=DEV)          # every pair to one expert, twice per token
    check_sort(one, 9)
    check_sort(torch.full((300, 2), -1, dtype=torch.int64, device=DEV), 4)    # all dropped
    odd = torch.tensor([[0, 4], [-7, 3], [2 ** 40, 1], [-2 ** 63, 2], [3, 2 ** 63 - 1]], dtype=torch.int64, device=DEV)
    check_sort(odd, 4)                                                      # far outside: dropped, not wrapped
    empty = mc.expert_sort(torch.empty(0, 2, dtype=torch.int64, device=DEV), 4)
    assert empty.offsets.tolist() == [0] * 5 and empty.position.shape == (0, 2)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,K,E,D", [(1, 1, 2, 8), (1, 8, 64, 7168), (48, 8, 64, 1000), (130, 2, 4, 33), (33, 6, 16, 1), (9, 40, 50, 264), (500, 4, 8, 513), (60, 3, 8, 1598), (7, 2, 4, 30)])
def test_gather_combine_and_gradient(T, K, E, D, dtype):
    idx, weights = routing(T + D, T, K, E)
    plan = check_sort(idx, E)
    x = draw(1, T, D, dtype=dtype)
    rows = torch.full((T * K, D), 7.0, dtype=dtype, device=DEV)
    assert mc.expert_gather(x, plan, out=rows) is rows
    src, pos, live = plan.source.cpu().numpy(), plan.position.cpu().numpy(), int(plan.offsets[-1])
    assert np.array_equal(n64(rows)[:live], n64(x)[src[:live] // K])
    assert (rows[live:] == 7.0).all()                       # behind the last row: as it was
    y = draw(2, T * K, D, dtype=dtype)
    y[live:] = float("nan")                                 # and never read
    y64, w64 = n64(y), n64(weights)
    eps = 2.0 ** -8 if dtype == BF else 0.0
    for w in (weights, None):
        ww = w64 if w is not None else np.ones_like(w64)
        out = mc.expert_combine(y, plan, w)
        want = oa.expert_combine(y64, pos, ww)
        size = oa.expert_combine(np.abs(np.nan_to_num(y64)), pos, ww)
        within(n64(out), want, (K + 1) * 2.0 ** -24 * size + eps * np.abs(want) + 2.0 ** -134, "combine")
    dout = draw(3, T, D, std=1e-2, dtype=dtype)
    dy = torch.full((T * K, D), 5.0, dtype=dtype, device=DEV)
    _, dw = mc.expert_combine_backward(dout, y, plan, weights, out=dy)
    want_dy, want_dw = oa.expert_combine_backward(n64(dout), y64, pos, w64, np.full((T * K, D), 5.0))
    within(n64(dy), want_dy, (2.0 ** -24 + eps) * np.abs(want_dy) + 2.0 ** -134, "dy")
    size = oa.expert_combine_backward(np.abs(n64(dout)), np.abs(y64), pos, w64, np.zeros((T * K, D)))[1]
    within(n64(dw), want_dw, (D + 2) * 2.0 ** -24 * size + 2.0 ** -140, "dweights")
    same = y.clone()                                        # dy in the place of y
    dy2, dw2 = mc.expert_combine_backward(dout, same, plan, weights, out=same)
    assert torch.equal(dy2[:live], dy[:live]) and torch.equal(dw2, dw)
    ok()


def test_positions_outside_the_rows_are_dropped():
    x = draw(1, 4, 64)
    position = torch.tensor([[0, 99], [-5, 3], [8, 1], [2, 7]], dtype=torch.int32, device=DEV)
    plan = mc.ExpertPlan(torch.tensor([0, 8], dtype=torch.int32, device=DEV), torch.zeros(8, dtype=torch.int32, device=DEV), position)
    rows = mc.expert_gather(x, plan, out=torch.zeros(8, 64, dtype=BF, device=DEV))
    want = torch.zeros_like(rows)
    for r, t in ((0, 0), (3, 1), (1, 2), (2, 3), (7, 3)):
        want[r] = x[t]
    assert torch.equal(rows, want)
    out = mc.expert_combine(rows, plan)
    assert torch.equal(out[0], x[0]) and torch.equal(out[2], x[2])
    dy, dw = mc.expert_combine_backward(x, rows, plan, torch.ones(4, 2, device=DEV))
    assert dw[0, 1] == 0 and dw[1, 0] == 0 and dw[2, 0] == 0 and torch.equal(dy[7], x[3])
    ok()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,K,E,M,N", [(1, 1, 3, 8, 16), (40, 2, 4, 64, 96), (100, 8, 64, 40, 48), (333, 2, 5, 300, 520), (64, 1, 2, 7, 33),
                                       (2000, 2, 3, 264, 136), (13000, 2, 3, 64, 72)])
def test_expert_weight_grad(T, K, E, M, N, dtype):
    idx, _ = routing(T + M, T, K, E)
    idx[idx == E - 1] = -1                                   # the last expert has no rows
    plan = check_sort(idx, E)
    live, off = int(plan.offsets[-1]), plan.offsets.tolist()
    dy = draw(1, T * K, M, std=1e-2)
    dy[live:] = float("nan")                                 # behind the last expert's rows
    x = mc.act8_pack(draw(2, T, N), "int8")
    g = mc.expert_weight_grad(dy, x, plan, gather=True, dtype=dtype)
    ok()
    xs, dy64 = values(x)[plan.source.cpu().numpy().clip(0) // K], n64(dy)
    for e in range(E):
        check_grad(g[e], dy64[off[e]:off[e + 1]], xs[off[e]:off[e + 1]], dtype)
    assert (g[E - 1] == 0).all()
    xr = draw(3, T * K, N)
    xr[live:] = float("inf")
    x8 = mc.act8_pack(xr, "e4m3")
    base = draw(4, E, M, N, dtype=F32)
    g = base.clone()
    mc.expert_weight_grad(dy, x8, plan, gather=False, out=g, accumulate=True)
    ok()
    xs = values(x8)
    for e in range(E):
        check_grad(g[e], dy64[off[e]:off[e + 1]], xs[off[e]:off[e + 1]], F32, n64(base[e]))
    assert torch.equal(g[E - 1], base[E - 1])


def test_one_experts_nan_stays_with_it():
    T, E = 90, 3
    idx = (torch.arange(T, device=DEV) % E).view(T, 1).to(torch.int64)      # 30 rows each: every boundary inside 64 rows
    plan = mc.expert_sort(idx, E)
    dy, x = draw(1, T, 64), draw(2, T, 64)
    dy[30:60] = float("nan")
    x8 = mc.act8_pack(x, "int8")
    g = mc.expert_weight_grad(dy, x8, plan, gather=True, dtype=F32)
    assert torch.isnan(g[1]).all() and torch.isfinite(g[0]).all() and torch.isfinite(g[2]).all()
    ok()


def test_offsets_outside_the_rows_are_clamped():
    dy, x8 = draw(1, 32, 16), mc.act8_pack(draw(2, 32, 16), "int8")
    plan = mc.ExpertPlan(torch.tensor([-9, 20, 5, 400], dtype=torch.int32, device=DEV), torch.arange(32, dtype=torch.int32, device=DEV),
                         torch.arange(32, dtype=torch.int32, device=DEV).view(32, 1))
    g = mc.expert_weight_grad(dy, x8, plan, gather=False, dtype=F32)
    xs = values(x8)
    check_grad(g[0], n64(dy)[:20], xs[:20], F32)
    assert (g[1] == 0).all()
    check_grad(g[2], n64(dy)[5:], xs[5:], F32)
    ok()

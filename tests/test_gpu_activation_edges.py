"""GPU tests of the activation operators where their results are decided exactly:
8-bit outputs of the norm at the borders of scales and codes, long sums of one
sign, pairs dropped after the sort, every path of the sort, and captured packing."""
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
    return (torch.randn(*shape, generator=gen(seed), device=DEV) * std).to(dtype)


def n64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def ok():
    assert mc.device_status() == mc.MC_OK, mc.last_error()


def stored(a):
    """(values, scale bytes) of an Act8, as the oracle reads them."""
    D = a.shape[-1]
    s = a.scale.cpu().numpy()
    return oa.act8_values(a.q.cpu().numpy(), s, D, a.fmt), s[:, :-(-D // 32)]


# ------------------------------------------------------- bf16 and fp32 sums
def one_signed(seed, rows, cols):
    return (torch.rand(rows, cols, generator=gen(seed), device=DEV) + 0.5).to(BF)


def check_long_sum(g, want):
    """fp32: 1024 rows are 64 tensor-core steps, each off by at most 2^-23 of the sum, and
    up to 64 chunks are added with 2^-24 each: 2^-17 + 2^-18.  bf16: 2048 rows are 128 steps,
    up to 32 chunks: 2^-16 + 2^-19, and half a step of bf16 on top."""
    bound = (2.0 ** -17 + 2.0 ** -18) * want
    if g.dtype == BF:
        bound = (2.0 ** -16 + 2.0 ** -19) * want + torch.exp2(torch.floor(torch.log2(want)) - 8)
    assert bool(((g.double() - want).abs() <= bound).all()), float(((g.double() - want).abs() - bound).max())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_sums_of_one_experts_whole_tiles(dtype):
    """One expert has all 65,536 rows: experts' contractions are never split, so each tile's
    sum runs over all of them."""
    T, M, N = 65536, 256, 256
    dy = one_signed(1, T, M)
    x = mc.act8_pack(one_signed(2, T, N), "int8")
    plan = mc.expert_sort(torch.zeros(T, 1, dtype=torch.int32, device=DEV), 1)
    want = dy.double().t() @ mc.act8_unpack(x).double()
    for gather in (True, False):
        check_long_sum(mc.expert_weight_grad(dy, x, plan, gather=gather, dtype=dtype)[0], want)
    ok()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_sums_of_split_tiles(dtype):
    """One tile for 74 SM pairs: its contraction is cut into ranges, which are joined."""
    T, M, N = 65536, 256, 256
    dy = one_signed(5, T, M)
    x = mc.act8_pack(one_signed(6, T, N), "e4m3")
    check_long_sum(mc.weight_grad(dy, x, dtype=dtype), dy.double().t() @ mc.act8_unpack(x).double())
    ok()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_sums_of_one_weights_whole_tiles(dtype):
    """2 x 37 tiles are one whole wave of the 74 SM pairs: none of them is split."""
    T, M, N = 65536, 512, 37 * 256
    dy = one_signed(3, T, M)
    x = mc.act8_empty((T, N), "int8", device=DEV)
    x.q.random_(64, 128, generator=gen(4))
    x.scale.fill_(120)
    g = mc.weight_grad(dy, x, dtype=dtype)
    some = torch.arange(5, N, 61, device=DEV)
    want = dy.double().t() @ (x.q[:, some].double() * 2.0 ** -7)
    check_long_sum(g[:, some], want)
    ok()


# ------------------------------------------------------------ dropped pairs
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,K,E,M,N", [(300, 2, 4, 64, 96), (130, 8, 9, 40, 33), (1000, 1, 3, 264, 520), (70, 3, 2, 33, 64), (2000, 4, 5, 128, 2056)])
def test_experts_gradient_without_pairs_dropped_after_the_sort(T, K, E, M, N, dtype):
    """Positions set outside the rows after the sort (an expert over its capacity): those
    pairs add nothing, whatever their rows of dy and the scratch hold."""
    g = gen(T)
    plan = mc.expert_sort(torch.randint(-1, E, (T, K), generator=g, device=DEV), E)
    off = plan.offsets.tolist()
    gone = torch.rand(T, K, generator=g, device=DEV) < 0.2
    gone |= (plan.position >= off[1]) & (plan.position < off[2])            # expert 1 loses every pair
    lost = plan.position[gone & (plan.position >= 0)].long()
    away = torch.tensor([-1, T * K, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=DEV)[torch.randint(0, 4, (T, K), generator=g, device=DEV)]
    kept = plan._replace(position=torch.where(gone, away, plan.position))
    dy = draw(T + 1, T * K, M)
    dy[lost] = float("nan")
    x = mc.act8_pack(draw(T + 2, T, N), "e4m3")
    x64, _ = stored(x)
    src, reached = plan.source.cpu().numpy().clip(0) // K, np.zeros(T * K, bool)
    pos = kept.position.cpu().numpy().reshape(-1)
    reached[pos[(pos >= 0) & (pos < T * K)]] = True
    need = mc.load_library().mc_expert_weight_grad_workspace_size(T * K, E, M, N)
    base = draw(T + 3, E, M, N, dtype=F32)
    for accumulate in ((False, True) if dtype == F32 else (False,)):
        ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)        # bf16 NaN
        out = base.clone() if accumulate else None
        got = n64(mc.expert_weight_grad(dy, x, kept, gather=True, dtype=dtype, out=out, accumulate=accumulate, workspace=ws))
        ok()
        for e in range(E):
            r = np.arange(off[e], off[e + 1])
            r = r[reached[r]]
            a, b = n64(dy)[r], x64[src[r]]
            want, size = a.T @ b, np.abs(a).T @ np.abs(b)
            bound = (len(r) + 64) * 2.0 ** -23 * size
            if accumulate:
                want = want + n64(base[e])
                bound = bound + 2.0 ** -23 * (np.abs(want) + size)
            if dtype == BF:
                bound = bound + 2.0 ** -8 * np.abs(want)
            assert np.all(np.abs(got[e] - want) <= bound + 2.0 ** -134), e
        assert accumulate or (got[1] == 0).all()


def test_a_captured_experts_gradient_follows_the_positions():
    """Replayed with pairs dropped, with others dropped, and with all of them back."""
    T, K, E, M, N = 500, 2, 3, 64, 72
    plan = mc.expert_sort(torch.randint(0, E, (T, K), generator=gen(1), device=DEV), E)
    dy, x = draw(2, T * K, M), mc.act8_pack(draw(3, T, N), "int8")
    whole = plan.position.clone()
    want = mc.expert_weight_grad(dy, x, plan, gather=True)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = mc.expert_weight_grad(dy, x, plan, gather=True)
    for seed in (4, 5, None):
        gone = torch.rand(T, K, generator=gen(seed), device=DEV) < 0.3 if seed else torch.zeros_like(whole, dtype=torch.bool)
        plan.position.copy_(torch.where(gone, torch.full_like(whole, -1), whole))
        g.replay()
        torch.cuda.synchronize()
        if seed is None:
            assert torch.equal(got, want)
            continue
        zeroed = dy.clone()
        zeroed[whole[gone].long()] = 0                                      # whole plan, those rows as zeros: the same sums
        assert torch.equal(got, mc.expert_weight_grad(zeroed, x, plan._replace(position=whole), gather=True))
    ok()
    del g


# ------------------------------------------------- the norm's 8-bit borders
BORDERS = {"int8": [127 / 64, 126.5 / 64, 125.5 / 64, 1.0, 0.5 / 64, 1.5 / 64, 64.5 / 64, 3.5 / 64],
           "e4m3": [1.75, 1.6875, 1.0625, 1.1875, 17 / 1024, 19 / 1024, 2.0 ** -17, 1.5 * 2.0 ** -17, 1.0]}


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [8, 64, 1000, 4096, 66, 1594, 67, 1789, 8200])
def test_norm_at_the_borders_of_scales_and_codes(D, dtype, fmt):
    """Rows whose y = h rstd w is known exactly: +-c everywhere gives +-w (eps = 0), +-1
    with eps = 3 gives +-w / 2.  The weights stand at the largest value of a
    scale and in the middle of two codes: the least scale, and ties to even."""
    w = torch.tensor(BORDERS[fmt], device=DEV).repeat(D // len(BORDERS[fmt]) + 1)[:D]
    w = torch.where(torch.rand(D, generator=gen(D), device=DEV) < 0.5, -w, w)
    sizes = torch.tensor([1.0, 2.0 ** -3, 2.0 ** 7, 3.0, 5.0, 0.109375, 113.0, 1.3125], device=DEV)
    sign = torch.where(torch.rand(sizes.numel(), D, generator=gen(D + 1), device=DEV) < 0.5, -1.0, 1.0)
    for wdtype in (BF, F32):
        w_ = w.to(wdtype)
        for x, eps, factor in (((sign * sizes[:, None]).to(dtype), 0.0, 1.0), (sign.to(dtype), 3.0, 0.5)):
            y = mc.rms_norm(x, w_, eps=eps, fmt=fmt).y
            ok()
            got, scale = stored(y)
            want, want_scale = oa.act8(n64(sign) * n64(w)[None, :] * factor, fmt)
            assert np.array_equal(scale, want_scale), (wdtype, eps)
            assert np.array_equal(got, want), (wdtype, eps)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("D", [256, 258, 1024])
def test_norm_of_one_value_a_row(D, fmt):
    """c alone in a row: y = sqrt(D) w there (a power of two times w where D is one of four)."""
    x = torch.zeros(64, D, dtype=BF, device=DEV)
    col = torch.randint(0, D, (64,), generator=gen(D), device=DEV)
    c = draw(D + 1, 64)
    x[torch.arange(64, device=DEV), col] = c
    w = torch.full((D,), oa.TOP[fmt], dtype=BF, device=DEV)
    got, scale = stored(mc.rms_norm(x, w, eps=0.0, fmt=fmt).y)
    y = np.zeros((64, D))
    y[np.arange(64), col.cpu().numpy()] = np.sign(n64(c)) * np.sqrt(D) * oa.TOP[fmt]
    want, want_scale = oa.act8(y, fmt)
    assert np.array_equal(got, want) and np.array_equal(scale, want_scale)
    ok()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype,wdtype", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("T,D", [(600, 4096), (700, 1594), (700, 1789)])
def test_norm_rounds_the_product_itself(T, D, dtype, wdtype, fmt):
    """Every code is that of a product within 2^-21 of the formula's: the sums of eight
    squares round eight times at most, 2^-24 each, and the root halves that; everything
    behind is kept to more bits."""
    x, w = draw(T, T, D, std=2.0, dtype=dtype), (1 + 0.2 * draw(D, D, dtype=F32)).to(wdtype)
    y, _ = oa.rms_norm(n64(x), n64(w), 1e-6)
    got, scale = stored(mc.rms_norm(x, w, fmt=fmt).y)
    ok()
    lo, lo_scale = oa.act8(y * (1 - 2.0 ** -21), fmt)
    hi, hi_scale = oa.act8(y * (1 + 2.0 ** -21), fmt)
    assert ((scale == lo_scale) | (scale == hi_scale)).all()
    assert ((got == lo) | (got == hi)).all(), int(((got != lo) & (got != hi)).sum())


# ----------------------------------------------------------------- the sort
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("T,K,E", [(2048, 1, 64), (2049, 1, 64), (4096, 8, 64), (32769, 1, 60), (8192, 8, 64), (8192, 8, 1024), (16384, 8, 3),
                                   (131073, 1, 64)])
def test_sort_by_every_path(T, K, E, dtype):
    """One block; the cluster launch up to 32,768 pairs; counting and placing launches
    up to 131,072; with a scan between them beyond that."""
    idx = torch.randint(0, E, (T, K), generator=gen(T + E), device=DEV)
    idx = torch.where(torch.rand(T, K, generator=gen(T), device=DEV) < 0.05, torch.full_like(idx, -1), idx).to(dtype)
    idx[:3] = E                                                             # dropped too
    plan = mc.expert_sort(idx, E)
    ok()
    offsets, source, position = oa.expert_sort(idx.cpu().numpy(), E)
    assert np.array_equal(plan.offsets.cpu().numpy(), offsets)
    assert np.array_equal(plan.source.cpu().numpy(), source)
    assert np.array_equal(plan.position.cpu().numpy(), position)


# ---------------------------------------------------------- captured packing
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("D", [520, 514, 521])
def test_captured_pack_writes_every_code_and_scale(D, fmt):
    x = draw(D, 300, D)
    out = mc.act8_pack(x, fmt)
    want, scale = oa.act8(n64(x), fmt)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mc.act8_pack(x, fmt, out=out)
        back = mc.act8_unpack(out)
    for _ in range(2):
        out.q.zero_()
        out.scale.zero_()
        back.zero_()
        g.replay()
        torch.cuda.synchronize()
        got, got_scale = stored(out)
        assert np.array_equal(got, want) and np.array_equal(got_scale, scale) and np.array_equal(n64(back), want)
    ok()
    del g

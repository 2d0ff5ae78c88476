"""GPU tests of the activation operators where their results are decided exactly:
long sums of one sign."""
import pytest
import torch

import matrix_orthogonalising_optimizer_step_b200 as mc

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def ok():
    assert mc.device_status() == mc.MC_OK, mc.last_error()


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

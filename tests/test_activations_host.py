"""CPU tests of the activation operators' entry points: refusals before any
memory or GPU is touched, workspace queries, structure layout."""
import ctypes

import pytest
import torch

import matrix_orthogonalising_optimizer_step_b200 as mc
from matrix_orthogonalising_optimizer_step_b200 import build as mcbuild

P = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    mcbuild.build()
    return mc.load_library()


def act8(q=0x1000000, s=0x2000000, rows=8, cols=64, q_ld=64, s_ld=16, fmt=mc.MC_ACT_INT8):
    return mc.McAct8(q, s, rows, cols, q_ld, s_ld, fmt, 0)


X = 0x4000000
Y = 0x5000000
Z = 0x6000000
W = 0x7000000


def test_structure_size(lib):
    assert lib.mc_struct_size(16) == ctypes.sizeof(mc.McAct8)


@pytest.mark.parametrize("bad, code", [
    (dict(fmt=3), mc.MC_ERR_INVAL), (dict(cols=0), mc.MC_ERR_INVAL), (dict(rows=-1), mc.MC_ERR_INVAL),
    (dict(rows=1 << 31), mc.MC_ERR_INVAL), (dict(q_ld=72), mc.MC_ERR_INVAL), (dict(q_ld=48), mc.MC_ERR_INVAL),
    (dict(s_ld=8), mc.MC_ERR_INVAL), (dict(cols=1024, q_ld=1024, s_ld=16), mc.MC_ERR_INVAL), (dict(q=None), mc.MC_ERR_INVAL),
    (dict(q_ld=1 << 31), mc.MC_ERR_INVAL), (dict(s_ld=1 << 31), mc.MC_ERR_INVAL),
    (dict(q=0x1000008), mc.MC_ERR_ALIGN), (dict(s=0x2000004), mc.MC_ERR_ALIGN)])
def test_bad_act8_is_refused_everywhere(lib, bad, code):
    a = act8(**bad)
    assert lib.mc_act8_pack(X, mc.MC_BF16, P(a), None) == code
    assert lib.mc_act8_unpack(P(a), X, mc.MC_BF16, None) == code
    assert lib.mc_weight_grad(X, P(a), 64, Y, mc.MC_F32, 0, None, 0, None) == code
    assert lib.mc_rms_norm(X, None, W, mc.MC_BF16, mc.MC_BF16, a.rows, a.cols, 1e-6, None, None, P(a), Z, None) < 0
    assert lib.mc_rms_norm_backward(X, None, None, P(a), W, Z, mc.MC_BF16, mc.MC_BF16, a.rows, a.cols, Y, Z + 4096, None, 0, None) < 0


def test_pack_and_unpack_refusals(lib):
    a = act8()
    assert lib.mc_act8_pack(X, 2, P(a), None) == mc.MC_ERR_INVAL
    assert lib.mc_act8_pack(None, mc.MC_BF16, P(a), None) == mc.MC_ERR_INVAL
    assert lib.mc_act8_pack(X + 2, mc.MC_BF16, P(a), None) == mc.MC_ERR_ALIGN
    assert lib.mc_act8_pack(a.q, mc.MC_BF16, P(a), None) == mc.MC_ERR_INVAL           # x is q
    assert lib.mc_act8_pack(a.scale - 16, mc.MC_BF16, P(a), None) == mc.MC_ERR_INVAL  # x runs into scale
    assert lib.mc_act8_unpack(P(a), a.q, mc.MC_F32, None) == mc.MC_ERR_INVAL
    assert lib.mc_act8_unpack(None, X, mc.MC_F32, None) == mc.MC_ERR_INVAL
    empty = act8(rows=0, q=None, s=None)
    assert lib.mc_act8_pack(None, mc.MC_BF16, P(empty), None) == mc.MC_OK             # no rows: a no-op
    assert lib.mc_act8_unpack(P(empty), None, mc.MC_BF16, None) == mc.MC_OK


def test_norm_refusals(lib):
    def norm(x=X, r=None, w=W, dt=mc.MC_BF16, wdt=mc.MC_BF16, rows=8, cols=64, eps=1e-6, h=None, y=Y, y8=None, rstd=Z):
        return lib.mc_rms_norm(x, r, w, dt, wdt, rows, cols, eps, h, y, P(y8) if y8 is not None else None, rstd, None)
    H = 0x8000000
    for bad in (dict(x=None), dict(w=None), dict(rstd=None), dict(y=None), dict(y8=act8()), dict(dt=5), dict(wdt=16),
                dict(cols=0), dict(cols=32769), dict(rows=-1), dict(eps=-1e-9), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(r=H), dict(h=H), dict(y=X), dict(r=H, h=Y),
                dict(y=None, y8=act8(rows=7)), dict(y=None, y8=act8(cols=48)), dict(r=H, h=X + 16), dict(rstd=X), dict(y=W)):
        assert norm(**bad) == mc.MC_ERR_INVAL, bad
    for bad in (dict(x=X + 8), dict(y=Y + 2), dict(w=W + 4), dict(rstd=Z + 4)):
        assert norm(**bad) == mc.MC_ERR_ALIGN, bad
    assert norm(rows=0, x=None, rstd=None) == mc.MC_OK


def test_norm_backward_refusals(lib):
    def back(dy=X, dh=None, h=Y, h8=None, w=W, rstd=Z, dt=mc.MC_BF16, wdt=mc.MC_BF16, rows=8, cols=64, dx=0x8000000,
             dw=0x9000000):
        return lib.mc_rms_norm_backward(dy, dh, h, P(h8) if h8 is not None else None, w, rstd, dt, wdt, rows, cols, dx, dw,
                                        None, 0, None)
    for bad in (dict(dy=None), dict(h=None), dict(rstd=None), dict(dx=None), dict(dw=None), dict(h8=act8()), dict(cols=40000),
                dict(h=None, h8=act8(rows=9)), dict(dx=Y), dict(dx=X + 16), dict(dw=X), dict(dx=W), dict(dt=1 << 20)):
        assert back(**bad) == mc.MC_ERR_INVAL, bad
    for bad in (dict(dy=X + 2), dict(dx=0x8000008), dict(dw=0x9000004)):
        assert back(**bad) == mc.MC_ERR_ALIGN, bad
    assert lib.mc_rms_norm_backward_workspace_size(-1, 64) == 0
    assert lib.mc_rms_norm_backward_workspace_size(8, 40000) == 0
    assert lib.mc_rms_norm_backward_workspace_size(0, 1) > 0


def test_weight_gradient_refusals_and_workspace(lib):
    def grad(dy=X, a=None, M=64, g=Y, dt=mc.MC_F32, acc=0):
        return lib.mc_weight_grad(dy, P(a or act8()), M, g, dt, acc, None, 0, None)
    for bad in (dict(dy=None), dict(M=0), dict(g=None), dict(dt=16), dict(dt=mc.MC_BF16, acc=1), dict(g=X), dict(g=0x1000000)):
        assert grad(**bad) == mc.MC_ERR_INVAL, bad
    for bad in (dict(dy=X + 2), dict(g=Y + 8)):
        assert grad(**bad) == mc.MC_ERR_ALIGN, bad
    size = lib.mc_weight_grad_workspace_size
    assert size(-1, 64, 64) == 0 and size(8, 0, 64) == 0 and size(8, 64, 0) == 0 and size(1 << 31, 64, 64) == 0
    assert size(1000, 64, 4096) >= 1000 * 4096 * 2                # the bf16 values of x
    assert size(1000, 63, 4096) >= size(1000, 64, 4096) + 1000 * 64 * 2 - 256   # and dy in whole 16-byte rows
    esize = lib.mc_expert_weight_grad_workspace_size
    assert esize(8, 0, 64, 64) == 0 and esize(8, 1025, 64, 64) == 0
    assert esize(8, 1024, 64, 64) >= 1024 * (2 * 128 + 8)         # two tensor maps and a row range each


def test_expert_refusals_and_workspace(lib):
    def sort(idx=X, bits=64, T=16, K=2, E=8, off=Y, src=Z, pos=W):
        return lib.mc_expert_sort(idx, bits, T, K, E, off, src, pos, None, 0, None)
    for bad in (dict(idx=None), dict(bits=16), dict(T=-1), dict(K=0), dict(K=1025), dict(E=0), dict(E=1025), dict(off=None),
                dict(src=None), dict(pos=None), dict(T=1 << 30, K=2), dict(src=X), dict(pos=Z), dict(off=Z)):
        assert sort(**bad) == mc.MC_ERR_INVAL, bad
    assert sort(src=Z + 4) == mc.MC_ERR_ALIGN
    assert lib.mc_expert_sort_workspace_size(1 << 30, 2, 8) == 0
    assert lib.mc_expert_sort_workspace_size(0, 2, 8) > 0

    def gather(x=X, dt=mc.MC_BF16, T=16, K=2, D=64, pos=Y, out=Z):
        return lib.mc_expert_gather(x, dt, T, K, D, pos, out, None)
    for bad in (dict(x=None), dict(dt=7), dict(T=-1), dict(K=0), dict(D=0), dict(pos=None), dict(out=None), dict(out=X),
                dict(out=X - 16), dict(out=Y)):
        assert gather(**bad) == mc.MC_ERR_INVAL, bad
    assert gather(out=Z + 2) == mc.MC_ERR_ALIGN
    assert gather(T=0, x=None, pos=None, out=None) == mc.MC_OK

    def combine(y=X, dt=mc.MC_BF16, T=16, K=2, D=64, pos=Y, w=Z, out=W):
        return lib.mc_expert_combine(y, dt, T, K, D, pos, w, out, None)
    for bad in (dict(y=None), dict(pos=None), dict(out=None), dict(out=X), dict(out=X + 64), dict(out=Z)):
        assert combine(**bad) == mc.MC_ERR_INVAL, bad
    assert combine(w=Z + 4) == mc.MC_ERR_ALIGN

    def back(dout=X, y=Y, dt=mc.MC_BF16, T=16, K=2, D=64, pos=Z, w=W, dy=0x8000000, dw=0x9000000):
        return lib.mc_expert_combine_backward(dout, y, dt, T, K, D, pos, w, dy, dw, None)
    for bad in (dict(dout=None), dict(y=None), dict(pos=None), dict(w=None), dict(dy=None), dict(dw=None), dict(dy=X),
                dict(dy=Y + 16), dict(dw=W), dict(dw=X)):
        assert back(**bad) == mc.MC_ERR_INVAL, bad

    def grad(dy=X, rows=16, a=None, off=Y, pos=Z, K=2, E=8, M=64, g=W, dt=mc.MC_F32, acc=0):
        return lib.mc_expert_weight_grad(dy, rows, P(a or act8()), off, pos, K, E, M, g, dt, acc, None, 0, None)
    for bad in (dict(off=None), dict(rows=15), dict(K=0), dict(K=3), dict(E=0), dict(E=1025), dict(pos=None),
                dict(pos=None, rows=9), dict(g=X), dict(g=Y), dict(dt=mc.MC_BF16, acc=1)):
        assert grad(**bad) == mc.MC_ERR_INVAL, bad
    assert grad(off=Y + 4) == mc.MC_ERR_ALIGN


def test_binding_refuses_host_tensors_and_bad_shapes():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    a = mc.Act8(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 16, dtype=torch.uint8), (4, 64), "int8")
    plan = mc.ExpertPlan(torch.zeros(3, dtype=torch.int32), torch.zeros(8, dtype=torch.int32), torch.zeros(4, 2, dtype=torch.int32))
    calls = [lambda: mc.act8_pack(x), lambda: mc.act8_unpack(a), lambda: mc.rms_norm(x, x[0]),
             lambda: mc.rms_norm_backward(x, x, x[0], torch.zeros(4)), lambda: mc.weight_grad(x, a),
             lambda: mc.expert_sort(torch.zeros(4, 2, dtype=torch.int64), 2), lambda: mc.expert_gather(x, plan),
             lambda: mc.expert_combine(x, plan), lambda: mc.expert_combine_backward(x, x, plan, torch.zeros(4, 2)),
             lambda: mc.expert_weight_grad(x, a, plan, gather=True)]
    for call in calls:
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="e4m3"):
        mc.act8_empty((4, 64), "fp8", "cpu")
    e = mc.act8_empty((2, 3, 70), "e4m3", "cpu")
    assert tuple(e.q.shape) == (6, 80) and tuple(e.scale.shape) == (6, 16) and e.shape == (2, 3, 70)
    with pytest.raises(TypeError, match="Act8"):
        mc.qk_max_logit_static(a, x, x, 1, 64)

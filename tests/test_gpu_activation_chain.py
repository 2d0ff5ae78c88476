"""GPU tests of the activation operators together and around the optimizer step:
a block and an expert layer from the norm to the Muon update, captured graphs,
other streams, indices past 32 bits, workspaces and alignment."""
import numpy as np
import pytest
import torch

import matrix_orthogonalising_optimizer_step_b200 as mc
import oracle
from oracle import activations as oa
from gpu_util import GAMMA_TOL, NS_TOL, SMAX_TOL, rel_fro, to64

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def draw(seed, *shape, std=1.0, dtype=BF):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def ok():
    assert mc.device_status() == mc.MC_OK, mc.last_error()


def muon_matches(W0, G, hp):
    """A Muon step on (W, G) against the oracle's on the same numbers."""
    W, M, U = W0.clone(), torch.zeros(W0.shape, device=DEV), torch.empty(W0.shape, device=DEV)
    mc.muon_step([W], [G], [M], update_outs=[U], **hp)
    ok()
    _, _, upd, _ = oracle.muon_step(to64(W0), to64(G), np.zeros(W0.shape), **hp)
    assert rel_fro(to64(U), upd) <= NS_TOL
    return W


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_attention_block_from_the_norm_to_the_step(hp, fmt):
    """x + r -> norm -> 8-bit layer input, kept; S_max and the clip from it; its
    projections' gradients from it; the Muon step on them; the norm's gradient."""
    B, S, D, H, dh = 2, 160, 128, 2, 64
    x, r, w = draw(1, B, S, D), draw(2, B, S, D), (1 + 0.1 * draw(3, D, dtype=F32)).to(BF)
    wq, wk = draw(4, H * dh, D, std=0.3), draw(5, H * dh, D, std=0.3)
    h, y, rstd = mc.rms_norm(x, w, residual=r, fmt=fmt)
    y64 = oa.act8_values(y.q.cpu().numpy(), y.scale.cpu().numpy(), D, fmt)
    smax = mc.qk_max_logit(y, wq, wk, H, dh)
    want = oracle.qk_max_logit(y64.reshape(B, S, D), to64(wq), to64(wk), H, dh)
    assert np.all(np.abs(to64(smax) - want) <= SMAX_TOL * np.abs(want))
    assert torch.equal(smax, mc.qk_max_logit(mc.act8_unpack(y), wq, wk, H, dh))
    tau = float(np.mean(want))
    gamma, mask = mc.qk_clip(wq.clone(), wk.clone(), smax, H, dh, tau=tau)
    _, _, og, om = oracle.qk_clip(to64(wq), to64(wk), want, tau, 0.5, H, dh)
    assert list(mask.cpu().numpy()) == list(om) and np.all(np.abs(to64(gamma) - og) <= GAMMA_TOL * og)
    dq = draw(6, B, S, H * dh, std=1e-2)
    G = mc.weight_grad(dq, y)
    g64 = to64(dq).reshape(-1, H * dh).T @ y64
    assert rel_fro(to64(G), g64) <= 2.0 ** -8            # one rounding to bf16 of each entry
    muon_matches(wq, G, hp)
    acc = mc.weight_grad(dq, y, dtype=F32)               # a second micro-batch on top
    mc.weight_grad(dq, y, out=acc, accumulate=True)
    assert rel_fro(to64(acc), 2 * g64) <= 1e-5
    muon_matches(wq, acc, hp)
    dy = (dq.float().reshape(-1, H * dh) @ wq.float()).to(BF).reshape(B, S, D)
    dx, dw = mc.rms_norm_backward(dy, mc.act8_pack(h, "int8"), w, rstd, dh=draw(7, B, S, D, std=1e-2))
    assert dx.shape == x.shape and dw.shape == (D,) and torch.isfinite(dx).all() and torch.isfinite(dw).all()
    ok()


def test_mla_max_logit_takes_an_8_bit_input():
    H, dc, dr, D = 2, 64, 32, 96
    x = mc.act8_pack(draw(1, 2, 100, D), "int8")
    w = [draw(2 + i, n, D, std=0.4) for i, n in enumerate((H * dc, H * dc, H * dr, dr))]
    a = mc.mla_max_logit(x, *w, H, dc, dr)
    assert torch.equal(a, mc.mla_max_logit(mc.act8_unpack(x), *w, H, dc, dr))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = mc.mla_max_logit(x, *w, H, dc, dr, stream=side)
    side.synchronize()
    assert torch.equal(a, b)
    ok()


def test_expert_layer_from_the_router_to_the_step(hp):
    """out = sum_k w_k (W_e x): forward, every gradient, and the Muon step on all
    experts' weights in one call."""
    T, K, E, D, M = 150, 2, 4, 96, 64
    x, W = draw(1, T, D), draw(2, E, M, D, std=0.1)
    idx = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(i))[:K] for i in range(T)]).to(DEV)
    idx[5, 1] = -1
    w = torch.softmax(draw(3, T, K, dtype=F32), dim=1)
    plan = mc.expert_sort(idx, E)
    off = plan.offsets.tolist()
    rows = mc.expert_gather(x, plan)
    y = torch.zeros(T * K, M, dtype=BF, device=DEV)
    for e in range(E):
        y[off[e]:off[e + 1]] = rows[off[e]:off[e + 1]] @ W[e].t()
    out = mc.expert_combine(y, plan, w)
    pos, y64, w64 = plan.position.cpu().numpy(), to64(y), to64(w)
    assert rel_fro(to64(out), oa.expert_combine(y64, pos, w64)) <= 2.0 ** -8
    dout = draw(4, T, M, std=1e-2)
    dy, dw = mc.expert_combine_backward(dout, y, plan, w)
    want_dy, want_dw = oa.expert_combine_backward(to64(dout), y64, pos, w64, np.zeros((T * K, M)))
    live = off[-1]
    assert rel_fro(to64(dy)[:live], want_dy[:live]) <= 2.0 ** -8 and rel_fro(to64(dw), want_dw) <= 1e-5
    x8 = mc.act8_pack(x, "int8")
    G = mc.expert_weight_grad(dy, x8, plan, gather=True)
    xs = oa.act8_values(x8.q.cpu().numpy(), x8.scale.cpu().numpy(), D, "int8")[plan.source.cpu().numpy().clip(0) // K]
    for e in range(E):
        assert rel_fro(to64(G[e]), to64(dy)[off[e]:off[e + 1]].T @ xs[off[e]:off[e + 1]]) <= 2.0 ** -8
    same = mc.expert_weight_grad(dy, mc.act8_pack(rows, "int8"), plan, gather=False)
    assert torch.equal(G, same)                          # the same rows, sorted before or after the packing
    dxs = torch.zeros(T * K, D, dtype=BF, device=DEV)
    for e in range(E):
        dxs[off[e]:off[e + 1]] = dy[off[e]:off[e + 1]] @ W[e]
    dx = mc.expert_combine(dxs, plan)                    # the gather's gradient
    assert rel_fro(to64(dx), oa.expert_combine(to64(dxs), pos, np.ones((T, K)))) <= 2.0 ** -8
    Ws, Ms, Us = [W[e].clone() for e in range(E)], [torch.zeros(M, D, device=DEV) for _ in range(E)], [torch.empty(M, D, device=DEV) for _ in range(E)]
    mc.muon_step(Ws, [G[e] for e in range(E)], Ms, update_outs=Us, **hp)
    ok()
    for e in range(E):
        _, _, upd, _ = oracle.muon_step(to64(W[e]), to64(G[e]), np.zeros((M, D)), **hp)
        assert rel_fro(to64(Us[e]), upd) <= NS_TOL


class Layer:
    """All operators on one set of inputs, for capture and replay."""

    def __init__(self, seed, T=300, D=520, M=264, E=6, K=2):
        self.x, self.r, self.w = draw(seed, T, D), draw(seed + 1, T, D), draw(seed + 2, D)
        self.dy, self.dq = draw(seed + 3, T, D, std=1e-2), draw(seed + 4, T * K, M, std=1e-2)
        self.idx = (draw(seed + 5, T, K, dtype=F32).abs() * 3).long() % (E + 1)      # some dropped
        self.rw, self.E = torch.rand(T, K, device=DEV), E
        self.acc = torch.zeros(M, D, device=DEV)

    def run(self):
        h, y, rstd = mc.rms_norm(self.x, self.w, residual=self.r, fmt="e4m3")
        dx, dw = mc.rms_norm_backward(self.dy, mc.act8_pack(h, "int8"), self.w, rstd, dh=self.dy)
        plan = mc.expert_sort(self.idx, self.E)
        rows = mc.expert_gather(h, plan, out=torch.zeros(self.dq.shape[0], h.shape[1], dtype=BF, device=DEV))
        out = mc.expert_combine(rows, plan, self.rw)
        dr, drw = mc.expert_combine_backward(self.dy, rows, plan, self.rw, out=torch.zeros_like(rows))
        g = mc.expert_weight_grad(self.dq, y, plan, gather=True, dtype=F32)
        g1 = mc.weight_grad(self.dq[:y.shape[0]], y)
        mc.weight_grad(self.dq[:y.shape[0]], y, out=self.acc, accumulate=True)
        return [h, mc.act8_unpack(y), rstd, dx, dw, plan.offsets, plan.source, plan.position, rows, out, dr, drw, g, g1]


def test_captured_graphs_replay_like_direct_calls_and_beside_each_other():
    layers = [Layer(10), Layer(30)]
    for a in layers:
        a.run()                                          # uncaptured first: sets the library up
    graphs, outs = [], []
    for a in layers:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(a.run())
        graphs.append(g)
    for step in range(3):
        want = []
        for k, a in enumerate(layers):                   # new inputs in the captured buffers
            a.x.copy_(draw(100 + 10 * step + k, *a.x.shape))
            a.idx.copy_((draw(200 + 10 * step + k, *a.idx.shape, dtype=F32).abs() * 3).long() % (a.E + 1))
            a.acc.zero_()
            want.append([t.clone() for t in a.run()] + [a.acc.clone()])
            a.acc.zero_()
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in layers]
        for g, s in zip(graphs, streams):                # both at once: each graph has scratch of its own
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for k, a in enumerate(layers):
            for i, (got, w) in enumerate(zip(outs[k] + [a.acc], want[k])):
                assert torch.equal(got, w), (step, k, i)
    ok()
    del graphs


def test_each_operator_alone_in_a_graph():
    """A graph of one operator (nothing of the library before it), replayed back to back."""
    a = Layer(110)
    h, y, rstd = mc.rms_norm(a.x, a.w, residual=a.r, fmt="int8")
    plan = mc.expert_sort(a.idx, a.E)
    rows = mc.expert_gather(h, plan, out=torch.zeros(a.dq.shape[0], h.shape[1], dtype=BF, device=DEV))
    dy = a.dq[:h.shape[0]].clone()
    keep = torch.zeros_like(rows)
    calls = [lambda: mc.act8_pack(a.x), lambda: (mc.act8_unpack(y),), lambda: mc.rms_norm(a.x, a.w, residual=a.r),
             lambda: mc.rms_norm_backward(a.dy, h, a.w, rstd), lambda: (mc.weight_grad(dy, y),), lambda: mc.expert_sort(a.idx, a.E),
             lambda: (mc.expert_gather(h, plan, out=keep),), lambda: (mc.expert_combine(rows, plan, a.rw),),
             lambda: mc.expert_combine_backward(a.dy, rows, plan, a.rw, out=torch.zeros_like(rows)),
             lambda: (mc.expert_weight_grad(a.dq, y, plan, gather=True),)]
    for i, call in enumerate(calls):
        want = [t.clone() for t in call() if isinstance(t, torch.Tensor)]
        keep.zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = [t for t in call() if isinstance(t, torch.Tensor)]
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        # (an Act8's padding is unset)
        skip = 1 if i == 0 else 0
        assert len(got) == len(want) and all(torch.equal(p[:, :64] if skip else p, q[:, :64] if skip else q)
                                             for p, q in zip(got[:1] if skip else got, want)), i
        del g
    ok()


@pytest.mark.parametrize("D", [333, 1002, 4096])
def test_what_follows_a_kernel_reads_what_it_wrote(D):
    """Sums written over the residual and gathered at once; codes written over the
    last ones and expanded at once; the same buffers every time."""
    T, E = 1500, 6
    x, w = draw(130, T, D), (1 + 0.1 * draw(131, D, dtype=F32)).to(BF)
    g = torch.Generator(device=DEV)
    g.manual_seed(132)
    plan = mc.expert_sort(torch.randint(0, E, (T, 2), generator=g, device=DEV), E)
    buf, rows = torch.empty_like(x), torch.empty(2 * T, D, dtype=BF, device=DEV)
    want, got = draw(133, T, D), []
    buf.copy_(want)
    code = mc.act8_empty((T, D), "e4m3", device=DEV)
    torch.cuda.synchronize()
    for _ in range(20):
        mc.rms_norm(x, w, residual=buf, h_out=buf)
        mc.expert_gather(buf, plan, out=rows)
        mc.act8_pack(buf, "e4m3", out=code)
        got.append((buf.clone(), rows.clone(), mc.act8_unpack(code)))
    src = plan.source.long()
    for h, r, u in got:
        want = (want.float() + x.float()).to(BF)         # fp32 sum, rounded to bf16: h to the bit
        assert torch.equal(h, want) and torch.equal(r, want[src // 2])
        assert torch.equal(u, mc.act8_unpack(mc.act8_pack(want, "e4m3")))
    ok()


def test_another_stream_and_two_at_once():
    layers = [Layer(50, T=700), Layer(70, T=700)]
    want = [[t.clone() for t in a.run()] for a in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    got = []
    for a, s in zip(layers, streams):
        with torch.cuda.stream(s):
            got.append(a.run())
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(g, w))
    # and the stream as an argument, with work before it on that stream
    a, s = layers[0], streams[0]
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
        x2 = a.x * 2
    x2.record_stream(s)
    p = mc.act8_pack(x2, "int8", stream=s)
    v = mc.act8_unpack(p, stream=s)
    g = mc.weight_grad(a.dq[:700], p, stream=s)
    s.synchronize()
    q = mc.act8_pack(a.x * 2, "int8")
    assert torch.equal(v, mc.act8_unpack(q)) and torch.equal(g, mc.weight_grad(a.dq[:700], q))
    ok()


def test_indices_past_32_bits():
    """Operands of more than 2^31 elements; checked at their ends against the same
    rows alone."""
    D = 32768
    T = (1 << 31) // D + 40
    x = torch.empty(T, D, dtype=BF, device=DEV)
    for a in range(0, T, 8192):
        x[a:a + 8192] = draw(a, min(8192, T - a), D)
    w = draw(1, D)
    tail = slice(T - 9, T)
    p = mc.act8_pack(x, "int8")
    few = mc.act8_pack(x[tail].clone(), "int8")
    assert torch.equal(p.q[tail], few.q) and torch.equal(p.scale[tail], few.scale)
    v = mc.act8_unpack(p)
    assert torch.equal(v[tail], mc.act8_unpack(few))
    del v, p
    n, m = mc.rms_norm(x, w, residual=x, fmt="e4m3"), mc.rms_norm(x[tail].clone(), w, residual=x[tail].clone(), fmt="e4m3")
    assert torch.equal(n.h[tail], m.h) and torch.equal(n.rstd[tail], m.rstd)
    assert torch.equal(n.y.q[tail], m.y.q)
    h, rstd = n.h, n.rstd
    del n
    dx, _ = mc.rms_norm_backward(x, h, w, rstd)
    dt, _ = mc.rms_norm_backward(x[tail].clone(), m.h, w, m.rstd)
    assert torch.equal(dx[tail], dt)
    del dx, h
    # tokens by expert: T * K rows of D
    T2 = T // 2
    idx = torch.arange(2 * T2, device=DEV).view(T2, 2) % 2
    plan = mc.expert_sort(idx, 2)
    rows = mc.expert_gather(x[:T2], plan)
    last = plan.position[T2 - 3:].long()
    assert torch.equal(rows[last[:, 0]], x[T2 - 3:T2]) and torch.equal(rows[last[:, 1]], x[T2 - 3:T2])
    out = mc.expert_combine(rows, plan)
    assert torch.equal(out[T2 - 3:], (x[T2 - 3:T2].float() * 2).to(BF))
    dy, dw = mc.expert_combine_backward(x[:T2], rows, plan, torch.ones(T2, 2, device=DEV), out=rows)
    assert torch.equal(dy[last[:, 1]], x[T2 - 3:T2])
    assert torch.allclose(dw[T2 - 1], x[T2 - 1].float().square().sum().expand(2), rtol=1e-5)
    ok()


def test_weight_gradient_past_32_bits():
    T, N, M = (1 << 31) // 4096 + 100, 4096, 16
    x8 = mc.act8_empty((T, N), "int8")
    x8.q.random_(0, 256)
    x8.scale.fill_(120)
    dy = torch.zeros(T, M, dtype=BF, device=DEV)
    dy[-50:] = draw(1, 50, M)                            # only the last rows count
    g = mc.weight_grad(dy, x8, dtype=F32)
    tail = mc.Act8(x8.q[-50:].clone(), x8.scale[-50:].clone(), (50, N), "int8")
    want = dy[-50:].double().t() @ mc.act8_unpack(tail).double()
    assert float((g.double() - want).norm() / want.norm()) <= 1e-6
    ok()


def test_workspaces_and_alignment():
    dy, x8 = draw(1, 300, 24), mc.act8_pack(draw(2, 300, 40), "int8")
    lib = mc.load_library()
    need = lib.mc_weight_grad_workspace_size(300, 24, 40)
    want = mc.weight_grad(dy, x8)
    ws = torch.full((need + 64,), 77, dtype=torch.uint8, device=DEV)
    got = mc.weight_grad(dy, x8, workspace=ws[16:16 + need])          # 16-byte aligned is enough
    assert torch.equal(got, want) and (ws[:16] == 77).all() and (ws[16 + need:] == 77).all()
    for call in (lambda w: mc.weight_grad(dy, x8, workspace=w), lambda w: mc.expert_sort(torch.zeros(9000, 8, dtype=torch.int64, device=DEV), 4, workspace=w),
                 lambda w: mc.rms_norm_backward(dy, dy, dy[0].clone(), torch.ones(300, device=DEV), workspace=w)):
        with pytest.raises(mc.MuonClipError) as e:
            call(torch.empty(16, dtype=torch.uint8, device=DEV))
        assert e.value.code == mc.MC_ERR_NOSPC
    odd = draw(3, 301 * 24 + 1)[1:1 + 300 * 24].view(300, 24)
    with pytest.raises(mc.MuonClipError) as e:
        mc.weight_grad(odd, x8)
    assert e.value.code == mc.MC_ERR_ALIGN
    with pytest.raises(ValueError, match="contiguous"):
        mc.act8_pack(draw(4, 8, 64).t())
    with pytest.raises(ValueError, match="rows"):
        mc.weight_grad(dy[:299], x8)
    with pytest.raises(ValueError, match="accumulate"):
        mc.weight_grad(dy, x8, accumulate=True)
    with pytest.raises(mc.MuonClipError) as e:
        mc.weight_grad(dy, x8, out=torch.zeros(24, 40, dtype=BF, device=DEV), accumulate=True)
    assert e.value.code == mc.MC_ERR_INVAL
    with pytest.raises(TypeError):
        mc.weight_grad(dy.float(), x8)
    ok()


def test_no_rows_at_all():
    """Every operator on an empty batch."""
    e, w, none = torch.empty(0, 64, dtype=BF, device=DEV), draw(1, 64), torch.empty(0, 2, device=DEV)
    for fmt in (None, "e4m3"):
        n = mc.rms_norm(e, w, residual=e.clone(), fmt=fmt)
        assert n.h.shape == (0, 64) and n.rstd.shape == (0,) and tuple(n.y.shape) == (0, 64)
    dx, dw = mc.rms_norm_backward(e, e.clone(), w, n.rstd)
    assert dx.shape == (0, 64) and dw.shape == (64,) and (dw == 0).all()
    plan = mc.expert_sort(torch.empty(0, 2, dtype=torch.int64, device=DEV), 3)
    rows = mc.expert_gather(e, plan)
    assert rows.shape == (0, 64) and mc.expert_combine(rows, plan, none).shape == (0, 64)
    dy, dwt = mc.expert_combine_backward(e, rows, plan, none)
    assert dy.shape == (0, 64) and dwt.shape == (0, 2)
    x8 = mc.act8_pack(e)
    for gather in (True, False):
        g = mc.expert_weight_grad(e, x8, plan, gather=gather)
        assert g.shape == (3, 64, 64) and (g == 0).all()
    base = draw(2, 3, 64, 64, dtype=F32)
    g = mc.expert_weight_grad(e, x8, plan, gather=True, out=base.clone(), accumulate=True)
    assert torch.equal(g, base)
    ok()


def test_kernels_are_profiled():
    mc.profile_begin()
    Layer(90).run()
    got = mc.profile_end()
    for kind in ("act8_pack", "act8_unpack", "rms_norm", "rms_norm_backward", "rms_norm_dw", "weight_grad_prepare", "weight_grad",
                 "expert_sort", "expert_gather", "expert_combine", "expert_combine_backward"):
        assert got[kind]["launches"] >= 1, kind

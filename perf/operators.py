"""Measured cases of the activation operators around the optimizer step.

Three families, which a training step runs in this order:

* ``norm`` and ``norm_grad``: the root-mean-square norm of a block's input with
  the residual's addition, its output in 8 bits with scales, and its gradient;
* ``pack`` and ``wgrad``: activations kept in 8 bits for the backward pass, and
  the weight gradient G = dY^T X (what the Muon step takes) from them;
* ``dispatch``, ``combine``, ``combine_grad`` and ``expert_wgrad``: tokens
  sorted by expert and back, with weights applied, their gradient, and the
  gradients of every expert's weight.

The 8-bit form of a row: blocks of 32 consecutive columns, each with one scale
byte s standing for 2^(s - 127), and one code per value (an e4m3 number, or an
int8).  The scale is the smallest power of two (at least 2^-120) that brings
the block's largest magnitude to at most 448 (e4m3) or 127 (int8); a block
that holds a NaN or an infinity has s = 255 and stands for NaN.

``own`` false computes everything in elementary torch operations in 32 bits;
``own`` true calls the package.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 32
EPS = 1e-6
TOP = {"e4m3": 448.0, "int8": 127.0}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # One token at decode time through a 4096-wide block's norm: latency.
        dict(name="norm-token", op="norm", T=1, D=4096, dtype="bf16", fmt="e4m3", residual=True),
        # 4 sequences of 4096 tokens (the attention workload's batch) through the same norm.
        dict(name="norm-batch", op="norm", T=16384, D=4096, dtype="bf16", fmt="e4m3", residual=True),
        # Its gradient, with the block input kept in bf16.
        dict(name="norm-grad-batch", op="norm_grad", T=16384, D=4096, dtype="bf16", fmt="", residual=True),
        # A short ragged batch of a 1000-wide model, the input kept in 8 bits.
        dict(name="norm-grad-odd", op="norm_grad", T=777, D=1000, dtype="bf16", fmt="int8", residual=False),
        # fp32 activations of an odd width and length to 8 bits and back.
        dict(name="pack-odd", op="pack", T=1021, D=1789, dtype="fp32", fmt="int8"),
        # The feed-forward activations of the 7B-shaped model for one batch.
        dict(name="pack-ffn", op="pack", T=16384, D=14336, dtype="bf16", fmt="e4m3"),
        # Gradient of a 4096 x 4096 attention projection from 8192 tokens, for an fp32 main gradient.
        dict(name="wgrad-attn", op="wgrad", T=8192, M=4096, N=4096, dtype="fp32", fmt="int8"),
        # Gradient of the gate projection (14336 x 4096) from a whole batch, in bf16 as the step takes it.
        dict(name="wgrad-ffn", op="wgrad", T=16384, M=14336, N=4096, dtype="bf16", fmt="e4m3"),
        # Gradients of the 64 experts' 2048 x 7168 gate projections, 4096 tokens to 8 experts each.
        dict(name="expert-wgrad", op="expert_wgrad", T=4096, K=8, E=64, M=2048, N=7168, dtype="bf16", fmt="int8"),
        # The same tokens sorted by expert.
        dict(name="dispatch-batch", op="dispatch", T=4096, K=8, E=64, D=7168, dtype="bf16"),
        # 48 tokens of a decode step brought back from their experts: latency.
        dict(name="combine-decode", op="combine", T=48, K=8, E=64, D=7168, dtype="bf16"),
        # Gradient of bringing the batch back: the experts' rows and the router's weights.
        dict(name="combine-grad-batch", op="combine_grad", T=4096, K=8, E=64, D=7168, dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width: three in four a multiple of 8, the others as they fall."""
    w = _spread(rng, lo, hi)
    return max(8, w // 8 * 8) if rng.random() < 0.75 else w


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "pack", "wgrad", "wgrad", "expert_wgrad", "dispatch", "combine",
                     "combine_grad"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    fmt = rng.choice(["e4m3", "int8"])
    if op in ("norm", "norm_grad"):
        D = _width(rng, 128, 8192)
        T = _spread(rng, 1, min(32768, (1 << 26) // D))
        kept = rng.choice(["", fmt]) if op == "norm_grad" else fmt
        return dict(op=op, T=T, D=D, dtype=dtype, fmt=kept, residual=rng.random() < 0.7)
    if op == "pack":
        D = _width(rng, 64, 14336)
        return dict(op=op, T=_spread(rng, 1, min(32768, (1 << 27) // D)), D=D, dtype=dtype, fmt=fmt)
    if op == "wgrad":
        M, N = _width(rng, 64, 14336), _width(rng, 64, 14336)
        T = _spread(rng, 1, max(1, min(32768, int(9e11 / (2.0 * M * N)))))
        return dict(op=op, T=T, M=M, N=N, dtype=dtype, fmt=fmt)
    E = rng.choice([4, 8, 16, 60, 64, 128])
    K = rng.choice([1, 2, 4, min(8, E)])
    if op == "expert_wgrad":
        E = min(E, 64)
        M, N = _width(rng, 128, 2048), _width(rng, 128, 4096)
        T = _spread(rng, 8, max(8, min(4096, int(2e11 / (2.0 * M * N * K)))))
        return dict(op=op, T=T, K=K, E=E, M=M, N=N, dtype=dtype, fmt=fmt)
    D = _width(rng, 128, 7168)
    T = _spread(rng, 1, max(1, min(16384, (1 << 26) // (D * K))))
    return dict(op=op, T=T, K=K, E=E, D=D, dtype=dtype)


# ------------------------------------------------------------------ inputs
def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _activations(gen, T, D, dtype):
    """Rows of a block's input: Gaussian, channels of unequal size, a few of them large."""
    dev = gen.device
    size = torch.exp(0.5 * torch.randn(D, generator=gen, device=dev))
    size = torch.where(torch.rand(D, generator=gen, device=dev) < 0.004, size * 20, size)
    return (torch.randn(T, D, generator=gen, device=dev) * size).to(dtype)


def _routing(gen, T, K, E):
    """The K experts of each token, as a router's top-k gives them (some experts liked
    better than others), one pair in a hundred dropped, and the router's weights."""
    dev = gen.device
    liked = 0.5 * torch.randn(E, generator=gen, device=dev)
    score = liked + torch.randn(T, E, generator=gen, device=dev)
    top, idx = torch.topk(score, K, dim=1)
    weights = torch.softmax(top.float(), dim=1)
    idx = torch.where(torch.rand(T, K, generator=gen, device=dev) < 0.01, torch.full_like(idx, -1), idx)
    return idx, weights


def _padded(n, to):
    return (n + to - 1) // to * to


def _store(codes, scale, fmt):
    """Codes and scale bytes in the layout a program keeps: rows of whole 16 bytes."""
    T, D = codes.shape
    q = torch.zeros(T, _padded(D, 16), dtype=torch.uint8, device=codes.device)
    q[:, :D] = codes
    s = torch.zeros(T, _padded(scale.shape[1], 16), dtype=torch.uint8, device=codes.device)
    s[:, :scale.shape[1]] = scale
    return dict(q=q, scale=s, shape=(T, D), fmt=fmt)


def prepare(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    op, T = case["op"], case["T"]
    state = dict(case=case)
    if op in ("norm", "norm_grad"):
        D, dt = case["D"], _dtype(case["dtype"])
        state["weight"] = (1.0 + 0.2 * torch.randn(D, generator=gen, device=dev)).to(dt)
        state["x"] = _activations(gen, T, D, dt)
        if op == "norm":
            state["residual"] = _activations(gen, T, D, dt) if case["residual"] else None
        else:
            x = state.pop("x")
            state["rstd"] = torch.rsqrt(x.float().square().mean(dim=1) + EPS)
            state["h"] = _store(*_quantise(x.float(), case["fmt"]), case["fmt"]) if case["fmt"] else x
            state["dy"] = (1e-3 * torch.randn(T, D, generator=gen, device=dev)).to(dt)
            state["dh"] = (1e-3 * torch.randn(T, D, generator=gen, device=dev)).to(dt) if case["residual"] else None
    elif op == "pack":
        state["x"] = _activations(gen, T, case["D"], _dtype(case["dtype"]))
    elif op == "wgrad":
        x = _activations(gen, T, case["N"], torch.bfloat16)
        state["x8"] = _store(*_quantise(x.float(), case["fmt"]), case["fmt"])
        state["dy"] = (1e-3 * torch.randn(T, case["M"], generator=gen, device=dev)).to(torch.bfloat16)
    else:
        K, E = case["K"], case["E"]
        idx, weights = _routing(gen, T, K, E)
        state["weights"] = weights
        if op == "dispatch":
            state["idx"] = idx
            state["x"] = _activations(gen, T, case["D"], _dtype(case["dtype"]))
            state["rows"] = torch.zeros(T * K, case["D"], dtype=state["x"].dtype, device=dev)
        else:
            # the order that the forward pass has left behind
            state["offsets"], state["source"], state["position"] = _sorted(idx, E)
            if op == "expert_wgrad":
                x = _activations(gen, T, case["N"], torch.bfloat16)
                state["x8"] = _store(*_quantise(x.float(), case["fmt"]), case["fmt"])
                state["dy"] = (1e-3 * torch.randn(T * K, case["M"], generator=gen, device=dev)).to(torch.bfloat16)
            else:
                dt = _dtype(case["dtype"])
                state["y"] = torch.randn(T * K, case["D"], generator=gen, device=dev).to(dt)
                if op == "combine_grad":
                    state["dout"] = (1e-3 * torch.randn(T, case["D"], generator=gen, device=dev)).to(dt)
                    state["rows"] = torch.zeros(T * K, case["D"], dtype=dt, device=dev)
    return state


# ------------------------------------------------------------- plain forms
def _quantise(x, fmt):
    """fp32 rows to (code bytes [T, D], scale bytes [T, ceil(D / 32)])."""
    T, D = x.shape
    nb = (D + BLOCK - 1) // BLOCK
    xb = torch.zeros(T, nb * BLOCK, dtype=torch.float32, device=x.device)
    xb[:, :D] = x
    xb = xb.view(T, nb, BLOCK)
    amax = xb.abs().amax(dim=2)
    fine = torch.isfinite(xb).all(dim=2)
    m, e = torch.frexp(torch.where(fine, amax, torch.zeros_like(amax)))   # amax = (2m) 2^(e-1), 2m in [1, 2)
    top_m, top_e = (1.75, 8) if fmt == "e4m3" else (1.984375, 6)
    k = (e - 1 - top_e + (2 * m > top_m).to(e.dtype))
    k = torch.where(amax > 0, k, torch.full_like(k, -120)).clamp(min=-120)
    v = torch.ldexp(torch.where(fine[..., None], xb, torch.zeros_like(xb)), -k[..., None])
    if fmt == "e4m3":
        codes = v.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        codes = torch.round(v).to(torch.int8).view(torch.uint8)
    scale = torch.where(fine, k + 127, torch.full_like(k, 255)).to(torch.uint8)
    return codes.view(T, nb * BLOCK)[:, :D], scale


def _values(a):
    """The fp32 values that a stored 8-bit activation stands for."""
    T, D = a["shape"]
    nb = (D + BLOCK - 1) // BLOCK
    codes = a["q"][:, :D].contiguous()
    v = codes.view(torch.float8_e4m3fn).float() if a["fmt"] == "e4m3" else codes.view(torch.int8).float()
    s = a["scale"][:, :nb].to(torch.int32)
    p = torch.where(s == 255, torch.full_like(s, 1, dtype=torch.float32) * float("nan"),
                    torch.ldexp(torch.ones_like(s, dtype=torch.float32), s - 127))
    return v * p.repeat_interleave(BLOCK, dim=1)[:, :D]


def _sorted(idx, E):
    """offsets [E + 1], source [T*K] (the pair of each sorted row, -1 behind the last),
    position [T, K] (the row of each pair, -1 where it is dropped); stable."""
    T, K = idx.shape
    flat = idx.reshape(-1)
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    count = torch.zeros(E + 1, dtype=torch.int64, device=idx.device)
    count.scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=idx.device)
    offsets[1:] = torch.cumsum(count[:E], 0).to(torch.int32)
    order = torch.sort(key, stable=True).indices
    rank = torch.empty_like(order)
    rank[order] = torch.arange(T * K, device=idx.device)
    source = torch.where(key[order] < E, order, torch.full_like(order, -1)).to(torch.int32)
    position = torch.where(key < E, rank, torch.full_like(rank, -1)).to(torch.int32).view(T, K)
    return offsets, source, position


def _plain(state):
    c = state["case"]
    op = c["op"]
    if op == "norm":
        h = state["x"].float()
        if state["residual"] is not None:
            h = (h + state["residual"].float()).to(state["x"].dtype).float()
        rstd = torch.rsqrt(h.square().mean(dim=1) + EPS)
        y = h * rstd[:, None] * state["weight"].float()
        codes, scale = _quantise(y, c["fmt"])
        y = _values(_store(codes, scale, c["fmt"])).to(torch.bfloat16)
        return dict(h=h.to(state["x"].dtype), y=y, rstd=rstd)
    if op == "norm_grad":
        h = _values(state["h"]) if c["fmt"] else state["h"].float()
        xhat = h * state["rstd"][:, None]
        dy = state["dy"].float()
        g = dy * state["weight"].float()
        dx = state["rstd"][:, None] * (g - xhat * (g * xhat).mean(dim=1, keepdim=True))
        if state["dh"] is not None:
            dx = dx + state["dh"].float()
        return dict(dx=dx.to(state["dy"].dtype), dw=(dy * xhat).sum(dim=0))
    if op == "pack":
        codes, scale = _quantise(state["x"].float(), c["fmt"])
        return dict(x=_values(_store(codes, scale, c["fmt"])).to(torch.bfloat16), scale=scale)
    if op == "wgrad":
        return (state["dy"].float().t() @ _values(state["x8"])).to(_dtype(c["dtype"]))
    T, K, E = c["T"], c["K"], c["E"]
    if op == "dispatch":
        offsets, source, position = _sorted(state["idx"], E)
        rows = torch.where(source[:, None] >= 0, state["x"][(source.clamp(min=0) // K).long()], state["rows"])
        return dict(offsets=offsets, source=source, position=position, rows=rows)
    if op == "expert_wgrad":
        # every expert's rows side by side, behind them zeros, and one batched product
        count = (state["offsets"][1:] - state["offsets"][:-1]).long()
        most = max(1, int(count.max()))
        at = torch.arange(most, device=count.device)
        inside = at[None, :] < count[:, None]
        row = torch.where(inside, state["offsets"][:-1, None].long() + at, torch.zeros_like(at)[None, :])
        x = _values(state["x8"])[state["source"][row].long().clamp(min=0) // K] * inside[..., None]
        dy = state["dy"][row].float() * inside[..., None]
        return torch.bmm(dy.transpose(1, 2), x).to(_dtype(c["dtype"]))
    kept = state["position"] >= 0
    row = state["position"].long().clamp(min=0)
    w = state["weights"] * kept
    if op == "combine":
        return (state["y"][row].float() * w[..., None]).sum(dim=1).to(state["y"].dtype)
    pair = state["source"].long().clamp(min=0)
    live = state["source"][:, None] >= 0
    dy = state["dout"][pair // K].float() * state["weights"].reshape(-1)[pair][:, None]
    dw = (state["y"][row].float() * state["dout"].float()[:, None, :]).sum(dim=2) * kept
    return dict(dy=torch.where(live, dy.to(state["rows"].dtype), state["rows"]), dweights=dw)


# ------------------------------------------------------- the package's calls
def _own(state):
    import matrix_orthogonalising_optimizer_step_b200 as mc
    c = state["case"]
    op = c["op"]
    if op == "norm":
        h, y, rstd = mc.rms_norm(state["x"], state["weight"], residual=state["residual"], eps=EPS, fmt=c["fmt"])
        return dict(h=h, y=mc.act8_unpack(y), rstd=rstd)
    if op == "norm_grad":
        h = mc.Act8(**state["h"]) if c["fmt"] else state["h"]
        dx, dw = mc.rms_norm_backward(state["dy"], h, state["weight"], state["rstd"], dh=state["dh"])
        return dict(dx=dx, dw=dw)
    if op == "pack":
        a = mc.act8_pack(state["x"], c["fmt"])
        return dict(x=mc.act8_unpack(a), scale=a.scale[:, :(c["D"] + BLOCK - 1) // BLOCK])
    if op == "wgrad":
        return mc.weight_grad(state["dy"], mc.Act8(**state["x8"]), dtype=_dtype(c["dtype"]))
    if op == "dispatch":
        plan = mc.expert_sort(state["idx"], c["E"])
        rows = mc.expert_gather(state["x"], plan, out=state["rows"])
        return dict(offsets=plan.offsets, source=plan.source, position=plan.position, rows=rows)
    plan = mc.ExpertPlan(state["offsets"], state["source"], state["position"])
    if op == "expert_wgrad":
        return mc.expert_weight_grad(state["dy"], mc.Act8(**state["x8"]), plan, gather=True, dtype=_dtype(c["dtype"]))
    if op == "combine":
        return mc.expert_combine(state["y"], plan, state["weights"])
    dy, dw = mc.expert_combine_backward(state["dout"], state["y"], plan, state["weights"], out=state["rows"])
    return dict(dy=dy, dweights=dw)


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------- the work
def _bytes8(T, D):
    return T * (D + (D + BLOCK - 1) // BLOCK)


def work(case):
    op, T = case["op"], case["T"]
    es = 2 if case["dtype"] == "bf16" else 4
    if op == "norm":      # x, residual and weight in; h, 8-bit y and its values, rstd out
        D = case["D"]
        n = T * D * es * (3 if case["residual"] else 1) + D * es + 4 * T
        return dict(bytes=n + 2 * _bytes8(T, D) + 2 * T * D, flops=8.0 * T * D)
    if op == "norm_grad":
        D = case["D"]
        kept = _bytes8(T, D) if case["fmt"] else T * D * es
        return dict(bytes=kept + T * D * es * (3 if case["residual"] else 2) + D * (es + 4) + 4 * T, flops=10.0 * T * D)
    if op == "pack":      # in, the 8-bit form out and in again, its values out
        return dict(bytes=T * case["D"] * (es + 2) + 2 * _bytes8(T, case["D"]), flops=3.0 * T * case["D"])
    if op == "wgrad":
        M, N = case["M"], case["N"]
        return dict(bytes=2 * T * M + _bytes8(T, N) + M * N * es, flops=2.0 * T * M * N)
    K, E = case["K"], case["E"]
    if op == "expert_wgrad":
        M, N = case["M"], case["N"]
        return dict(bytes=2 * T * K * M + _bytes8(T, N) + E * M * N * es + 4 * T * K, flops=2.0 * T * K * M * N)
    D = case["D"]
    if op == "dispatch":  # x once, its rows out; the pairs in (64 bits) and the order out
        return dict(bytes=T * D * es * (1 + K) + T * K * (8 + 8) + 4 * (E + 1), flops=0.0)
    if op == "combine":
        return dict(bytes=T * D * es * (1 + K) + T * K * 8, flops=2.0 * T * K * D)
    return dict(bytes=T * D * es * (1 + 2 * K) + T * K * 12, flops=3.0 * T * K * D)


# ----------------------------------------------------------- in 64 bits
def _round64(v, fmt):
    """Values (64 bits, at most the format's largest) to the nearest code's value, ties to even."""
    if fmt == "int8":
        return torch.round(v)
    e = torch.frexp(v).exponent.clamp(min=-5) - 4       # v in [2^(e+3), 2^(e+4)): steps of 2^e, 2^-9 the least
    step = torch.ldexp(torch.ones_like(v), e)
    return torch.round(v / step) * step


def _through8(x, fmt):
    """What 64-bit rows stand for after a passage through the 8-bit form, and the scale bytes."""
    T, D = x.shape
    pad = (-D) % BLOCK
    xb = torch.cat([x, x.new_zeros(T, pad)], dim=1).reshape(T, -1, BLOCK)
    amax = xb.abs().amax(dim=2, keepdim=True)
    # the least k with amax <= TOP 2^k: from a first guess, one step up or down
    k = torch.ceil(torch.log2(torch.where(amax > 0, amax, torch.ones_like(amax)) / TOP[fmt]))
    k = torch.where(amax > TOP[fmt] * torch.exp2(k), k + 1, k)
    k = torch.where(amax <= TOP[fmt] * torch.exp2(k - 1), k - 1, k)
    k = torch.where(amax > 0, k, torch.full_like(k, -120)).clamp(min=-120)
    v = _round64(xb * torch.exp2(-k), fmt) * torch.exp2(k)
    return v.reshape(T, -1)[:, :D], (k[..., 0] + 127).to(torch.uint8)


def _values64(a):
    T, D = a["shape"]
    q = a["q"][:, :D].to(torch.int64)
    if a["fmt"] == "int8":
        v = torch.where(q > 127, q - 256, q).double()
    else:                                               # sign, 4 bits of exponent, 3 of fraction
        e, f = (q >> 3) & 15, (q & 7).double()
        v = torch.where(e > 0, (8 + f) * torch.exp2((e - 10).double()), f * 2.0 ** -9)
        v = torch.where(q > 127, -v, v)
    col = torch.arange(D, device=q.device) // BLOCK
    return v * torch.exp2(a["scale"].double()[:, col] - 127)


def exact(case, seed):
    s = prepare(case, seed)
    op, T = case["op"], case["T"]
    if op == "norm":
        h = s["x"].double()
        if s["residual"] is not None:                   # the sum is stored in the inputs' type
            h = (h + s["residual"].double()).to(s["x"].dtype).double()
        rstd = 1.0 / torch.sqrt((h * h).sum(dim=1) / case["D"] + EPS)
        y = h * rstd[:, None] * s["weight"].double()
        return dict(h=h, y=_through8(y, case["fmt"])[0], rstd=rstd)
    if op == "norm_grad":
        x = _values64(s["h"]) if case["fmt"] else s["h"].double()
        r, w, dy = s["rstd"].double()[:, None], s["weight"].double(), s["dy"].double()
        dot = (dy * w * x).sum(dim=1, keepdim=True)
        dx = r * w * dy - r ** 3 * x * dot / case["D"]
        return dict(dx=dx if s["dh"] is None else dx + s["dh"].double(), dw=(dy * x * r).sum(dim=0))
    if op == "pack":
        x, scale = _through8(s["x"].double(), case["fmt"])
        return dict(x=x, scale=scale)
    if op == "wgrad":
        return torch.einsum("tm,tn->mn", s["dy"].double(), _values64(s["x8"]))
    K, E = case["K"], case["E"]
    if op == "dispatch":
        # counted on the host: one expert after the other, pairs in their order
        idx = s["idx"].reshape(-1).cpu().numpy()
        found = [np.flatnonzero(idx == e) for e in range(E)]
        offsets = np.concatenate([[0], np.cumsum([len(f) for f in found])])
        order = np.concatenate(found).astype(np.int64)
        source = np.full(T * K, -1, np.int64)
        source[:len(order)] = order
        position = np.full(T * K, -1, np.int64)
        position[order] = np.arange(len(order))
        rows = torch.zeros(T * K, case["D"], dtype=torch.float64, device=s["x"].device)
        rows[:len(order)] = s["x"].double()[torch.from_numpy(order // K).to(rows.device)]
        return dict(offsets=torch.from_numpy(offsets).int(), source=torch.from_numpy(source).int(),
                    position=torch.from_numpy(position).int().view(T, K), rows=rows)
    if op == "expert_wgrad":
        x, off = _values64(s["x8"]), s["offsets"].tolist()
        token = s["source"].long() // K
        out = torch.zeros(E, case["M"], case["N"], dtype=torch.float64, device=x.device)
        for e in range(E):
            a, b = off[e], off[e + 1]
            out[e] = s["dy"][a:b].double().t() @ x[token[a:b]]
        return out
    w, pos = s["weights"].double(), s["position"]
    if op == "combine":
        out = torch.zeros(T, case["D"], dtype=torch.float64, device=w.device)
        for k in range(K):
            t = torch.nonzero(pos[:, k] >= 0)[:, 0]
            out[t] += w[t, k, None] * s["y"][pos[t, k].long()].double()
        return out
    dy, dw = s["rows"].double(), torch.zeros_like(w)
    for k in range(K):
        t = torch.nonzero(pos[:, k] >= 0)[:, 0]
        r = pos[t, k].long()
        dy[r] = w[t, k, None] * s["dout"][t].double()
        dw[t, k] = (s["dout"][t].double() * s["y"][r].double()).sum(dim=1)
    return dict(dy=dy, dweights=dw)

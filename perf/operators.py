"""Cases of the linear recurrence and of layer normalisation: inputs, the plain
forms, and the library's calls.

``own`` selects which side ``run`` takes: the operators in elementary torch
operations (False), or the calls a user makes of the library (True).

The operators, per sequence and channel (tokens t in order, fp32 inside):

  linear_fwd       h_t = alpha_t h_{t-1} + x_t, out_t = h_t, alpha = e^log_alpha
                   (one per token and head, or per token and channel, or 1)
  linear_step      the same for one token per sequence, on a resident state
  linear_train     linear_fwd, then its gradients from those of out and of the
                   final state: G_t = dout_t + alpha_{t+1} G_{t+1},
                   dx_t = G_t, dlog_alpha_t = G_t alpha_t h_{t-1}
                   (summed over a head's channels for a decay per head)
  layer_norm       y = (x - mean) rstd w + b over each (token, head)'s d
                   channels; w, b per head and channel
  layer_norm_bwd   dx, dw, db of layer_norm
"""
from __future__ import annotations

import math
import random

import torch

own = False

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
# the largest drawn case, in elements of x, per operator: none costs more than
# the largest listed case
DRAW_LIMIT = {"linear_fwd": 1 << 26, "linear_step": 1 << 24,
              "linear_train": 1 << 25, "layer_norm": 1 << 26,
              "layer_norm_bwd": 1 << 26}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # decoding one sequence: the call's latency is all there is
        dict(name="step_n1_h16_d128_bf16", op="linear_step", B=1, H=16, d=128,
             dtype="bf16", gate="channel"),
        # decoding a large batch: every state read and written once
        dict(name="step_n256_h16_d128_bf16", op="linear_step", B=256, H=16,
             d=128, dtype="bf16", gate="channel"),
        # the smallest sequence mixed, in fp32, without a decay (a prefix sum)
        dict(name="fwd_b1_h1_t256_d16_fp32", op="linear_fwd", B=1, T=256, H=1,
             d=16, dtype="fp32", gate="none", init=False),
        # the prefill of a batch, one decay per token and channel
        dict(name="fwd_b8_h16_t4096_d128_bf16", op="linear_fwd", B=8, T=4096,
             H=16, d=128, dtype="bf16", gate="channel", init=True),
        # the prefill of one long sequence, few channels per GPU to go round
        dict(name="fwd_b1_h16_t65536_d128_bf16", op="linear_fwd", B=1, T=65536,
             H=16, d=128, dtype="bf16", gate="channel", init=True),
        # a training step on a ragged packed batch with a decay per head and
        # an odd head width
        dict(name="train_packed5_h6_d72_fp32", op="linear_train", nseq=5,
             lo=0, hi=2500, lens=3, H=6, d=72, dtype="fp32", gate="scalar",
             init=True),
        # a training step on long packed sequences: the largest case
        dict(name="train_packed8_h16_d128_bf16", op="linear_train", nseq=8,
             lo=2048, hi=16384, lens=0, H=16, d=128, dtype="bf16",
             gate="channel", init=True),
        # the input norm of one decoded token
        dict(name="norm_n1_d2048_bf16", op="layer_norm", ntok=1, H=1, d=2048,
             dtype="bf16"),
        # the norm of the heads' outputs over a batch of prompts
        dict(name="norm_n32768_h16_d128_bf16", op="layer_norm", ntok=32768,
             H=16, d=128, dtype="bf16"),
        # a short fine-tuning batch of odd width in fp32
        dict(name="norm_bwd_n333_d1001_fp32", op="layer_norm_bwd", ntok=333,
             H=1, d=1001, dtype="fp32"),
        # the backward of the input norm over a training batch
        dict(name="norm_bwd_n32768_d2048_bf16", op="layer_norm_bwd",
             ntok=32768, H=1, d=2048, dtype="bf16"),
        # the backward of the heads' output norm over a training batch
        dict(name="norm_bwd_n8192_h16_d128_bf16", op="layer_norm_bwd",
             ntok=8192, H=16, d=128, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear_fwd", "linear_step", "linear_train", "layer_norm",
                     "layer_norm_bwd"])
    limit = DRAW_LIMIT[op]
    case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp32"]))
    if op.startswith("layer_norm"):
        if rng.random() < 0.5:            # a model's width
            case["H"], case["d"] = 1, _log_int(rng, 16, 8192)
        else:                             # a norm per head
            case["H"], case["d"] = rng.randint(2, 32), _log_int(rng, 8, 512)
        case["ntok"] = _log_int(rng, 1, max(1, min(
            65536, limit // (case["H"] * case["d"]))))
        return case
    case["H"] = rng.randint(1, 32)
    case["d"] = _log_int(rng, 8, 256)
    width = case["H"] * case["d"]
    case["gate"] = rng.choice(["channel", "channel", "scalar", "none"])
    if op == "linear_step":
        case["B"] = _log_int(rng, 1, max(1, min(1024, limit // width)))
        return case
    case["init"] = rng.random() < 0.5
    if rng.random() < 0.4:                # packed sequences of mixed lengths
        case["nseq"] = rng.randint(1, 24)
        case["hi"] = _log_int(rng, 1, max(1, min(16384, limit // (
            width * case["nseq"]))))
        case["lo"] = rng.choice([0, case["hi"] // 4, case["hi"]])
        case["lens"] = rng.randint(0, 10 ** 6)
    else:
        case["B"] = rng.randint(1, 16)
        case["T"] = _log_int(rng, 1, max(1, min(65536, limit // (
            width * case["B"]))))
    return case


def _lengths(case):
    """The packed sequences' lengths (at least one token in all)."""
    rng = random.Random(case["lens"])
    n = [rng.randint(case["lo"], case["hi"]) for _ in range(case["nseq"])]
    if sum(n) == 0:
        n[-1] = 1
    return n


def _grid(case):
    """(leading sizes of x, number of sequences, number of tokens)."""
    if case["op"] == "linear_step":
        return (case["B"],), case["B"], case["B"]
    if "nseq" in case:
        n = _lengths(case)
        return (1, sum(n)), len(n), sum(n)
    return (case["B"], case["T"]), case["B"], case["B"] * case["T"]


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(seed)
    H, d = case["H"], case["d"]
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    st = {"case": case}
    if case["op"].startswith("layer_norm"):
        ntok = case["ntok"]
        # rows of a residual stream: their own scales and offsets, and a few
        # channels far larger than the rest
        x = normal(ntok, H, d)
        x *= torch.exp(0.5 * normal(ntok, 1, 1))
        x += 0.5 * normal(ntok, H, 1)
        x[..., :: max(1, d // 3)] *= 8.0
        shape = (d,) if H == 1 else (H, d)
        st["x"] = (x.reshape(ntok, d) if H == 1 else x).to(dt)
        st["weight"] = 1.0 + 0.2 * normal(*shape)
        st["bias"] = 0.1 * normal(*shape)
        if case["op"] == "layer_norm_bwd":
            st["d_out"] = normal(*st["x"].shape).to(dt)
        return st
    lead, nseq, _ = _grid(case)
    st["x"] = normal(*lead, H, d).to(dt)
    st["log_alpha"] = None
    if case["gate"] != "none":
        shape = (*lead, H) if case["gate"] == "scalar" else (*lead, H, d)
        # decays of 0.5 to 10 percent a token, drawn as the library's
        # workloads draw them
        u = torch.rand(*shape, generator=gen, device=dev)
        st["log_alpha"] = -torch.nn.functional.softplus(normal(*shape)) * (
            0.005 + 0.095 * u)
    if case["op"] == "linear_step":
        st["state"] = normal(nseq, H, d)
        st["state_out"] = torch.empty_like(st["state"])
        return st
    st["s0"] = normal(nseq, H, d) if case["init"] else None
    st["cu"] = None
    if "nseq" in case:
        cu = [0]
        for n in _lengths(case):
            cu.append(cu[-1] + n)
        st["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        st["first"] = torch.tensor(
            [a for a, b in zip(cu, cu[1:]) if b > a], device=dev)
        st["last"] = torch.tensor(
            [b - 1 for a, b in zip(cu, cu[1:]) if b > a], device=dev)
        st["some"] = torch.tensor(
            [i for i, (a, b) in enumerate(zip(cu, cu[1:])) if b > a],
            device=dev)
    if case["op"] == "linear_train":
        st["d_out"] = normal(*lead, H, d).to(dt)
        st["d_state"] = normal(nseq, H, d)
    return st


# ------------------------------------------------------------- plain forms

def _scan(x, la):
    """h_t = e^la_t h_{t-1} + x_t along dim 1 of x [B, T, H, d], fp32; la
    [B, T, H, d or 1] or None.  Blocks of about sqrt(T) tokens: the tokens of
    every block in turn, then the blocks in turn.  e^la - 1 is used in place
    of e^la, which near 1 would lose the decay's digits; la = -inf clears."""
    B, T, H, d = x.shape
    C = max(1, int(round(math.sqrt(T))))
    n = (T + C - 1) // C
    h = torch.zeros(B, n * C, H, d, dtype=x.dtype, device=x.device)
    h[:, :T] = x
    h = h.view(B, n, C, H, d)
    if la is None:
        la = torch.zeros(1, 1, 1, 1, dtype=x.dtype, device=x.device).expand(
            B, T, 1, 1)
    g = torch.zeros(B, n * C, la.shape[2], la.shape[3], dtype=x.dtype,
                    device=x.device)
    g[:, :T] = la
    g = g.view(B, n, C, *g.shape[2:])
    e = torch.expm1(g)
    for i in range(1, C):
        h[:, :, i] += h[:, :, i - 1] + e[:, :, i] * h[:, :, i - 1]
    e = torch.expm1(torch.cumsum(g, 2))
    carry = torch.zeros_like(h[:, 0, 0])
    carries = []
    for j in range(n):
        carries.append(carry)
        carry = h[:, j, C - 1] + carry + e[:, j, C - 1] * carry
    c = torch.stack(carries, 1)[:, :, None]
    h = h + c + e * c
    return h.view(B, n * C, H, d)[:, :T]


def _plain_decay(st):
    """log_alpha as [.., H, d or 1] fp32, cleared where a sequence starts."""
    la = st["log_alpha"]
    x = st["x"]
    if la is None:
        la = torch.zeros(*x.shape[:-1], 1, device=x.device)
    elif la.dim() < x.dim():
        la = la[..., None]
    return la


def _plain_linear(st):
    x = st["x"].float()
    la = _plain_decay(st)
    s0, cu = st["s0"], st["cu"]
    final = (s0.clone() if s0 is not None else
             torch.zeros(len(x) if cu is None else len(cu) - 1, *x.shape[2:],
                         device=x.device))
    if cu is None:
        if s0 is not None:
            x = x.clone() if x is st["x"] else x
            x[:, 0] += s0 + torch.expm1(la[:, 0]) * s0
        h = _scan(x, la)
        final[:] = h[:, -1]
        prev = torch.cat([torch.zeros_like(h[:, :1]) if s0 is None else
                          s0[:, None], h[:, :-1]], 1)
        return h, prev, la, final
    first, last, some = st["first"], st["last"], st["some"]
    reset = la.clone()
    reset[0, first] = float("-inf")
    if s0 is not None:
        x = x.clone() if x is st["x"] else x
        x[0, first] += s0[some] + torch.expm1(la[0, first]) * s0[some]
    h = _scan(x, reset)
    final[some] = h[0, last]
    prev = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    prev[0, first] = 0.0 if s0 is None else s0[some]
    return h, prev, la, final


def _plain_linear_train(st):
    dt = st["x"].dtype
    h, prev, la, final = _plain_linear(st)
    dout = st["d_out"].float()
    ds = st["d_state"]
    cu = st["cu"]
    dout = dout.clone() if dout is st["d_out"] else dout
    ds0 = ds.clone()
    nxt = torch.zeros_like(la)
    nxt[:, :-1] = la[:, 1:]
    if cu is None:
        dout[:, -1] += ds
    else:
        dout[0, st["last"]] += ds[st["some"]]
        nxt[0, st["last"]] = float("-inf")
    G = _scan(dout.flip(1), nxt.flip(1)).flip(1)
    alpha = torch.exp(la)
    aG = alpha * G
    if cu is None:
        ds0[:] = aG[:, 0]
    else:
        ds0[st["some"]] = aG[0, st["first"]]
    gate = st["case"]["gate"]
    dla = None if gate == "none" else aG * prev
    if gate == "scalar":
        dla = dla.sum(-1)
    out = dict(out=h.to(dt), final_state=final, dx=G.to(dt))
    if dla is not None:
        out["dlog_alpha"] = dla
    if st["s0"] is not None:
        out["dinitial_state"] = ds0
    return out


def _plain_norm(st):
    x = st["x"].float()
    c = x - x.mean(-1, keepdim=True)
    rstd = torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS)
    return (c * rstd * st["weight"] + st["bias"]).to(st["x"].dtype)


def _plain_norm_bwd(st):
    x, dy, w = st["x"].float(), st["d_out"].float(), st["weight"]
    c = x - x.mean(-1, keepdim=True)
    rstd = torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS)
    xh = c * rstd
    g = dy * w
    dx = rstd * (g - g.mean(-1, keepdim=True)
                 - xh * (g * xh).mean(-1, keepdim=True))
    return dict(dx=dx.to(st["x"].dtype), dweight=(dy * xh).sum(0),
                dbias=dy.sum(0))


# --------------------------------------------------------------------- run

def run(st):
    op = st["case"]["op"]
    if own:
        return _run_own(op, st)
    if op == "linear_fwd":
        h, _, _, final = _plain_linear(st)
        return h.to(st["x"].dtype), final
    if op == "linear_step":
        x, s = st["x"].float(), st["state"]
        h = s + torch.expm1(_plain_decay(st)) * s + x
        return h.to(st["x"].dtype), h
    if op == "linear_train":
        return _plain_linear_train(st)
    if op == "layer_norm":
        return _plain_norm(st)
    return _plain_norm_bwd(st)


def _run_own(op, st):
    import chunkwise_recurrence_b200 as gdr
    if op == "linear_fwd":
        return gdr.linear_fwd(st["x"], st["log_alpha"], st["s0"],
                              cu_seqlens=st["cu"])
    if op == "linear_step":
        return gdr.linear_step(st["x"], st["log_alpha"], st["state"],
                               state_out=st["state_out"])
    if op == "linear_train":
        out, final, chunk_states = gdr.linear_fwd(
            st["x"], st["log_alpha"], st["s0"], cu_seqlens=st["cu"],
            output_chunk_states=True)
        grads = gdr.linear_backward(
            st["x"], st["log_alpha"], st["s0"], st["d_out"], st["d_state"],
            chunk_states=chunk_states, cu_seqlens=st["cu"],
            need_initial_state_grad=st["s0"] is not None)
        res = dict(out=out, final_state=final, dx=grads["dx"])
        for key in ("dlog_alpha", "dinitial_state"):
            if grads[key] is not None:
                res[key] = grads[key]
        return res
    if op == "layer_norm":
        return gdr.layer_norm(st["x"], st["weight"], st["bias"], eps=EPS)
    g = gdr.layer_norm_backward(st["x"], st["weight"], st["d_out"], eps=EPS)
    return dict(dx=g["dx"], dweight=g["dweight"], dbias=g["dbias"])


# -------------------------------------------------------------------- work

def work(case):
    H, d = case["H"], case["d"]
    es = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op.startswith("layer_norm"):
        n = case["ntok"] * H * d
        if op == "layer_norm":
            return {"bytes": 2 * es * n + 8 * H * d, "flops": 8 * n}
        return {"bytes": 3 * es * n + 12 * H * d, "flops": 18 * n}
    _, nseq, ntok = _grid(case)
    n = ntok * H * d
    la = {"none": 0, "scalar": 4 * ntok * H, "channel": 4 * n}[case["gate"]]
    state = 4 * nseq * H * d
    if op == "linear_step":
        return {"bytes": 2 * es * n + la + 2 * state, "flops": 4 * n}
    init = state if case["init"] else 0
    if op == "linear_fwd":
        return {"bytes": 2 * es * n + la + init + state, "flops": 4 * n}
    return {"bytes": 4 * es * n + 2 * la + 2 * init + 2 * state,
            "flops": 12 * n}


# ------------------------------------------------------------------- exact

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    f = lambda t: None if t is None else t.double()  # noqa: E731
    x = f(st["x"])
    if op.startswith("layer_norm"):
        w, b = f(st["weight"]), f(st["bias"])
        d = x.shape[-1]
        mu = x.sum(-1, keepdim=True) / d
        var = ((x - mu) ** 2).sum(-1, keepdim=True) / d
        xh = (x - mu) / torch.sqrt(var + EPS)
        if op == "layer_norm":
            return xh * w + b
        dy = f(st["d_out"])
        g = dy * w
        m1 = g.sum(-1, keepdim=True) / d
        m2 = (g * xh).sum(-1, keepdim=True) / d
        return dict(dx=(g - m1 - xh * m2) / torch.sqrt(var + EPS),
                    dweight=(dy * xh).sum(0), dbias=dy.sum(0))
    la = f(st["log_alpha"])
    if la is None:
        a = torch.ones_like(x[..., :1])
    else:
        a = torch.exp(la if la.dim() == x.dim() else la[..., None])
    if op == "linear_step":
        h = a * f(st["state"]) + x
        return h, h
    # one sequence after the other, token by token
    B, T = x.shape[:2]
    x, a = x.flatten(0, 1), a.flatten(0, 1)
    cu = ([i * T for i in range(B + 1)] if st["cu"] is None
          else st["cu"].tolist())
    nseq = len(cu) - 1
    s0 = f(st["s0"])
    if s0 is None:
        s0 = torch.zeros(nseq, *x.shape[1:], dtype=x.dtype, device=x.device)
    h = torch.empty_like(x)
    prev = torch.empty_like(x)
    final = s0.clone()
    for n in range(nseq):
        s = s0[n]
        for t in range(cu[n], cu[n + 1]):
            prev[t] = s
            s = torch.addcmul(x[t], a[t], s, out=h[t])
        final[n] = s
    shape = st["x"].shape
    if op == "linear_fwd":
        return h.view(shape), final
    dout, ds = f(st["d_out"]).flatten(0, 1), f(st["d_state"])
    G = torch.empty_like(x)
    ds0 = ds.clone()
    for n in range(nseq):
        c = ds[n]
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            torch.add(dout[t], c, out=G[t])
            c = a[t] * G[t]
        ds0[n] = c
    out = dict(out=h.view(shape), final_state=final, dx=G.view(shape))
    if case["gate"] != "none":
        dla = a * G * prev
        if case["gate"] == "scalar":
            dla = dla.sum(-1)
        out["dlog_alpha"] = dla.view(st["log_alpha"].shape)
    if st["s0"] is not None:
        out["dinitial_state"] = ds0
    return out

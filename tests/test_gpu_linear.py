"""GPU parity of the gated linear recurrence (forward, step, backward) with
the fp64 token loop of oracle/linear_ref.py.

Tolerances, from the arithmetic (u = 2^-24).  M_t, the same recurrence run on
|x| and |h0|, bounds every partial result.  A term of h_t is rounded at most
four times in each join it passes (the composed decay, its product with the
value, the multiply-add, the sum): its run (at most 32 tokens, twice), the
joins inside a warp, a block and a cluster (at most 16) and one per 32-token
tile of the sequence.  A decay e^s with s below -1/8 is off by up to 3 + 1.2
|s| units of 2^-23 of e^s, which no more than 1 / (1 - e^-1/8) = 8.5 such
steps in a row carry on: e^s (3 + 1.2 |s|) <= 3, so 2 * 3 * 8.5 u; the sum of
a run's log-decays adds another 12 u at most.  (A product of decays that is
held as alpha - 1 is off by up to 3 u of the value before it, not of itself;
M changes little over the tokens of a tile of these inputs.)  Together
    |h - ref| <= K_T u M_t,   K_T = 4 (64 + 16 + T / 32) + 64,
and half a step of the output's type.  The same holds for G backwards.  A
product G alpha h adds the two errors and its own rounding; a sum over d
channels up to d u of the sum of magnitudes."""
import ctypes
import threading

import numpy as np
import pytest
import torch

import chunkwise_recurrence_b200 as gdr
import oracle

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


def kt(T):
    return 4 * (80 + T / 32) + 64


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def mag(t):
    return None if t is None else np.abs(f64(t))


def inputs(B, T, H, d, dtype, gate, *, cu=None, init=True, seed=0, scale=0.3,
           special=False):
    g = torch.Generator().manual_seed(seed)
    n = B if cu is None else len(cu) - 1
    x = torch.randn(B, T, H, d, generator=g).to(DT[dtype])
    shape = {"none": None, "scalar": (B, T, H),
             "channel": (B, T, H, d)}[gate]
    la = None
    if shape is not None:
        la = -torch.rand(*shape, generator=g) * scale
        if special:    # no decay at all, hardly any, hard resets
            u = torch.rand(*shape, generator=g)
            la[u < 0.3] = 0.0
            la[(u >= 0.3) & (u < 0.6)] *= 1e-4
            la[u > 0.95] = -30.0
            la[u > 0.98] = float("-inf")
    s0 = torch.randn(n, H, d, generator=g) if init else None
    dO = torch.randn(B, T, H, d, generator=g).to(DT[dtype])
    dS = torch.randn(n, H, d, generator=g)
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    return c(x), c(la), c(s0), c(dO), c(dS)


def cu_tensor(cu):
    return None if cu is None else torch.tensor(cu, dtype=torch.int32,
                                                device="cuda")


def rev_bound(la, dO, dS, cu, shape):
    """M of the backward scan, and of alpha_1 G_1."""
    got = oracle.linear_grads(np.zeros(shape), f64(la), None, mag(dO),
                              mag(dS), cu)
    return got["dx"], got["dinitial_state"]


def check_fwd(x, la, s0, out, fin, cu=None):
    T = x.shape[1]
    ref, rf, _ = oracle.linear_fwd(f64(x), f64(la), f64(s0), cu)
    m, mf, _ = oracle.linear_fwd(mag(x), f64(la), mag(s0), cu)
    tol = kt(T) * U * m
    assert (np.abs(f64(out) - ref) <= tol + HALF[x.dtype] * (np.abs(ref) +
                                                              tol)).all()
    if fin is not None:
        assert (np.abs(f64(fin) - rf) <= kt(T) * U * mf).all()


def check_bwd(x, la, s0, dO, dS, res, cu=None):
    T, d = x.shape[1], x.shape[3]
    ref = oracle.linear_grads(f64(x), f64(la), f64(s0), f64(dO), f64(dS), cu)
    mg, mc = rev_bound(la, dO, dS, cu, x.shape)
    k = kt(T) * U
    tol = k * mg
    assert (np.abs(f64(res["dx"]) - ref["dx"]) <=
            tol + HALF[x.dtype] * (np.abs(ref["dx"]) + tol)).all()
    if res["dinitial_state"] is not None:
        assert (np.abs(f64(res["dinitial_state"]) - ref["dinitial_state"]) <=
                k * mc).all()
    if la is None:
        assert res["dlog_alpha"] is None
        return
    _, _, mah = oracle.linear_fwd(mag(x), f64(la), mag(s0), cu)
    bound = mg * mah
    if la.dim() == 3:
        tol = (2 * k + (d + 8) * U) * bound.sum(-1)
    else:
        tol = (2 * k + 2 * U) * bound
    assert (np.abs(f64(res["dlog_alpha"]) - ref["dlog_alpha"]) <= tol).all()


SHAPES = [(1, 1, 1, 16), (2, 7, 3, 33), (1, 31, 2, 100), (3, 32, 1, 4),
          (2, 33, 5, 1), (1, 64, 16, 128), (2, 65, 2, 72), (1, 255, 2, 36),
          (1, 256, 1, 64), (2, 257, 4, 20), (1, 1000, 3, 50),
          (1, 2600, 2, 48), (1, 1500, 1, 37), (3, 300, 5, 13)]


@pytest.mark.parametrize("gate", ["none", "scalar", "channel"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward_match_oracle(shape, dtype, gate):
    for init in (True, False):
        x, la, s0, dO, dS = inputs(*shape, dtype, gate, init=init)
        out, fin, cs = gdr.linear_fwd(x, la, s0, output_chunk_states=True)
        res = gdr.linear_backward(x, la, s0, dO, dS, chunk_states=cs)
        again = gdr.linear_backward(x, la, s0, dO, dS)
        torch.cuda.synchronize()
        check_fwd(x, la, s0, out, fin)
        check_bwd(x, la, s0, dO, dS, res)
        # the chunk states computed again are the same, bit for bit
        for key in res:
            assert res[key] is None and again[key] is None or torch.equal(
                res[key], again[key]), key


PACKED = [([0, 1], 2, 8), ([0, 0, 5, 5, 6, 40], 3, 12),
          ([0, 300, 300, 301, 700, 1500], 2, 40),
          ([0, 33, 66, 99, 131, 163, 196], 1, 7)]


@pytest.mark.parametrize("gate", ["none", "scalar", "channel"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("case", PACKED)
def test_packed_sequences_match_oracle(case, dtype, gate):
    cu, H, d = case
    x, la, s0, dO, dS = inputs(1, cu[-1], H, d, dtype, gate, cu=cu)
    cut = cu_tensor(cu)
    out, fin, cs = gdr.linear_fwd(x, la, s0, cu_seqlens=cut,
                                  output_chunk_states=True)
    res = gdr.linear_backward(x, la, s0, dO, dS, cu_seqlens=cut,
                              chunk_states=cs)
    torch.cuda.synchronize()
    check_fwd(x, la, s0, out, fin, cu)
    check_bwd(x, la, s0, dO, dS, res, cu)


@pytest.mark.parametrize("gate", ["scalar", "channel"])
@pytest.mark.parametrize("shape", [(2, 90, 2, 40), (1, 1200, 2, 36)])
def test_resets_and_no_decay_match_oracle(shape, gate):
    """log_alpha of 0, of next to nothing, of -30 and of -inf."""
    x, la, s0, dO, dS = inputs(*shape, "fp32", gate, special=True)
    out, fin, cs = gdr.linear_fwd(x, la, s0, output_chunk_states=True)
    res = gdr.linear_backward(x, la, s0, dO, dS, chunk_states=cs)
    torch.cuda.synchronize()
    check_fwd(x, la, s0, out, fin)
    check_bwd(x, la, s0, dO, dS, res)


def test_reset_clears_a_huge_state_exactly():
    T = 300
    x = torch.zeros(1, T, 1, 32, device="cuda")
    la = torch.full((1, T, 1, 32), -0.01, device="cuda")
    la[0, ::50] = float("-inf")
    s0 = torch.full((1, 1, 32), 1e30, device="cuda")
    out, fin = gdr.linear_fwd(x, la, s0)
    assert not out.any() and not fin.any()


def test_long_memory_keeps_the_decay_s_digits():
    """A constant decay of 1e-5 a token: h -> 1e5 (1 - e^{-1e-5 t}).  alpha
    rounded to fp32 would be off by 1e-3 of the decay, and h with it."""
    T = 40000
    x = torch.ones(1, T, 1, 4, device="cuda")
    la = torch.full((1, T, 1, 4), -1e-5, device="cuda")
    out, _ = gdr.linear_fwd(x, la)
    l64 = float(np.float32(-1e-5))
    t = np.arange(1, T + 1)
    ref = np.expm1(l64 * t) / np.expm1(l64)
    got = f64(out)[0, :, 0, :]
    # no rounding is carried on but those of h itself: one per token of a run,
    # join and tile
    assert (np.abs(got - ref[:, None]) <= kt(T) * U * ref[:, None]).all()


@pytest.mark.parametrize("gate", ["scalar", "channel"])
@pytest.mark.parametrize("decay", [0.01, 0.05, 0.12, 0.124, 0.126, 0.3])
def test_a_decaying_state_keeps_its_digits(decay, gate):
    """A state that nothing is added to, token after token.  Decays of a warp's
    32 tokens are composed as alpha - 1, off by 3 u of the state before them:
    3 u e^(32 decay) of the state after them, where they are at all (a run of 8
    tokens no further down than 1 / e); the rest as elsewhere."""
    T = 640
    x = torch.zeros(1, T, 1, 64, device="cuda")
    la = torch.full((1, T, 1) if gate == "scalar" else (1, T, 1, 64), -decay,
                    device="cuda")
    s0 = torch.ones(1, 1, 64, device="cuda")
    out, fin = gdr.linear_fwd(x, la, s0)
    ref = np.exp(-float(np.float32(decay)) * np.arange(1, T + 1))
    per_tile = 3 * np.exp(32 * min(decay, 0.125))
    tol = (kt(T) + per_tile * T / 32) * U * ref + 2.0 ** -126
    assert (np.abs(f64(out)[0, :, 0, :] - ref[:, None]) <= tol[:, None]).all()


def test_rows_outside_the_sequences_are_left_as_they_were():
    cu = [4, 40, 40, 90]
    T, H, d = 130, 2, 20
    for gate in ("none", "scalar", "channel"):
        x, la, s0, dO, dS = inputs(1, T, H, d, "fp32", gate, cu=cu)
        out = torch.full_like(x, 7.0)
        _, fin = gdr.linear_fwd(x, la, s0, cu_seqlens=cu_tensor(cu), out=out)
        assert (out[0, :4] == 7).all() and (out[0, 90:] == 7).all()
        ref, rf, _ = oracle.linear_fwd(f64(x), f64(la), f64(s0), cu)
        assert np.allclose(f64(out)[0, 4:90], ref[0, 4:90], atol=1e-4)
        assert np.allclose(f64(fin), rf, atol=1e-4)


@pytest.mark.parametrize("gate", ["none", "scalar", "channel"])
@pytest.mark.parametrize("d", [20, 100])
def test_gradients_outside_the_sequences_are_left_as_they_were(gate, d):
    """Through the C ABI, into buffers that already hold something."""
    cu, T, H = [4, 40, 40, 90], 130, 2
    x, la, s0, dO, dS = inputs(1, T, H, d, "fp32", gate, cu=cu)
    dx = torch.full_like(x, 7.0)
    dla = None if la is None else torch.full_like(la, 7.0)
    ds0 = torch.empty_like(s0)
    cut = cu_tensor(cu)
    opts = gdr._Opts(dtype=gdr.DTYPES[torch.float32], gate=gdr.GATES[gate],
                     cu_seqlens=cut.data_ptr(), num_seqs=len(cu) - 1,
                     algo=gdr.ALGOS["auto"])
    fp = ctypes.POINTER(ctypes.c_float)
    f = lambda t: None if t is None else ctypes.cast(t.data_ptr(), fp)  # noqa: E731
    rc = gdr.load_library().gdr_linear_backward(
        x.data_ptr(), H * d, f(la), f(s0), None, dO.data_ptr(), f(dS),
        dx.data_ptr(), f(dla), f(ds0), 1, T, H, d,
        torch.cuda.current_stream().cuda_stream, ctypes.byref(opts))
    assert rc == 0
    torch.cuda.synchronize()
    for t in (dx, dla):
        if t is not None:
            assert (t[0, :4] == 7).all() and (t[0, 90:] == 7).all()
            t[0, :4] = 0
            t[0, 90:] = 0
    check_bwd(x, la, s0, dO, dS, dict(dx=dx, dlog_alpha=dla,
                                      dinitial_state=ds0), cu)


def test_many_short_sequences():
    """A warp per chain, more chains than the GPU holds at once."""
    B, T, H, d = 700, 40, 4, 64
    x, la, s0, dO, dS = inputs(B, T, H, d, "bf16", "channel")
    out, fin, cs = gdr.linear_fwd(x, la, s0, output_chunk_states=True)
    res = gdr.linear_backward(x, la, s0, dO, dS, chunk_states=cs)
    torch.cuda.synchronize()
    check_fwd(x, la, s0, out, fin)
    check_bwd(x, la, s0, dO, dS, res)


@pytest.mark.parametrize("gate", ["none", "scalar", "channel"])
def test_strided_tokens(gate):
    """x as a column range of a wider projection."""
    B, T, H, d = 2, 70, 2, 24
    x, la, s0, dO, dS = inputs(B, T, H, d, "bf16", gate)
    for width, at in ((H * d + 48, 16), (H * d + 9, 0)):
        wide = torch.randn(B, T, width, device="cuda").to(x.dtype)
        wide[..., at:at + H * d] = x.view(B, T, H * d)
        xs = wide[..., at:at + H * d].unflatten(-1, (H, d))
        assert not xs.is_contiguous()
        a = gdr.linear_fwd(x, la, s0, output_chunk_states=True)
        b = gdr.linear_fwd(xs, la, s0, output_chunk_states=True)
        ga = gdr.linear_backward(x, la, s0, dO, dS)
        gb = gdr.linear_backward(xs, la, s0, dO, dS, chunk_states=b[2])
        torch.cuda.synchronize()
        check_fwd(x, la, s0, b[0], b[1])
        check_bwd(x, la, s0, dO, dS, gb)
        if width % 4 == 0:      # the same loads, hence the same bits
            assert all(torch.equal(p, q) for p, q in zip(a[:2], b[:2]))
            assert torch.equal(ga["dx"], gb["dx"])
        sa = gdr.linear_step(x[:, 0], None if la is None else
                             la[:, 0].contiguous(), s0, state_out=s0.clone())
        sb = gdr.linear_step(xs[:, 0], None if la is None else
                             la[:, 0].contiguous(), s0, state_out=s0.clone())
        assert torch.equal(sa[0], sb[0]) and torch.equal(sa[1], sb[1])


@pytest.mark.parametrize("gate", ["none", "scalar", "channel"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 41, 1, 37), (2, 300, 3, 20),
                                   (1, 700, 1, 5)])
def test_nothing_is_written_beside_the_results(shape, dtype, gate):
    x, la, s0, dO, dS = inputs(*shape, dtype, gate)
    n = x.numel()
    wide = torch.full((n + 64,), 7.0, dtype=x.dtype, device="cuda")
    fin = torch.full((s0.numel() + 64,), 7.0, device="cuda")
    gdr.linear_fwd(x, la, s0, out=wide[32:32 + n].view(x.shape),
                   final_state=fin[32:32 + s0.numel()].view(s0.shape))
    torch.cuda.synchronize()
    check_fwd(x, la, s0, wide[32:32 + n].view(x.shape),
              fin[32:32 + s0.numel()].view(s0.shape))
    for t, m in ((wide, n), (fin, s0.numel())):
        assert (t[:32] == 7).all() and (t[32 + m:] == 7).all()


@pytest.mark.parametrize("gate", ["none", "scalar", "channel"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("nhd", [(1, 1, 1), (3, 2, 33), (5, 4, 64),
                                 (300, 16, 128)])
def test_step_matches_oracle_and_updates_in_place(nhd, dtype, gate):
    N, H, d = nhd
    x, la, s0, _, _ = inputs(N, 1, H, d, dtype, gate)
    x1 = x[:, 0]
    la1 = None if la is None else la[:, 0].contiguous()
    state = s0.clone()
    out, st = gdr.linear_step(x1, la1, state)
    torch.cuda.synchronize()
    assert st is state
    check_fwd(x, la, s0, out[:, None], state)
    out2, st2 = gdr.linear_step(x1, la1, s0, state_out=torch.empty_like(s0))
    assert torch.equal(out, out2) and torch.equal(state, st2)
    out3, st3 = gdr.linear_step(x1, la1)      # no state: zero
    torch.cuda.synchronize()
    check_fwd(x, la, None, out3[:, None], st3)


def test_step_continues_a_prompt():
    T, extra = 100, 5
    x, la, s0, _, _ = inputs(2, T + extra, 2, 20, "fp32", "channel")
    out, fin = gdr.linear_fwd(x[:, :T].contiguous(), la[:, :T].contiguous(),
                              s0)
    outs = [out]
    for t in range(T, T + extra):
        o, fin = gdr.linear_step(x[:, t], la[:, t].contiguous(), fin)
        outs.append(o[:, None])
    torch.cuda.synchronize()
    check_fwd(x, la, s0, torch.cat(outs, 1), fin)


def test_no_tokens_keep_the_state():
    H, d = 2, 12
    s0 = torch.randn(3, H, d, device="cuda")
    x = torch.empty(3, 0, H, d, device="cuda")
    la = torch.empty(3, 0, H, device="cuda")
    out, fin, cs = gdr.linear_fwd(x, la, s0, output_chunk_states=True)
    assert out.numel() == 0 and torch.equal(fin, s0)
    res = gdr.linear_backward(x, la, s0, torch.empty_like(x), s0,
                              chunk_states=cs)
    assert torch.equal(res["dinitial_state"], s0)
    res = gdr.linear_backward(x, la, s0, torch.empty_like(x))
    assert not res["dinitial_state"].any()
    none = gdr.linear_fwd(torch.empty(0, 5, H, d, device="cuda"))
    assert none[0].shape == (0, 5, H, d) and none[1].shape == (0, H, d)
    assert gdr.linear_step(torch.empty(0, H, d, device="cuda"))[0].numel() == 0


def test_not_a_number_stays_in_its_channel():
    x, la, s0, dO, dS = inputs(1, 600, 2, 32, "fp32", "channel")
    clean = gdr.linear_fwd(x, la, s0)[0]
    x[0, 300, 0, 5] = float("nan")
    x[0, 300, 1, 7] = float("inf")
    out = gdr.linear_fwd(x, la, s0)[0]
    torch.cuda.synchronize()
    assert torch.isnan(out[0, 300:, 0, 5]).all()
    assert torch.isinf(out[0, 300, 1, 7])
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[0, 300:, 0, 5] = keep[0, 300:, 1, 7] = False
    assert torch.equal(out[keep], clean[keep])


def test_other_stream_and_repeatable():
    x, la, s0, dO, dS = inputs(1, 2000, 3, 40, "bf16", "scalar")
    a = gdr.linear_fwd(x, la, s0)
    ga = gdr.linear_backward(x, la, s0, dO, dS)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        b = gdr.linear_fwd(x, la, s0, stream=s)
        gb = gdr.linear_backward(x, la, s0, dO, dS, stream=s)
        s.synchronize()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        assert all(torch.equal(ga[k], gb[k]) for k in ga)


def test_two_streams_at_once():
    """Training steps with scratch, in flight on two streams together."""
    cases = [inputs(1, 3000, 2, 40, "fp32", "scalar", seed=s) for s in (1, 2)]
    want = [gdr.linear_backward(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        got = [gdr.linear_backward(*c, stream=s)
               for c, s in zip(cases, streams)]
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            assert all(torch.equal(w[k], g[k]) for k in w)


@pytest.mark.parametrize("T", [20, 300, 3000])
def test_growing_states(T):
    """log_alpha above 0 is outside what is expected, but means what it
    says."""
    x, la, s0, dO, dS = inputs(1, T, 1, 36, "fp32", "channel")
    la = -la * (3.0 / T)
    out, fin = gdr.linear_fwd(x, la, s0)
    res = gdr.linear_backward(x, la, s0, dO, dS)
    torch.cuda.synchronize()
    check_fwd(x, la, s0, out, fin)
    check_bwd(x, la, s0, dO, dS, res)


def test_captured_steps_share_nothing():
    """Two captured training steps with scratch, replayed in turn on new
    inputs, and the eager calls agree bit for bit."""
    cases, graphs = [], []
    for seed, gate in ((1, "scalar"), (2, "channel")):
        x, la, s0, dO, dS = inputs(2, 700, 2, 40, "fp32", gate, seed=seed)
        run = lambda a=(x, la, s0, dO, dS): (  # noqa: E731
            gdr.linear_fwd(*a[:3]), gdr.linear_backward(*a))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            run()
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = run()
        cases.append((x, la, s0, dO, dS, run, res))
        graphs.append(g)
    for rep in range(3):
        for i in (0, 1):
            for t in cases[i][:1] + cases[i][2:5]:
                t.normal_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for x, la, s0, dO, dS, run, ((o, f), gr) in cases:
            (o2, f2), gr2 = run()
            torch.cuda.synchronize()
            assert torch.equal(o, o2) and torch.equal(f, f2)
            assert all(torch.equal(gr[k], gr2[k]) for k in gr)


def test_binding_refuses_what_the_kernels_cannot_take():
    x, la, s0, dO, dS = inputs(2, 8, 2, 16, "bf16", "channel")
    bad = [
        lambda: gdr.linear_fwd(x.cpu(), la),
        lambda: gdr.linear_fwd(x.half(), la),
        lambda: gdr.linear_fwd(x[0], la),
        lambda: gdr.linear_fwd(x.transpose(2, 3), la),
        lambda: gdr.linear_fwd(x.transpose(0, 1), la),
        lambda: gdr.linear_fwd(x[:, :1].expand(2, 8, 2, 16), la),
        lambda: gdr.linear_fwd(x, la.bfloat16()),
        lambda: gdr.linear_fwd(x, la[:, :-1]),
        lambda: gdr.linear_fwd(x, la, gate="scalar"),
        lambda: gdr.linear_fwd(x, None, gate="scalar"),
        lambda: gdr.linear_fwd(x, la, gate="none"),
        lambda: gdr.linear_fwd(x, la, gate="both"),
        lambda: gdr.linear_fwd(x, la, s0[:1]),
        lambda: gdr.linear_fwd(x, la, s0.cpu()),
        lambda: gdr.linear_fwd(x, la, cu_seqlens=cu_tensor([0, 8])),
        lambda: gdr.linear_fwd(x[:1], la[:1], cu_seqlens=torch.tensor(
            [0, 8], device="cuda")),
        lambda: gdr.linear_fwd(x, la, out=x.float()),
        lambda: gdr.linear_backward(x, la, s0, dO.float(), dS),
        lambda: gdr.linear_backward(x, la, s0, dO.transpose(2, 3), dS),
        lambda: gdr.linear_backward(x, la, s0, dO, dS, chunk_states=s0[:1]),
        lambda: gdr.linear_step(x, la),
        lambda: gdr.linear_step(x[:, 0], la[:, 0].contiguous(), s0.double()),
        lambda: gdr.linear_step(x[:, 0], la[:, 0]),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(gdr.GdrError):          # written over its input
        gdr.linear_fwd(x, la, out=x)
    with pytest.raises(gdr.GdrError):          # base off by two bytes
        wide = torch.zeros(2, 8, 40, device="cuda", dtype=torch.bfloat16)
        gdr.linear_fwd(wide[..., 1:33].unflatten(-1, (2, 16)), la)


def test_an_expired_wait_is_reported(monkeypatch):
    """CTAs of a cluster that never hear from one another give up, the call
    ends and says so, and the next one is right."""
    x, la, s0, dO, dS = inputs(1, 2000, 1, 64, "fp32", "channel")
    monkeypatch.setenv("GDR_FAULT_INJECT_LINEAR_TIMEOUT", "1")
    gdr.linear_fwd(x, la, s0)
    assert gdr.STATUS[gdr.device_error()] == "GDR_ERR_TIMEOUT"
    monkeypatch.delenv("GDR_FAULT_INJECT_LINEAR_TIMEOUT")
    out, fin = gdr.linear_fwd(x, la, s0)
    assert gdr.device_error() == 0
    check_fwd(x, la, s0, out, fin)


@pytest.mark.parametrize("d", [128, 127])
def test_more_values_than_32_bits_can_count(d):
    """The last tokens of 2^31 values and more, forward and backward, against
    the same tokens on their own."""
    H, T, last = 16, (2 ** 31 + 2 ** 23) // (16 * d), 700
    x = torch.zeros(1, T, H, d, dtype=torch.bfloat16, device="cuda")
    la = torch.full((1, T, H), -0.05, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    x[:, -last:] = torch.randn(last, H, d, generator=g, device="cuda").to(x)
    out, fin = gdr.linear_fwd(x, la)
    tail, latail = x[:, -last:].contiguous(), la[:, -last:].contiguous()
    check_fwd(tail, latail, None, out[:, -last:], fin)
    del out
    res = gdr.linear_backward(x, la, None, x, fin)
    torch.cuda.synchronize()
    check_bwd(tail, latail, torch.zeros_like(fin), tail, fin,
              dict(dx=res["dx"][:, -last:], dinitial_state=None,
                   dlog_alpha=res["dlog_alpha"][:, -last:]))
    # far before the last tokens nothing is left of anything
    assert res["dx"][:, :T // 2].abs().max() <= 2.0 ** -126
    assert res["dinitial_state"].abs().max() <= 2.0 ** -126
    del x, res
    torch.cuda.empty_cache()


def test_two_threads_at_once():
    """Each on a stream of its own; launches do not hold the interpreter."""
    cases = [inputs(1, 2000, 2, 40, "fp32", "scalar", seed=s) for s in (1, 2)]
    want = [gdr.linear_backward(*c) for c in cases]
    torch.cuda.synchronize()
    got = [None, None]

    def run(i):
        s = torch.cuda.Stream()
        for _ in range(20):
            got[i] = gdr.linear_backward(*cases[i], stream=s)
        s.synchronize()

    threads = [threading.Thread(target=run, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for w, g in zip(want, got):
        assert all(torch.equal(w[k], g[k]) for k in w)

"""GPU parity of layer normalisation (forward, backward) with fp64
(oracle/norm_ref.py), and of a norm, a linear recurrence and a per-head norm
run together.

Tolerances, from the arithmetic (u = 2^-24).  A sum over a row passes at most
64 additions in a thread, 5 in a warp and 32 over warps: K = 104 u of the mean
of magnitudes.  Per element then
    e_c  = K mean|x| + 2 u |x|                  error of x - mean
    e_r  = K + 6 u + 2 u rms(x) rstd            relative error of rstd
    e_xh = rstd e_c + |xh| e_r                  error of xh = (x - mean) rstd
and y = xh w + b is off by |w| e_xh + 3 u (|xh w| + |b|) and half a step of
its type.  Backwards m1 = mean(g) by K mean|g|, m2 = mean(g xh) by
K mean|g xh| + mean(|g| e_xh), dx by what those leave times rstd, and a sum
over n tokens by (n + 20) u of the sum of magnitudes and sum |dy| e_xh."""
import numpy as np
import pytest
import torch

import chunkwise_recurrence_b200 as gdr
import oracle

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
K = 104 * U
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def inputs(n, H, d, dtype, seed=0, offset=2.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, H, d, generator=g)
    x *= torch.exp(torch.randn(n, 1, 1, generator=g))
    x += offset * torch.randn(n, H, 1, generator=g)
    x[..., :: max(1, d // 3)] *= 10.0
    w = torch.randn(H, d, generator=g)
    b = torch.randn(H, d, generator=g)
    dy = torch.randn(n, H, d, generator=g)
    dt = DT[dtype]
    return x.to(dt).cuda(), w.cuda(), b.cuda(), dy.to(dt).cuda()


def parts(x, eps):
    mean = lambda a: a.mean(-1, keepdims=True)  # noqa: E731
    c = x - mean(x)
    rstd = 1 / np.sqrt(mean(c * c) + eps)
    xh = c * rstd
    e_c = K * mean(np.abs(x)) + 2 * U * np.abs(x)
    e_r = K + 6 * U + 2 * U * np.sqrt(mean(x * x)) * rstd
    return xh, rstd, rstd * e_c + np.abs(xh) * e_r, e_r


def check_fwd(x, w, b, y, eps=1e-5):
    half = HALF[x.dtype]
    x, w, b = f64(x), f64(w), f64(b)
    ref = oracle.layer_norm(x, w, b, eps)
    xh, _, e_xh, _ = parts(x, eps)
    w = np.ones_like(xh) if w is None else w
    b = np.zeros_like(xh) if b is None else b
    tol = np.abs(w) * e_xh + 3 * U * (np.abs(xh * w) + np.abs(b))
    assert (np.abs(f64(y).reshape(ref.shape) - ref) <=
            tol + half * (np.abs(ref) + tol)).all()


def check_bwd(x, w, dy, res, eps=1e-5):
    half = HALF[x.dtype]
    n = x.shape[0]
    x, w, dy = f64(x), f64(w), f64(dy)
    ref = oracle.layer_norm_grads(x, w, dy, eps)
    xh, rstd, e_xh, e_r = parts(x, eps)
    g = dy if w is None else dy * w
    mean = lambda a: a.mean(-1, keepdims=True)  # noqa: E731
    a = np.abs
    m1, m2 = mean(g), mean(g * xh)
    e_m1 = K * mean(a(g))
    e_m2 = K * mean(a(g * xh)) + mean(a(g) * e_xh)
    size = a(g) + a(m1) + a(xh * m2)
    tol = rstd * (e_m1 + e_xh * a(m2) + a(xh) * e_m2 + 6 * U * size
                  + e_r * size)
    got = f64(res["dx"]).reshape(ref["dx"].shape)
    assert (a(got - ref["dx"]) <= tol + half * (a(ref["dx"]) + tol)).all()
    if res["dweight"] is not None:
        sum_u = (n + 20) * U
        tw = sum_u * a(dy * xh).sum(0) + (a(dy) * e_xh).sum(0)
        tb = sum_u * a(dy).sum(0)
        shape = ref["dweight"].shape
        assert (a(f64(res["dweight"]).reshape(shape) - ref["dweight"]) <=
                tw).all()
        assert (a(f64(res["dbias"]).reshape(shape) - ref["dbias"]) <=
                tb).all()


SHAPES = [(1, 1, 1), (3, 1, 2), (5, 2, 8), (7, 3, 9), (4, 5, 16), (9, 1, 31),
          (33, 16, 128), (6, 7, 64), (2, 3, 100), (65, 1, 257), (17, 2, 300),
          (40, 1, 1001), (21, 1, 2048), (9, 2, 2056), (300, 1, 512),
          (5, 1, 4097), (6, 1, 5120), (3, 1, 8192), (2, 1, 12000),
          (3, 1, 16383), (2, 1, 16384), (700, 33, 24), (10000, 1, 77),
          (4000, 5, 101), (3001, 1, 1001), (1300, 1, 2047), (900, 1, 4101)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward_match_oracle(shape, dtype):
    x, w, b, dy = inputs(*shape, dtype)
    y = gdr.layer_norm(x, w, b)
    res = gdr.layer_norm_backward(x, w, dy)
    torch.cuda.synchronize()
    check_fwd(x, w, b, y)
    check_bwd(x, w, dy, res)


# many tokens: persistent blocks, with the sums added per group, per block by
# one or several groups of a head, and heads that do not fill the last block
MANY = [(3000, 1, 24), (2500, 1, 77), (1500, 5, 101), (900, 7, 64),
        (1200, 40, 16), (333, 1, 1001), (700, 1, 2048), (2000, 3, 40)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shape", MANY)
def test_many_tokens_match_oracle(shape, dtype):
    x, w, b, dy = inputs(*shape, dtype, seed=3)
    y = gdr.layer_norm(x, w, b)
    res = gdr.layer_norm_backward(x, w, dy)
    again = gdr.layer_norm_backward(x, w, dy)
    torch.cuda.synchronize()
    check_fwd(x, w, b, y)
    check_bwd(x, w, dy, res)
    assert all(torch.equal(res[k], again[k]) for k in res)


@pytest.mark.parametrize("captured", [False, True])
def test_calls_wait_for_the_ones_before(captured):
    """Launches overlap; a chain of calls that each read what the one before
    wrote, with buffers written over and over, gives what it gives one call
    at a time."""
    x, w, b, dy = inputs(1200, 8, 64, "bf16")
    la = -torch.rand(4, 300, 8, 64, device="cuda") * 0.1
    buf = torch.empty_like(x)
    out = torch.empty(4, 300, 8, 64, dtype=x.dtype, device="cuda")

    def chain(wait):
        got, cur = [], x
        for i in range(6):
            gdr.layer_norm(cur, w, b, out=buf)
            wait()
            _, fin = gdr.linear_fwd(buf.view(4, 300, 8, 64), la, out=out)
            wait()
            res = gdr.layer_norm_backward(out.view(1200, 8, 64), w, buf)
            wait()
            g = gdr.linear_backward(res["dx"].view(4, 300, 8, 64), la, fin,
                                    out, fin)
            wait()
            cur = g["dx"].view(1200, 8, 64)
            step, _ = gdr.linear_step(cur[:7], None, None)
            got += [fin, res["dweight"], res["dbias"], g["dlog_alpha"],
                    g["dinitial_state"], cur, step]
        return got

    want = chain(torch.cuda.synchronize)
    nothing = lambda: None  # noqa: E731
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = chain(nothing)
        for _ in range(2):
            graph.replay()
    else:
        got = chain(nothing)
    torch.cuda.synchronize()
    assert len(got) == len(want)
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_calls_wait_for_copies_and_for_other_streams():
    """What a call reads comes from a copy on its stream, or from another
    stream by an event, with a short call of its own just before."""
    x, w, b, dy = inputs(4000, 16, 128, "bf16")
    xl = x.view(1, 4000, 16, 128)
    small = inputs(64, 16, 128, "bf16")[0]
    want = gdr.linear_fwd(xl)[0]
    norm = gdr.layer_norm(want.view_as(x), w, b)
    host = torch.empty(x.shape, dtype=x.dtype, pin_memory=True)
    host.copy_(x)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    back = torch.empty(x.shape, dtype=x.dtype, pin_memory=True)
    dev, mid, out = (torch.empty_like(x) for _ in range(3))
    for _ in range(10):
        for t in (dev, mid, out):
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            gdr.layer_norm(small, w, b)
            dev.copy_(host, non_blocking=True)
            gdr.linear_fwd(dev.view_as(xl), out=mid.view_as(xl))
            done = s1.record_event()
        with torch.cuda.stream(s2):
            gdr.layer_norm(small, w, b)
            s2.wait_event(done)
            gdr.layer_norm(mid, w, b, out=out)
            back.copy_(out, non_blocking=True)
        torch.cuda.synchronize()
        assert torch.equal(mid, want.view_as(mid))
        assert torch.equal(out, norm) and torch.equal(back, norm.cpu())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_shared_parameters_and_none(dtype):
    x, w, b, dy = inputs(50, 3, 40, dtype)
    flat = x.view(150, 1, 40)
    dyf = dy.view(150, 1, 40)
    w1, b1 = w[0].contiguous(), b[0].contiguous()
    check_fwd(flat, w1, b1, gdr.layer_norm(x, w1, b1))
    check_fwd(flat, w1, None, gdr.layer_norm(x, w1))
    check_fwd(flat, None, None, gdr.layer_norm(x))
    check_bwd(flat, w1, dyf, gdr.layer_norm_backward(x, w1, dy))
    res = gdr.layer_norm_backward(x, None, dy)
    assert res["dweight"] is None and res["dbias"] is None
    check_bwd(flat, None, dyf, res)
    res = gdr.layer_norm_backward(x, w, dy, need_param_grads=False)
    assert res["dweight"] is None and res["dbias"] is None
    check_bwd(x, w, dy, res)


def test_large_offsets_keep_the_variance():
    """Rows whose mean is a thousand times their spread."""
    x, w, b, dy = inputs(20, 1, 600, "fp32", offset=0.0)
    x = x + 1000.0
    check_fwd(x, w, b, gdr.layer_norm(x, w, b))
    check_bwd(x, w, dy, gdr.layer_norm_backward(x, w, dy))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shape", [(37, 1, 13), (5, 3, 7), (300, 1, 1001),
                                   (3, 2, 64)])
def test_nothing_is_written_beside_the_result(shape, dtype):
    x, w, b, _ = inputs(*shape, dtype)
    n = x.numel()
    wide = torch.full((n + 64,), 7.0, dtype=x.dtype, device="cuda")
    y = gdr.layer_norm(x, w, b, out=wide[32:32 + n].view(x.shape))
    check_fwd(x, w, b, y)
    assert (wide[:32] == 7).all() and (wide[32 + n:] == 7).all()


def test_constant_rows_give_the_bias():
    x = torch.full((4, 96), 3.0, device="cuda")
    w, b = torch.randn(96, device="cuda"), torch.randn(96, device="cuda")
    assert torch.equal(gdr.layer_norm(x, w, b), b.expand(4, 96))
    g = gdr.layer_norm_backward(x, w, torch.randn(4, 96, device="cuda"))
    assert not g["dweight"].any()


def test_not_a_number_stays_in_its_row():
    x, w, b, dy = inputs(64, 4, 128, "bf16")
    clean = gdr.layer_norm(x, w, b)
    gclean = gdr.layer_norm_backward(x, w, dy)["dx"]
    x[7, 1, 3] = float("nan")
    x[9, 2, 5] = float("inf")
    y = gdr.layer_norm(x, w, b)
    dx = gdr.layer_norm_backward(x, w, dy)["dx"]
    keep = torch.ones(64, 4, dtype=torch.bool, device="cuda")
    keep[7, 1] = keep[9, 2] = False
    assert torch.isnan(y[7, 1]).all() and torch.isnan(dx[7, 1]).all()
    assert torch.equal(y[keep], clean[keep])
    assert torch.equal(dx[keep], gclean[keep])


def test_strided_tokens():
    x, w, b, dy = inputs(37, 2, 48, "bf16")
    for width, at in ((96 + 32, 8), (96 + 3, 0)):
        wide = torch.randn(37, width, device="cuda").to(x.dtype)
        wide[:, at:at + 96] = x.view(37, 96)
        xs = wide[:, at:at + 96].unflatten(-1, (2, 48))
        check_fwd(x, w, b, gdr.layer_norm(xs, w, b))
        check_bwd(x, w, dy, gdr.layer_norm_backward(xs, w, dy))
        # one row per head, parameters shared: heads of one token are
        # contiguous, tokens are not, so the rows are not evenly spaced
        with pytest.raises(ValueError):
            gdr.layer_norm(xs, w[0].contiguous())


def test_no_tokens():
    w = torch.ones(2, 24, device="cuda")
    x = torch.empty(0, 2, 24, device="cuda")
    assert gdr.layer_norm(x, w, w).shape == x.shape
    g = gdr.layer_norm_backward(x, w, x)
    torch.cuda.synchronize()
    assert not g["dweight"].any() and not g["dbias"].any()


def test_other_stream_and_captured():
    x, w, b, dy = inputs(900, 4, 128, "bf16")
    run = lambda **k: (gdr.layer_norm(x, w, b, **k),  # noqa: E731
                       gdr.layer_norm_backward(x, w, dy, **k))
    y, g = run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y2, g2 = run(stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y3, g3 = run()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for yy, gg in ((y2, g2), (y3, g3)):
        assert torch.equal(y, yy)
        assert all(torch.equal(g[k], gg[k]) for k in g)


def test_binding_refuses_what_the_kernels_cannot_take():
    x, w, b, dy = inputs(6, 2, 16, "bf16")
    bad = [lambda: gdr.layer_norm(x.cpu(), w, b),
           lambda: gdr.layer_norm(x.half(), w, b),
           lambda: gdr.layer_norm(x, w.bfloat16(), b),
           lambda: gdr.layer_norm(x, w[:1], b),
           lambda: gdr.layer_norm(x, w, b[0]),
           lambda: gdr.layer_norm(x, None, b),
           lambda: gdr.layer_norm(x, w[None], b),
           lambda: gdr.layer_norm(x.transpose(1, 2), None),
           lambda: gdr.layer_norm(x, w, b, out=x.float()),
           lambda: gdr.layer_norm_backward(x, w, dy.float()),
           lambda: gdr.layer_norm_backward(x, w, dy[:3]),
           lambda: gdr.layer_norm_backward(x, w, dy.transpose(1, 2))]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(gdr.GdrError):
        gdr.layer_norm(x, w, b, out=x)
    with pytest.raises(gdr.GdrError):
        gdr.layer_norm(x, w, b, eps=-1.0)
    with pytest.raises(gdr.GdrError):
        gdr.layer_norm(torch.zeros(2, 16385, device="cuda"))


@pytest.mark.parametrize("packed", [False, True])
def test_a_block_of_norm_recurrence_and_head_norm(packed):
    """Norm over the width, linear recurrence, norm per head, and back, with
    every intermediate in fp32: against fp64 end to end.  The parts' own tests
    bound their errors; what is bounded here is their sum, 1e-4 of the
    gradient's largest value (five operators of under 400 u each, amplified
    by rstd <= 4)."""
    g = torch.Generator().manual_seed(5)
    B, T, H, d = (1, 210, 3, 20) if packed else (2, 90, 3, 20)
    cu = [0, 64, 64, 210] if packed else None
    n = 3 if packed else B
    x = torch.randn(B, T, H * d, generator=g)
    w1, b1 = torch.rand(H * d, generator=g) + 0.5, torch.randn(H * d,
                                                               generator=g)
    w2, b2 = torch.rand(H, d, generator=g) + 0.5, torch.randn(H, d,
                                                              generator=g)
    la = -torch.rand(B, T, H, d, generator=g) * 0.5
    s0 = torch.randn(n, H, d, generator=g)
    dy = torch.randn(B, T, H, d, generator=g)
    c = lambda t: t.cuda()  # noqa: E731
    cut = None if cu is None else torch.tensor(cu, dtype=torch.int32,
                                               device="cuda")
    y1 = gdr.layer_norm(c(x), c(w1), c(b1))
    h, fin, cs = gdr.linear_fwd(y1.unflatten(-1, (H, d)), c(la), c(s0),
                                cu_seqlens=cut, output_chunk_states=True)
    y2 = gdr.layer_norm(h, c(w2), c(b2))
    g2 = gdr.layer_norm_backward(h, c(w2), c(dy))
    gl = gdr.linear_backward(y1.unflatten(-1, (H, d)), c(la), c(s0), g2["dx"],
                             chunk_states=cs, cu_seqlens=cut)
    g1 = gdr.layer_norm_backward(c(x), c(w1), gl["dx"].flatten(2))
    torch.cuda.synchronize()
    n64 = lambda t: t.double().numpy()  # noqa: E731
    r1 = oracle.layer_norm(n64(x)[:, :, None], n64(w1), n64(b1), 1e-5)
    rh, rf, _ = oracle.linear_fwd(r1.reshape(B, T, H, d), n64(la), n64(s0),
                                  cu)
    r2 = oracle.layer_norm(rh, n64(w2), n64(b2), 1e-5)
    flat = lambda a, *s: a.reshape(B * T, *s)  # noqa: E731
    rg2 = oracle.layer_norm_grads(flat(rh, H, d), n64(w2),
                                  flat(n64(dy), H, d), 1e-5)
    rgl = oracle.linear_grads(r1.reshape(B, T, H, d), n64(la), n64(s0),
                              rg2["dx"].reshape(B, T, H, d), None, cu)
    rg1 = oracle.layer_norm_grads(flat(n64(x), 1, H * d), n64(w1)[None],
                                  flat(rgl["dx"], 1, H * d), 1e-5)
    pairs = [(y2, r2), (fin, rf), (g2["dweight"], rg2["dweight"]),
             (g2["dbias"], rg2["dbias"]), (gl["dlog_alpha"],
                                           rgl["dlog_alpha"]),
             (gl["dinitial_state"], rgl["dinitial_state"]),
             (g1["dx"], rg1["dx"]), (g1["dweight"], rg1["dweight"]),
             (g1["dbias"], rg1["dbias"])]
    for i, (a, b) in enumerate(pairs):
        a = f64(a).reshape(b.shape)
        assert np.abs(a - b).max() <= 1e-4 * np.abs(b).max(), i


@pytest.mark.parametrize("d", [2048, 2047])
def test_more_values_than_32_bits_can_count(d):
    """The last rows of 2^31 values and more against the same rows on their
    own."""
    n, last = (2 ** 31 + 2 ** 23) // d, 300
    x = torch.zeros(n, d, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    x[-last:] = torch.randn(last, d, generator=g, device="cuda").to(x)
    w, b = (torch.randn(d, generator=g, device="cuda") for _ in range(2))
    tail = x[-last:].clone()
    y = gdr.layer_norm(x, w, b)
    check_fwd(tail.unsqueeze(1), w.unsqueeze(0), b.unsqueeze(0),
              y[-last:].unsqueeze(1))
    del y
    # (rows of zeros have no distances, and a gradient of zeros)
    res = gdr.layer_norm_backward(x, w, x)
    torch.cuda.synchronize()
    check_bwd(tail.unsqueeze(1), w.unsqueeze(0), tail.unsqueeze(1),
              dict(dx=res["dx"][-last:].unsqueeze(1), dweight=res["dweight"],
                   dbias=res["dbias"]))
    del x, res
    torch.cuda.empty_cache()


# eps = 0, token counts that do not fill a block's last round: sums written
# per cluster, per group and per block, and heads that share a block
NO_EPS = [(1, 1, 8), (1, 1, 64), (5, 1, 77), (37, 1, 128), (1, 1, 2048),
          (7, 1, 2048), (333, 1, 1001), (701, 1, 2048), (2501, 1, 77),
          (1501, 5, 101), (41, 3, 40)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shape", NO_EPS)
def test_gradients_without_eps(shape, dtype):
    """(No row of these inputs is constant, so every one has an answer.)"""
    x, w, b, dy = inputs(*shape, dtype, seed=7)
    check_fwd(x, w, b, gdr.layer_norm(x, w, b, eps=0.0), eps=0.0)
    check_bwd(x, w, dy, gdr.layer_norm_backward(x, w, dy, eps=0.0), eps=0.0)
    n, H, d = shape
    wide = torch.full((n, H * d + 24), 5.0, dtype=x.dtype, device="cuda")
    wide[:, 8:8 + H * d] = x.view(n, H * d)
    xs = wide[:, 8:8 + H * d].unflatten(-1, (H, d))
    if xs.data_ptr() % 16 == 0:
        check_bwd(x, w, dy, gdr.layer_norm_backward(xs, w, dy, eps=0.0),
                  eps=0.0)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shape", [(10, 1, 1), (9, 1, 3), (5, 2, 2),
                                   (13, 3, 1), (700, 1, 5), (41, 2, 3)])
def test_tokens_narrower_than_a_vector(shape, dtype):
    """Several tokens to a 16-byte vector; the last ones' vectors end with the
    tensor."""
    x, w, b, dy = inputs(*shape, dtype, seed=8)
    check_fwd(x, w, b, gdr.layer_norm(x, w, b))
    check_bwd(x, w, dy, gdr.layer_norm_backward(x, w, dy))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("d", [3, 37, 77, 640, 1000, 1001, 2047, 2048, 3030,
                               5120, 12000, 16384])
def test_constant_rows_have_no_distances(d, dtype):
    """Values of 8 bits, so that a row's sum is exact: of every size the
    rows' answer is the bias, and the weight gets no gradient."""
    v = torch.arange(128, 256, dtype=torch.float32)
    v = torch.cat([v, -v / 128, v * 256, v / 2 ** 20]).to(DT[dtype]).cuda()
    x = v[:, None].expand(-1, d).contiguous()
    w, b = torch.randn(d, device="cuda"), torch.randn(d, device="cuda")
    y = gdr.layer_norm(x, w, b)
    assert torch.equal(y, b.to(x.dtype).expand(len(v), d))
    g = gdr.layer_norm_backward(x, w, torch.randn_like(x))
    assert not g["dweight"].any()
    assert torch.isfinite(g["dx"]).all()

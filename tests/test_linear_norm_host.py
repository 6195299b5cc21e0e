"""Linear recurrence and layer normalisation without a GPU: the fp64
references are pinned by closed forms and central differences, and the C ABI
rejects bad arguments on the host before any CUDA call."""
import ctypes
import os
import subprocess
import sys
import threading

import numpy as np
import pytest

import chunkwise_recurrence_b200 as gdr
import oracle
from chunkwise_recurrence_b200 import build as gdr_build

OK, INVALID, UNSUPPORTED, CUDA, OOM = range(5)
A = 0x10000       # 16-byte-aligned fake device addresses, far apart and never
STEP = 1 << 40    # dereferenced


@pytest.fixture(scope="module")
def lib():
    gdr_build.build()
    return gdr.load_library()


def _rng(seed):
    return np.random.default_rng(seed)


# -------------------------------------------------------------- references

def test_linear_prefix_sum_and_geometric_series():
    x = _rng(0).normal(size=(2, 9, 2, 3))
    out, fin, _ = oracle.linear_fwd(x)
    assert np.allclose(out, np.cumsum(x, 1)) and np.allclose(fin, x.sum(1))
    la = np.full((1, 40, 1), np.log(0.5))
    out, _, _ = oracle.linear_fwd(np.ones((1, 40, 1, 2)), la)
    t = np.arange(1, 41)
    assert np.allclose(out[0, :, 0, 0], 2 * (1 - 0.5 ** t))


def test_linear_split_and_packed_equal_one_call():
    r = _rng(1)
    x, la = r.normal(size=(1, 20, 2, 3)), -r.random((1, 20, 2, 3))
    s0 = r.normal(size=(1, 2, 3))
    out, fin, _ = oracle.linear_fwd(x, la, s0)
    o1, f1, _ = oracle.linear_fwd(x[:, :7], la[:, :7], s0)
    o2, f2, _ = oracle.linear_fwd(x[:, 7:], la[:, 7:], f1)
    assert np.allclose(np.concatenate([o1, o2], 1), out)
    assert np.allclose(f2, fin)
    s = r.normal(size=(3, 2, 3))
    cu = [0, 5, 5, 20]
    po, pf, _ = oracle.linear_fwd(x, la, s, cu)
    for n in range(3):
        o, f, _ = oracle.linear_fwd(x[:, cu[n]:cu[n + 1]],
                                    la[:, cu[n]:cu[n + 1]], s[n:n + 1])
        assert np.allclose(po[:, cu[n]:cu[n + 1]], o)
        assert np.allclose(pf[n:n + 1], f)


@pytest.mark.parametrize("gate", ["none", "scalar", "channel"])
def test_linear_gradients_are_the_differences(gate):
    r = _rng(2)
    cu = [0, 4, 4, 9]
    x, s0 = r.normal(size=(1, 9, 2, 3)), r.normal(size=(3, 2, 3))
    la = {"none": None, "scalar": -r.random((1, 9, 2)),
          "channel": -r.random((1, 9, 2, 3))}[gate]
    dO, dS = r.normal(size=x.shape), r.normal(size=s0.shape)

    def loss(x, la, s0):
        o, f, _ = oracle.linear_fwd(x, la, s0, cu)
        return (o * dO).sum() + (f * dS).sum()

    got = oracle.linear_grads(x, la, s0, dO, dS, cu)
    for key, i in (("dx", 0), ("dlog_alpha", 1), ("dinitial_state", 2)):
        args = [x, la, s0]
        if args[i] is None:
            assert got[key] is None
            continue
        num = np.zeros_like(args[i])
        for j in np.ndindex(args[i].shape):
            for sg in (1, -1):
                a = args[i].copy()
                a[j] += sg * 1e-6
                num[j] += sg * loss(*(args[:i] + [a] + args[i + 1:])) / 2e-6
        assert np.allclose(got[key], num, rtol=1e-6, atol=1e-7), key


def test_norm_output_moments_and_gradients():
    r = _rng(3)
    x = r.normal(size=(4, 2, 7)) * 3 + 5
    y = oracle.layer_norm(x, None, None, 0.0)
    assert np.allclose(y.mean(-1), 0) and np.allclose((y * y).mean(-1), 1)
    w, b = r.normal(size=(2, 7)), r.normal(size=(2, 7))
    dO = r.normal(size=x.shape)
    got = oracle.layer_norm_grads(x, w, dO, 1e-3)
    for key, i in (("dx", 0), ("dweight", 1), ("dbias", 2)):
        args = [x, w, b]
        num = np.zeros_like(args[i])
        for j in np.ndindex(args[i].shape):
            for sg in (1, -1):
                a = args[i].copy()
                a[j] += sg * 1e-6
                full = args[:i] + [a] + args[i + 1:]
                num[j] += sg * (oracle.layer_norm(*full, 1e-3) * dO).sum() \
                    / 2e-6
        assert np.allclose(got[key], num, rtol=1e-6, atol=1e-6), key


# ---------------------------------------------------------------- refusals

def _opts(a):
    return gdr._Opts(a["dtype"], a["gate"], a["cu"], a["nseq"], a["algo"])


def _fwd(lib, **kw):
    a = dict(x=A, ldx=128, la=A + STEP, s0=None, out=A + 2 * STEP,
             sT=A + 3 * STEP, cs=None, B=2, T=64, H=2, d=64, dtype=0, gate=1,
             cu=None, nseq=0, algo=0)
    a.update(kw)
    return lib.gdr_linear_fwd(a["x"], a["ldx"], a["la"], a["s0"], a["out"],
                              a["sT"], a["cs"], a["B"], a["T"], a["H"],
                              a["d"], None, ctypes.byref(_opts(a)))


def _bwd(lib, **kw):
    a = dict(x=A, ldx=128, la=A + STEP, s0=None, cs=None, dO=A + 2 * STEP,
             dS=None, dx=A + 3 * STEP, dla=A + 4 * STEP, ds0=None, B=2, T=64,
             H=2, d=64, dtype=0, gate=1, cu=None, nseq=0, algo=0)
    a.update(kw)
    return lib.gdr_linear_backward(
        a["x"], a["ldx"], a["la"], a["s0"], a["cs"], a["dO"], a["dS"],
        a["dx"], a["dla"], a["ds0"], a["B"], a["T"], a["H"], a["d"], None,
        ctypes.byref(_opts(a)))


def _step(lib, **kw):
    a = dict(x=A, ldx=128, la=A + STEP, sin=A + 2 * STEP, sout=A + 3 * STEP,
             out=A + 4 * STEP, N=4, H=2, d=64, dtype=0, gate=1, cu=None,
             nseq=0, algo=0)
    a.update(kw)
    return lib.gdr_linear_step(a["x"], a["ldx"], a["la"], a["sin"],
                               a["sout"], a["out"], a["N"], a["H"], a["d"],
                               None, ctypes.byref(_opts(a)))


@pytest.mark.parametrize("call", [_fwd, _bwd, _step])
def test_linear_entries_reject_bad_arguments(lib, call):
    c = lambda **kw: call(lib, **kw)  # noqa: E731
    assert c(x=None) == INVALID
    assert c(x=A + 8) == INVALID                   # misaligned
    assert c(la=A + STEP + 4) == INVALID
    assert c(la=None) == INVALID                   # a gate needs its decays
    assert c(gate=0) == INVALID                    # ... and no gate none
    assert c(gate=3) == INVALID
    assert c(dtype=2) == INVALID
    assert c(ldx=127) == INVALID                   # tokens would overlap
    assert c(H=-1) == INVALID
    assert c(d=0) == INVALID
    assert c(algo=9) == INVALID
    assert c(algo=1) == UNSUPPORTED
    assert c(H=70000, ldx=1 << 30) == UNSUPPORTED
    assert c(H=65535, d=65535, ldx=1 << 40) == UNSUPPORTED   # H d > 2^24
    assert c(nseq=3) == INVALID                    # num_seqs without offsets


def test_linear_fwd_rejects_bad_buffers(lib):
    c = lambda **kw: _fwd(lib, **kw)  # noqa: E731
    assert c(out=None) == INVALID
    assert c(T=-1) == INVALID
    assert c(cu=A, nseq=1) == INVALID              # packed needs B = 1
    assert c(B=1, cu=A, nseq=-1) == INVALID
    assert c(B=1, cu=A + 2, nseq=1) == INVALID
    assert c(B=1 << 20, T=1 << 12) == UNSUPPORTED  # too many tokens
    assert c(out=A) == INVALID                     # written over its input
    assert c(out=A + 2 * 64 * 128 * 2 - 16) == INVALID
    assert c(out=A + STEP) == INVALID
    assert c(sT=A + 2 * STEP) == INVALID
    assert c(cs=A + 2 * STEP + 16) == INVALID
    assert c(s0=A + 3 * STEP) == INVALID
    assert c(B=1 << 24, T=1, H=16, d=64, ldx=1024) == UNSUPPORTED  # chains
    empty = dict(x=None, la=None, out=None, sT=None, gate=0)
    assert c(B=0, **empty) == OK
    assert c(H=0, **empty) == OK
    assert c(B=1, cu=A, nseq=0, **empty) == OK


def test_linear_backward_rejects_bad_buffers(lib, monkeypatch):
    c = lambda **kw: _bwd(lib, **kw)  # noqa: E731
    assert c(dO=None) == INVALID
    assert c(dx=None) == INVALID
    assert c(dla=None) == INVALID
    assert c(gate=0, la=None) == INVALID           # d_log_alpha without a gate
    assert c(dx=A) == INVALID
    assert c(dx=A + 2 * STEP) == INVALID
    assert c(dla=A + STEP) == INVALID
    assert c(ds0=A + 8) == INVALID
    assert c(cs=A + 4) == INVALID
    assert c(dS=A + 3 * STEP) == INVALID
    assert c(x=None, la=None, dO=None, dx=None, dla=None, gate=0, B=0) == OK
    # the chunk states that were not given need scratch
    monkeypatch.setenv("GDR_FAULT_INJECT_ALLOC", "1")
    assert c() == OOM


def test_linear_step_rejects_bad_buffers(lib):
    c = lambda **kw: _step(lib, **kw)  # noqa: E731
    assert c(out=None) == INVALID
    assert c(sout=None) == INVALID
    assert c(N=-1) == INVALID
    assert c(cu=A, nseq=4) == INVALID
    assert c(sout=A + 2 * STEP + 64) == INVALID    # neither in place nor apart
    assert c(sout=A + 4 * STEP) == INVALID
    assert c(x=None, la=None, sin=None, sout=None, out=None, gate=0,
             N=0) == OK


def _norm(lib, **kw):
    a = dict(x=A, ldx=128, w=A + STEP, b=A + 2 * STEP, out=A + 3 * STEP,
             n=8, H=2, d=64, eps=1e-5, dtype=0)
    a.update(kw)
    return lib.gdr_layer_norm(a["x"], a["ldx"], a["w"], a["b"], a["out"],
                              a["n"], a["H"], a["d"], a["eps"], a["dtype"],
                              None)


def _norm_bwd(lib, **kw):
    a = dict(x=A, ldx=128, w=A + STEP, dO=A + 2 * STEP, out=A + 3 * STEP,
             dw=A + 4 * STEP, db=A + 5 * STEP, n=8, H=2, d=64, eps=1e-5,
             dtype=0)
    a.update(kw)
    return lib.gdr_layer_norm_backward(
        a["x"], a["ldx"], a["w"], a["dO"], a["out"], a["dw"], a["db"], a["n"],
        a["H"], a["d"], a["eps"], a["dtype"], None)


@pytest.mark.parametrize("call", [_norm, _norm_bwd])
def test_norm_entries_reject_bad_arguments(lib, call):
    c = lambda **kw: call(lib, **kw)  # noqa: E731
    assert c(x=None) == INVALID
    assert c(out=None) == INVALID
    assert c(x=A + 2) == INVALID
    assert c(w=A + STEP + 4) == INVALID
    assert c(n=-1) == INVALID
    assert c(H=-1) == INVALID
    assert c(d=0) == INVALID
    assert c(ldx=127) == INVALID
    assert c(dtype=3) == INVALID
    assert c(eps=-1e-5) == INVALID
    assert c(eps=float("nan")) == INVALID
    assert c(d=16385, ldx=1 << 20) == UNSUPPORTED
    assert c(H=65536, ldx=1 << 30) == UNSUPPORTED
    assert c(n=1 << 29, H=8, d=16) == UNSUPPORTED  # rows
    assert c(out=A + 16) == INVALID                # overlaps
    assert c(out=A + STEP) == INVALID
    assert c(H=0, x=None, out=None, w=None) == OK


def test_norm_backward_rejects_bad_buffers(lib, monkeypatch):
    c = lambda **kw: _norm_bwd(lib, **kw)  # noqa: E731
    assert c(dO=None) == INVALID
    assert c(dw=A + 5 * STEP) == INVALID
    assert c(db=A + 2 * STEP) == INVALID
    assert c(db=A + 5 * STEP + 8) == INVALID
    assert _norm(lib, n=0, x=None, out=None) == OK
    # (few tokens need no scratch)
    monkeypatch.setenv("GDR_FAULT_INJECT_ALLOC", "1")
    assert c(n=1 << 20) == OOM


# ------------------------------------------------------- reads of norm rows

_ROWS = r"""
#include <cstdio>
#include "norm_rows.h"
// every row of [ntok][H][d] by 16-byte vectors: nothing outside the tensor is
// read, and every element of the row is
int main() {
  using namespace gdr::rows;
  for (int es = 2; es <= 4; es += 2)
    for (int ntok = 1; ntok <= 20; ++ntok)
      for (int H = 1; H <= 4; ++H)
        for (int d = 1; d <= 20; ++d) {
          const int V = 16 / es;
          const long long all = (long long)ntok * H * d;
          for (int tok = 0; tok < ntok; ++tok)
            for (int h = 0; h < H; ++h) {
              const long long at = ((long long)tok * H + h) * d;
              const int s = shift(at, V), n = vectors(s, d, V);
              long long covered = at - s;
              for (int i = 0; i < n; ++i) {
                const long long from = at - s + i * V;
                const int b = may_end(tok, ntok, V)
                                  ? vector_bytes(all - from, V, es) : 16;
                if (from < 0 || from % V || b <= 0 ||
                    from * es + b > all * es) {
                  std::printf("es %d ntok %d H %d d %d tok %d h %d: %lld + %d "
                              "of %lld bytes", es, ntok, H, d, tok, h,
                              from * es, b, all * es);
                  return 1;
                }
                covered = from + b / es;
              }
              if (covered < at + d) return 2;
            }
        }
}
"""


def test_norm_rows_are_read_within_their_tensor(tmp_path):
    src, exe = tmp_path / "rows.cpp", tmp_path / "rows"
    src.write_text(_ROWS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", gdr_build.CSRC,
                    str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


# --------------------------------------------- loads of overlapping launches

def test_kernels_that_start_early_do_not_use_the_read_only_path():
    """A kernel that may start while the one before it still writes must read
    what that one wrote by ordinary loads: the wait for it does not order
    those of the read-only path."""
    early = []
    for path in gdr_build.sources():
        with open(path) as f:
            text = f.read()
        if "prior_done" in text:
            early.append(os.path.basename(path))
            assert "__ldg" not in text and "ld.global.nc" not in text, path
            assert "__restrict__" not in text, path
    assert early == ["linear.cu", "norm.cu"]


# -------------------------------------------------------------- size limits

def test_size_limits_are_the_documented_ones(lib):
    """The largest size of each kind is taken (a misaligned pointer stops the
    call there, before any CUDA call), the next is not."""
    with open(os.path.join(gdr_build.INCLUDE, "gdr.h")) as f:
        text = " ".join(f.read().replace("\n *", " ").split())
    for stated in ("B T < 2^30 (packed: T < 2^30), ldx < 2^30",
                   "H <= 65535, H d <= 2^24",
                   "H <= 65535, ntok < 2^30, ntok H < 2^31"):
        assert stated in text
    top = 1 << 30
    one = dict(B=1, H=1, d=1, ldx=1, x=A + 8)
    for call in (_fwd, _bwd):
        assert call(lib, **one, T=top - 1) == INVALID
        assert call(lib, **one, T=top) == UNSUPPORTED
        assert call(lib, **one, T=top - 1, cu=A, nseq=1) == INVALID
        assert call(lib, **one, T=top, cu=A, nseq=1) == UNSUPPORTED
        wide = dict(B=1, T=1, x=A + 8)
        assert call(lib, **wide, ldx=top - 1) == INVALID
        assert call(lib, **wide, ldx=top) == UNSUPPORTED
        assert call(lib, **wide, H=1, d=1 << 24, ldx=1 << 24) == INVALID
        assert call(lib, **wide, H=1, d=(1 << 24) + 1,
                    ldx=1 << 25) == UNSUPPORTED
        assert call(lib, **wide, H=65535, d=1, ldx=65535) == INVALID
        assert call(lib, **wide, H=65536, d=1, ldx=65536) == UNSUPPORTED
    small = dict(H=1, d=1, ldx=1, x=A + 8)
    assert _step(lib, **small, N=top - 1) == INVALID
    assert _step(lib, **small, N=top) == UNSUPPORTED
    for call in (_norm, _norm_bwd):
        assert call(lib, **small, n=top - 1) == INVALID
        assert call(lib, **small, n=top) == UNSUPPORTED
        two = dict(H=3, d=1, ldx=3, x=A + 8)
        assert call(lib, **two, n=((1 << 31) - 1) // 3) == INVALID
        assert call(lib, **two, n=((1 << 31) - 1) // 3 + 1) == UNSUPPORTED
        assert call(lib, H=1, d=16384, ldx=16384, x=A + 8) == INVALID
        assert call(lib, H=65535, d=1, ldx=65535, x=A + 8) == INVALID


# -------------------------------------------------------------------- build

def _in_another_python(code):
    root = os.path.dirname(gdr_build.PKG)
    return subprocess.run([sys.executable, "-c", code], cwd=root,
                          capture_output=True, text=True)


@pytest.mark.parametrize("missing", ["torch", "headers", "g++"])
def test_the_library_builds_without_the_binding(lib, missing):
    """A fresh libgdr.so: build() leaves it and does without the binding."""
    r = _in_another_python(f"""
import importlib.util, sys
missing = {missing!r}
if missing == "torch":
    sys.modules["torch"] = None
spec = importlib.util.spec_from_file_location("b", {gdr_build.__file__!r})
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
if missing == "headers":
    exists = b.os.path.exists
    b.os.path.exists = lambda p: not str(p).endswith("variable.h") and exists(p)
if missing == "g++":
    which = b.shutil.which
    b.shutil.which = lambda n: None if n == "g++" else which(n)
b._stale = lambda: False
assert b.build() == b.LIB
try:
    b.build_binding()
except RuntimeError as e:
    assert "cannot be built" in str(e)
else:
    raise SystemExit("the binding was built")
""")
    assert r.returncode == 0, r.stderr
    assert "without its PyTorch binding" in r.stderr


def test_the_binding_belongs_to_one_torch_and_one_python(lib, monkeypatch):
    import sysconfig

    import torch
    assert gdr.BINDING_PATH == gdr_build.binding_path()
    assert os.path.exists(gdr.BINDING_PATH)
    assert not gdr_build._binding_stale()
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    assert gdr_build.binding_path() != gdr.BINDING_PATH
    assert gdr_build._binding_stale()
    monkeypatch.undo()
    monkeypatch.setattr(sysconfig, "get_config_var", lambda n: "cpython-0")
    assert gdr_build.binding_path() != gdr.BINDING_PATH
    assert gdr_build._binding_stale()


def test_a_missing_binding_is_an_error(lib, monkeypatch):
    import torch
    monkeypatch.setattr(gdr, "_native", None)
    monkeypatch.setattr(gdr, "BINDING_PATH", gdr.BINDING_PATH + ".none")
    with pytest.raises(RuntimeError, match="is missing"):
        gdr.layer_norm(torch.zeros(2, 8))


def test_sources_are_compiled_side_by_side(monkeypatch, tmp_path):
    """Nothing is compiled: the compiler is replaced by one that waits until
    two of it run at once, and notes what it was asked to do."""
    meet = threading.Barrier(2)
    asked, met = [], []

    def run(cmd, check):
        assert check
        asked.append(cmd)
        if "-c" in cmd:
            try:
                meet.wait(timeout=10)
                met.append(cmd)
            except threading.BrokenBarrierError:
                pass
        else:
            open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(gdr_build.subprocess, "run", run)
    monkeypatch.setattr(gdr_build.os, "cpu_count", lambda: 2)
    monkeypatch.setattr(gdr_build, "ROOT", str(tmp_path))
    monkeypatch.setattr(gdr_build, "LIB", str(tmp_path / "libgdr.so"))
    monkeypatch.setattr(gdr_build, "_nvcc", lambda: "nvcc")
    monkeypatch.setattr(gdr_build, "_build_binding_if_possible",
                        lambda force: None)
    assert gdr_build.build(force=True) == str(tmp_path / "libgdr.so")
    assert met
    compiled = [c[c.index("-c") + 1] for c in asked if "-c" in c]
    assert sorted(compiled) == gdr_build.sources()
    objects = [a for a in asked[-1] if a.endswith(".o")]
    assert [os.path.basename(o)[:-2] for o in objects] == \
        [os.path.basename(s) for s in gdr_build.sources()]


def test_a_fresh_library_needs_no_compiler(lib, monkeypatch, capsys):
    """Neither for itself nor for a binding that belongs to another torch."""
    import torch

    def none():
        raise RuntimeError("nvcc not found")

    monkeypatch.setattr(gdr_build, "_stale", lambda: False)
    monkeypatch.setattr(gdr_build, "_nvcc", none)
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    assert gdr_build.build() == gdr_build.LIB
    assert "nvcc not found" in capsys.readouterr().err

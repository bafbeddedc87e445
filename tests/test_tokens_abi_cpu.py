"""Contract of the token path's C entry points that needs no GPU: exported symbols, and refusals before any HIP call
(fake, never-dereferenced pointers)."""
import ctypes
import subprocess

import pytest

from scan_linear_rnns_amd import _lib
from scan_linear_rnns_amd._lib import GatedDesc, SampleDesc
from tests.test_abi_cpu import INVALID, OK, UNSUPPORTED, WORKSPACE, fake

NAN, INF = float("nan"), float("inf")
BIG = 1 << 31


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def test_exports_every_declared_symbol(lib):
    declared = _lib.declared_functions(_lib.TOKENS_HEADER)
    assert len(declared) == 9, declared
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    for name in declared:
        assert name in exported and name in _lib.SIGNATURES, name


# -------------------------------------------------------------- embedding

def embed_size(lib, n=100, vocab=50, d=64):
    out = ctypes.c_size_t(0)
    return lib.mgs_embed_workspace_size(n, vocab, d, ctypes.byref(out)), out.value


def test_embed_workspace(lib):
    st, small = embed_size(lib)
    assert st == OK and small >= 256 and embed_size(lib, n=10000)[1] > small
    assert lib.mgs_embed_workspace_size(1, 1, 1, None) == INVALID
    for bad in (dict(n=-1), dict(vocab=-1), dict(d=0), dict(d=-8)):
        assert embed_size(lib, **bad)[0] == INVALID, bad
    for bad in (dict(n=BIG), dict(vocab=BIG), dict(d=BIG), dict(n=1 << 30, d=1 << 20), dict(vocab=1 << 30, d=1 << 20)):
        assert embed_size(lib, **bad)[0] == UNSUPPORTED, bad
    assert embed_size(lib, n=0)[0] == OK and embed_size(lib, vocab=0)[0] == OK


def test_an_embed_workspace_serves_fewer_ids(lib):
    for d in (1, 64, 2050):
        sizes = [embed_size(lib, n=n, vocab=700, d=d)[1] for n in range(0, 40000, 13)]
        assert sizes == sorted(sizes), d


def test_embed_fwd_refusals(lib):
    def fwd(ids=fake(0), bits=64, W=fake(1), y=fake(2), n=100, vocab=50, d=64, stride=64, dtype=1):
        return lib.mgs_embed_fwd(ids, bits, W, y, n, vocab, d, stride, 1.0, dtype, None)

    for name in ("ids", "W", "y"):
        assert fwd(**{name: None}) == INVALID, name
    assert fwd(y=fake(1)) == INVALID and fwd(y=fake(0, 16)) == INVALID     # over the table, over the ids
    assert fwd(W=fake(1, 1)) == INVALID and fwd(y=fake(2, 2), dtype=0) == INVALID and fwd(ids=fake(0, 4)) == INVALID
    assert fwd(stride=-64) == INVALID and fwd(stride=1 << 60) == INVALID
    assert fwd(n=-1) == INVALID and fwd(vocab=-1) == INVALID and fwd(d=0) == INVALID
    assert fwd(bits=16) == UNSUPPORTED and fwd(dtype=2) == UNSUPPORTED and fwd(n=BIG) == UNSUPPORTED
    assert fwd(n=0, ids=None, y=None) == OK


def test_embed_bwd_refusals(lib):
    def bwd(ids=fake(0), bits=32, dy=fake(1), dW=fake(2), n=100, vocab=50, d=64, stride=64, add=0, dtype=1, out=0,
            ws=fake(9), nbytes=1 << 30):
        return lib.mgs_embed_bwd(ids, bits, dy, dW, n, vocab, d, stride, 1.0, add, dtype, out, ws, nbytes, None)

    for name in ("ids", "dy", "dW"):
        assert bwd(**{name: None}) == INVALID, name
    assert bwd(dW=fake(1)) == INVALID and bwd(dW=fake(0)) == INVALID
    assert bwd(dW=fake(2, 2)) == INVALID and bwd(dy=fake(1, 1)) == INVALID and bwd(stride=-1) == INVALID
    assert bwd(dtype=3) == UNSUPPORTED and bwd(out=-1) == UNSUPPORTED and bwd(bits=8) == UNSUPPORTED
    assert bwd(ws=None) == WORKSPACE and bwd(nbytes=255) == WORKSPACE and bwd(ws=fake(9, 8)) == INVALID
    assert bwd(vocab=0, dW=None, ws=None) == OK and bwd(n=0, ids=None, dy=None, add=1, ws=None) == OK


# ------------------------------------------------- gated linear recurrence

def gated(B=2, T=300, D=200, dtype=0, rate=8.0, **strides):
    st = dict(x=(T * D, D), r=(T * D, D), i=(T * D, D), dy=(T * D, D))
    st.update(strides)
    return GatedDesc(B, T, D, dtype, rate, st["x"], st["r"], st["i"], st["dy"])


def gated_size(lib, d, backward=0):
    out = ctypes.c_size_t(0)
    return lib.mgs_gated_workspace_size(ctypes.byref(d), backward, ctypes.byref(out)), out.value


def test_gated_workspace(lib):
    st, fwd = gated_size(lib, gated())
    st2, both = gated_size(lib, gated(), 1)
    assert st == OK and st2 == OK and both >= fwd >= 256
    assert lib.mgs_gated_workspace_size(None, 0, ctypes.byref(ctypes.c_size_t())) == INVALID
    assert lib.mgs_gated_workspace_size(ctypes.byref(gated()), 0, None) == INVALID
    for bad in (dict(B=-1), dict(T=-1), dict(D=0), dict(rate=-1.0), dict(rate=NAN), dict(rate=INF)):
        assert gated_size(lib, gated(**bad))[0] == INVALID, bad
    for bad in (dict(dtype=2), dict(B=BIG), dict(T=BIG), dict(D=BIG), dict(B=1 << 20, T=1 << 20, D=2),
                dict(B=1 << 30, T=0, D=1 << 20), dict(B=1 << 23, T=1, D=1), dict(T=1 << 30, D=128)):
        for backward in (0, 1):
            assert gated_size(lib, gated(**bad), backward)[0] == UNSUPPORTED, bad
    assert gated_size(lib, gated(B=0))[0] == OK and gated_size(lib, gated(T=0), 1)[0] == OK
    # a workspace of the forward and backward of a size is one of either alone
    for T in (1, 64, 65, 128, 129, 1000, 5000):
        assert gated_size(lib, gated(T=T), 1)[1] >= gated_size(lib, gated(T=T))[1]


@pytest.mark.parametrize("backward", [0, 1])
def test_a_gated_workspace_serves_fewer_sequences_and_steps(lib, backward):
    for D in (1, 128, 300, 1024, 5000):
        for T in (64, 65, 129, 1000, 40000):
            sizes = [gated_size(lib, gated(B=B, T=T, D=D), backward)[1] for B in range(100)]
            assert sizes == sorted(sizes), (D, T)
        for B in (1, 3, 40):
            sizes = [gated_size(lib, gated(B=B, T=T, D=D), backward)[1] for T in range(0, 3000, 7)]
            assert sizes == sorted(sizes), (D, B)


def test_gated_fwd_refusals(lib):
    good = dict(x=fake(0), r=fake(1), i=fake(2), lam=fake(3), h0=None, lengths=None, reset=None, y=fake(4), hT=fake(5),
                states=fake(6))

    def fwd(d=None, ws=fake(9), nbytes=1 << 30, **change):
        a = {**good, **change}
        return lib.mgs_gated_fwd(ctypes.byref(d or gated()), *a.values(), ws, nbytes, None)

    assert lib.mgs_gated_fwd(None, *good.values(), fake(9), 1 << 30, None) == INVALID
    for name in ("x", "r", "i", "lam", "y"):
        assert fwd(**{name: None}) == INVALID, name
    assert fwd(y=fake(0)) == INVALID                                        # over an input
    assert fwd(hT=fake(4, 64)) == INVALID and fwd(states=fake(5)) == INVALID  # over another output
    assert fwd(h0=fake(5)) == INVALID                                       # the state in place
    assert fwd(reset=fake(4, 1)) == INVALID and fwd(y=fake(3)) == INVALID
    assert fwd(x=fake(0, 2)) == INVALID and fwd(lam=fake(3, 1)) == INVALID and fwd(lengths=fake(7, 2)) == INVALID
    assert fwd(d=gated(x=(-1, 200))) == INVALID and fwd(d=gated(i=(1 << 60, 1 << 60))) == INVALID
    assert fwd(d=gated(dtype=7)) == UNSUPPORTED and fwd(d=gated(rate=NAN)) == INVALID
    assert fwd(ws=None) == WORKSPACE and fwd(nbytes=255) == WORKSPACE and fwd(ws=fake(9, 8)) == INVALID
    none = dict(x=None, r=None, i=None, y=None, hT=None, states=None, ws=None)
    assert fwd(d=gated(B=0), **none) == OK and fwd(d=gated(T=0), **none) == OK


def test_gated_bwd_refusals(lib):
    good = dict(x=fake(0), r=fake(1), i=fake(2), lam=fake(3), dy=fake(4), dhT=None, states=fake(5), lengths=None,
                reset=None, dx=fake(6), dr=fake(7), di=fake(8), dlam=fake(9), dh0=fake(10))

    def bwd(d=None, ws=fake(12), nbytes=1 << 30, **change):
        a = {**good, **change}
        return lib.mgs_gated_bwd(ctypes.byref(d or gated()), *a.values(), ws, nbytes, None)

    assert lib.mgs_gated_bwd(None, *good.values(), fake(12), 1 << 30, None) == INVALID
    for name in ("x", "r", "i", "lam", "dy", "states", "dx", "dr", "di", "dlam"):
        assert bwd(**{name: None}) == INVALID, name
    for name, over in (("dx", 0), ("dr", 6), ("di", 4), ("dlam", 3), ("dh0", 5), ("dh0", 9)):
        assert bwd(**{name: fake(over)}) == INVALID, (name, over)
    assert bwd(dh0=fake(11), dhT=fake(11)) == INVALID
    assert bwd(dx=fake(6, 2)) == INVALID and bwd(dlam=fake(9, 2)) == INVALID and bwd(dhT=fake(11, 1)) == INVALID
    assert bwd(d=gated(dy=(5, -1))) == INVALID
    assert bwd(ws=None) == WORKSPACE and bwd(nbytes=1024) == WORKSPACE
    assert bwd(d=gated(B=0), dlam=None) == INVALID


def test_gated_step_refusals(lib):
    good = dict(x=fake(0), r=fake(1), i=fake(2), lam=fake(3), h=fake(4), n=5, slots=None, y=fake(5))

    def step(d=None, **change):
        return lib.mgs_gated_step(ctypes.byref(d or gated(T=1)), *{**good, **change}.values(), None)

    assert lib.mgs_gated_step(None, *good.values(), None) == INVALID
    for name in ("x", "r", "i", "lam", "h", "y"):
        assert step(**{name: None}) == INVALID, name
    assert step(n=1) == INVALID                     # two sequences, one state
    assert step(n=-1) == INVALID and step(n=1, slots=fake(6, 2)) == INVALID
    assert step(y=fake(4)) == INVALID and step(h=fake(0)) == INVALID and step(slots=fake(5)) == INVALID
    assert step(n=1 << 40) == UNSUPPORTED and step(d=gated(dtype=9)) == UNSUPPORTED
    assert step(d=gated(T=-3, x=(400, -1)), x=None) == INVALID   # T and its strides are not read, x is
    assert step(d=gated(B=0), x=None, r=None, i=None, y=None) == OK


# --------------------------------------------------------------- sampling

def sampling(B=4, vocab=1000, stride=1000, dtype=0, top_k=0, temperature=1.0, top_p=1.0, min_p=0.0):
    return SampleDesc(B, vocab, stride, dtype, top_k, temperature, top_p, min_p)


def test_sample_workspace(lib):
    def size(d):
        out = ctypes.c_size_t(0)
        return lib.mgs_sample_workspace_size(ctypes.byref(d), ctypes.byref(out)), out.value

    assert size(sampling())[0] == OK and size(sampling())[1] >= 256 and size(sampling(B=0))[0] == OK
    assert lib.mgs_sample_workspace_size(None, ctypes.byref(ctypes.c_size_t())) == INVALID
    assert lib.mgs_sample_workspace_size(ctypes.byref(sampling()), None) == INVALID
    for bad in (dict(B=-1), dict(vocab=0), dict(vocab=-5), dict(stride=-1)):
        assert size(sampling(**bad))[0] == INVALID, bad
    for bad in (dict(dtype=2), dict(vocab=(1 << 20) + 1), dict(B=1 << 22), dict(B=BIG)):
        assert size(sampling(**bad))[0] == UNSUPPORTED, bad
    assert size(sampling(vocab=1 << 20))[0] == OK


@pytest.mark.parametrize("dtype", [0, 1])
def test_a_sample_workspace_serves_fewer_rows(lib, dtype):
    out = ctypes.c_size_t(0)
    for vocab in (1000, 16385, 32769, 40000, 128000, 1 << 20):
        sizes = []
        for B in range(300):
            d = sampling(B=B, vocab=vocab, stride=vocab, dtype=dtype)
            assert lib.mgs_sample_workspace_size(ctypes.byref(d), ctypes.byref(out)) == OK
            sizes.append(out.value)
        assert sizes == sorted(sizes), vocab


def test_sample_refusals(lib):
    good = dict(logits=fake(0), u=fake(1), temperature=None, top_k=None, top_p=None, min_p=None, token=fake(2),
                logp=fake(3))

    def sample(d=None, ws=fake(9), nbytes=1 << 30, **change):
        return lib.mgs_sample(ctypes.byref(d or sampling()), *{**good, **change}.values(), ws, nbytes, None)

    assert lib.mgs_sample(None, *good.values(), fake(9), 1 << 30, None) == INVALID
    for name in ("logits", "u", "token"):
        assert sample(**{name: None}) == INVALID, name
    assert sample(token=fake(0)) == INVALID and sample(logp=fake(2, 8)) == INVALID and sample(logp=fake(1)) == INVALID
    assert sample(top_p=fake(3)) == INVALID
    for name in ("logits", "u", "temperature", "top_k", "top_p", "min_p", "logp"):
        assert sample(**{name: fake(5, 2)}) == INVALID, name
    assert sample(token=fake(2, 4)) == INVALID
    assert sample(d=sampling(stride=-1)) == INVALID and sample(d=sampling(stride=1 << 60)) == INVALID
    assert sample(ws=None) == WORKSPACE and sample(nbytes=16) == WORKSPACE and sample(ws=fake(9, 8)) == INVALID
    assert sample(d=sampling(B=0), logits=None, u=None, token=None, ws=None) == OK

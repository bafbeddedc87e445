"""Contract of the layer operators' C entry points that needs no GPU: exported symbols, and refusals before any HIP
call (fake, never-dereferenced pointers)."""
import ctypes
import subprocess

import pytest

from scan_linear_rnns_amd import _lib
from scan_linear_rnns_amd._lib import LinattnDesc
from tests.test_abi_cpu import INVALID, OK, UNSUPPORTED, WORKSPACE, fake

I64 = ctypes.c_int64


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def test_exports_every_declared_symbol(lib):
    declared = _lib.declared_functions(_lib.LAYERS_HEADER)
    assert len(declared) == 10, declared
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    for name in declared:
        assert name in exported and name in _lib.SIGNATURES, name


def desc(B=2, T=100, H=4, Hk=2, dk=64, dv=64, dtype=0, per_head=0, **strides):
    st = dict(q=(T * Hk * dk, Hk * dk, dk), k=(T * Hk * dk, Hk * dk, dk), v=(T * H * dv, H * dv, dv),
              do=(T * H * dv, H * dv, dv), g=(T * H, H, 1))
    st.update(strides)
    return LinattnDesc(B, T, H, Hk, dk, dv, dtype, per_head, 1.0, st["q"], st["k"], st["v"], st["do"], st["g"])


def size(lib, d, backward=0):
    out = ctypes.c_size_t(0)
    return lib.mgs_linattn_workspace_size(ctypes.byref(d), backward, ctypes.byref(out)), out.value


def test_linattn_workspace(lib):
    st, fwd = size(lib, desc())
    st2, both = size(lib, desc(), 1)
    assert st == OK and st2 == OK and both >= fwd >= 256
    assert lib.mgs_linattn_workspace_size(None, 0, ctypes.byref(ctypes.c_size_t())) == INVALID
    assert lib.mgs_linattn_workspace_size(ctypes.byref(desc()), 0, None) == INVALID
    for bad in (dict(B=-1), dict(T=-1), dict(H=-4), dict(Hk=3), dict(Hk=0), dict(dk=0), dict(dv=-1), dict(H=0)):
        assert size(lib, desc(**bad))[0] == INVALID, bad
    for bad in (dict(dk=129), dict(dv=256), dict(dtype=2), dict(dtype=-1)):
        assert size(lib, desc(**bad))[0] == UNSUPPORTED, bad
    # sizes whose products pass the limits, with and without wrapping int64
    for bad in (dict(B=1 << 40), dict(T=1 << 31), dict(B=1 << 20, T=1 << 20), dict(B=1 << 30, T=0, H=1 << 30, Hk=1),
                dict(B=(1 << 31) - 100, T=1, H=1, Hk=1, dk=1, dv=1)):
        for backward in (0, 1):
            assert size(lib, desc(**bad), backward)[0] == UNSUPPORTED, bad
    assert size(lib, desc(B=0, T=5))[0] == OK and size(lib, desc(T=0), 1)[0] == OK


def test_linattn_fwd_refusals(lib):
    big = 1 << 30
    d0 = desc()

    def fwd(d=d0, q=fake(0), k=fake(1), v=fake(2), g=fake(3), S0=None, n=None, o=fake(5), ST=fake(6), ws=fake(9),
            nbytes=big):
        return lib.mgs_linattn_fwd(ctypes.byref(d) if d else None, q, k, v, g, S0, n, o, ST, ws, nbytes, None)

    assert fwd(d=None) == INVALID
    for name in ("q", "k", "v", "g", "o"):
        assert fwd(**{name: None}) == INVALID, name
    assert fwd(o=fake(0)) == INVALID                                   # the output over an input
    assert fwd(ST=fake(5, 64)) == INVALID                              # over the other output
    assert fwd(S0=fake(6)) == INVALID                                  # the state in place
    assert fwd(q=fake(0, 2)) == INVALID                                # not aligned to its element
    assert fwd(S0=fake(4, 2)) == INVALID and fwd(n=fake(4, 1)) == INVALID
    assert fwd(d=desc(q=(-1, 64, 64))) == INVALID                      # negative stride
    assert fwd(d=desc(v=(1 << 62, 1 << 62, 1))) == INVALID             # a span past any memory
    assert fwd(d=desc(dk=200)) == UNSUPPORTED
    assert fwd(ws=None) == WORKSPACE and fwd(nbytes=255) == WORKSPACE
    assert fwd(ws=fake(9, 8)) == INVALID
    assert fwd(d=desc(B=0), q=None, k=None, v=None, g=None, o=None, ST=None, ws=None) == OK
    assert fwd(d=desc(T=0), q=None, k=None, v=None, g=None, o=None, ST=None, ws=None) == OK


def test_linattn_bwd_and_step_refusals(lib):
    big = 1 << 30
    names = ("q", "k", "v", "g", "do", "S0", "dST", "lengths", "dq", "dk", "dv", "dg", "dS0")
    good = {n: fake(i) for i, n in enumerate(names)}
    good.update(S0=None, dST=None, lengths=None)

    def bwd(d=None, ws=fake(20), nbytes=big, **change):
        a = {**good, **change}
        return lib.mgs_linattn_bwd(ctypes.byref(d or desc()), *(a[n] for n in names), ws, nbytes, None)

    for n in ("q", "k", "v", "g", "do", "dq", "dk", "dv", "dg"):
        assert bwd(**{n: None}) == INVALID, n
    assert bwd(dq=fake(0)) == INVALID and bwd(dk=fake(8)) == INVALID and bwd(dS0=fake(6), dST=fake(6)) == INVALID
    assert bwd(dg=fake(11, 2)) == INVALID
    assert bwd(ws=None) == WORKSPACE and bwd(nbytes=1024) == WORKSPACE
    assert bwd(d=desc(dv=130)) == UNSUPPORTED
    assert bwd(d=desc(B=0), **{n: None for n in names}) == OK

    def step(d=None, q=fake(0), k=fake(1), v=fake(2), g=fake(3), S=fake(4), n=5, slots=None, o=fake(6)):
        return lib.mgs_linattn_step(ctypes.byref(d or desc()), q, k, v, g, S, n, slots, o, None)

    for name in ("q", "k", "v", "g", "S", "o"):
        assert step(**{name: None}) == INVALID, name
    assert step(n=1) == INVALID                                        # two sequences, one state, no slots
    assert step(n=-1) == INVALID and step(S=fake(6)) == INVALID and step(slots=fake(4)) == INVALID
    assert step(n=1 << 40) == UNSUPPORTED and step(d=desc(dk=500)) == UNSUPPORTED
    assert step(d=desc(B=0), q=None, k=None, v=None, g=None, S=None, n=0, o=None) == OK


def test_rmsnorm_refusals(lib):
    def fwd(x=fake(0), r=fake(1), w=fake(2), y=fake(3), h=fake(4), rstd=fake(5), rows=4, d=64, xs=64, rs=64, eps=1e-6,
            dtype=0):
        return lib.mgs_rmsnorm_fwd(x, r, w, y, h, rstd, rows, d, xs, rs, eps, dtype, None)

    for name in ("x", "w", "y"):
        assert fwd(**{name: None}) == INVALID, name
    assert fwd(y=fake(0)) == INVALID and fwd(h=fake(0, 4), r=None) == INVALID and fwd(rstd=fake(2)) == INVALID
    assert fwd(h=fake(1), rs=80) == INVALID                  # in place needs the same rows
    assert fwd(rows=-1) == INVALID and fwd(d=0) == INVALID and fwd(xs=-64) == INVALID
    assert fwd(eps=-1.0) == INVALID and fwd(eps=float("nan")) == INVALID and fwd(x=fake(0, 2)) == INVALID
    assert fwd(dtype=7) == UNSUPPORTED and fwd(d=65537) == UNSUPPORTED and fwd(rows=1 << 36) == UNSUPPORTED
    assert fwd(rows=0, x=None, r=None, w=None, y=None, h=None, rstd=None) == OK

    def fp8(y=fake(3), scale=fake(5), group=0, d=64):
        return lib.mgs_rmsnorm_fwd_fp8(fake(0), None, fake(2), y, scale, None, 4, d, d, d, 1e-6, group, 1, None)

    assert fp8(y=None) == INVALID and fp8(scale=None) == INVALID and fp8(scale=fake(3)) == INVALID
    assert fp8(group=-128) == INVALID and fp8(group=64) == UNSUPPORTED

    out = ctypes.c_size_t(0)
    assert lib.mgs_rmsnorm_workspace_size(100, 64, ctypes.byref(out)) == OK and out.value > 256
    assert lib.mgs_rmsnorm_workspace_size(100, 64, None) == INVALID
    assert lib.mgs_rmsnorm_workspace_size(-1, 64, ctypes.byref(out)) == INVALID

    def bwd(dy=fake(0), h=fake(1), w=fake(2), rstd=fake(3), dh=None, dx=fake(5), dw=fake(6), ws=fake(9), nbytes=1 << 20):
        return lib.mgs_rmsnorm_bwd(dy, h, w, rstd, dh, dx, dw, 4, 64, 0, ws, nbytes, None)

    for name in ("dy", "h", "w", "rstd", "dx", "dw"):
        assert bwd(**{name: None}) == INVALID, name
    assert bwd(dx=fake(1)) == INVALID and bwd(dw=fake(5)) == INVALID and bwd(dx=fake(0, 16)) == INVALID
    assert bwd(ws=None) == WORKSPACE and bwd(nbytes=300) == WORKSPACE


def test_clip_norm_refusals(lib):
    def call(sizes=(10, 20), ins=(0, 1), outs=(2, 3), dtypes=(0, 1), max_norm=1.0, norm=fake(8), ws=fake(9),
             nbytes=1 << 20, n=None):
        n = len(sizes) if n is None else n
        p = lambda t: None if t is None else (ctypes.c_void_p * len(sizes))(  # noqa: E731
            *[None if x is None else (x.value if isinstance(x, ctypes.c_void_p) else fake(x).value) for x in t])
        return lib.mgs_clip_norm(n, p(ins), p(outs), (I64 * len(sizes))(*sizes), (ctypes.c_int * len(sizes))(*dtypes),
                                 max_norm, norm, ws, nbytes, None)

    assert call(ins=(0, None)) == INVALID and call(outs=(None, 3)) == INVALID and call(ins=None) == INVALID
    assert call(norm=None) == INVALID and call(norm=fake(8, 2)) == INVALID and call(norm=fake(0)) == INVALID
    assert call(sizes=(10, -1)) == INVALID and call(n=-1) == INVALID
    assert call(max_norm=-0.5) == INVALID and call(max_norm=float("nan")) == INVALID
    assert call(ins=(fake(0, 2), 1)) == INVALID                       # fp32 at an odd half-word
    assert call(outs=(fake(0, 16), 3)) == INVALID                     # shifted over its input
    assert call(dtypes=(0, 3)) == UNSUPPORTED and call(sizes=(10, 1 << 41)) == UNSUPPORTED
    assert call(sizes=((1 << 62), 1 << 62)) == UNSUPPORTED
    assert call(ws=None) == WORKSPACE and call(nbytes=100) == WORKSPACE
    out = ctypes.c_size_t(0)
    assert lib.mgs_clip_norm_workspace_size(2, (I64 * 2)(5, 1 << 20), ctypes.byref(out)) == OK and out.value > 256
    assert lib.mgs_clip_norm_workspace_size(1, None, ctypes.byref(out)) == INVALID
    assert lib.mgs_clip_norm_workspace_size(0, None, ctypes.byref(out)) == OK


def test_linattn_bwd_of_no_sequences_needs_the_decay_gradient(lib):
    """With decays per head dg is (H) however many sequences there are, so it is required for B = 0 too."""
    names = ("q", "k", "v", "g", "do", "S0", "dST", "lengths", "dq", "dk", "dv", "dg", "dS0")
    none = {n: None for n in names}
    call = lambda d, a: lib.mgs_linattn_bwd(ctypes.byref(d), *(a[n] for n in names), None, 0, None)  # noqa: E731
    for T in (0, 100):
        assert call(desc(B=0, T=T, per_head=1), {**none, "g": fake(3)}) == INVALID
        assert call(desc(B=0, T=T, per_head=0), none) == OK
    assert call(desc(B=0, H=0, Hk=0, per_head=1), none) == OK


def test_rmsnorm_bwd_of_no_rows_needs_the_weights(lib):
    """w and dw are (d), not empty with the rows: a launch would read the one and write the other."""
    def bwd(w=fake(2), dw=fake(6), ws=fake(9)):
        return lib.mgs_rmsnorm_bwd(None, None, w, None, None, None, dw, 0, 64, 0, ws, 1 << 20, None)

    assert bwd(w=None) == INVALID and bwd(dw=None) == INVALID
    assert bwd(ws=None) == WORKSPACE


def test_clip_norm_outputs_over_other_tensors(lib):
    """Two workgroups would read and write the same memory: a tensor listed twice and scaled in place, an output over
    another's input or output, wherever they stand in the list.  Inputs may overlap each other."""
    def call(spans, nbytes=0):
        """spans: (in, out) addresses in bytes past a base, 10 fp32 elements each; WORKSPACE says the checks passed."""
        n = len(spans)
        p = lambda t: (ctypes.c_void_p * n)(*[fake(0, x).value for x in t])  # noqa: E731
        return lib.mgs_clip_norm(n, p([i for i, _ in spans]), p([o for _, o in spans]), (I64 * n)(*[10] * n),
                                 (ctypes.c_int * n)(*[0] * n), 1.0, fake(8), fake(9), nbytes, None)

    far = [(4000 + 80 * i, 8000 + 80 * i) for i in range(20)]
    for rest in ([], far):
        assert call(rest + [(0, 0), (0, 0)]) == INVALID                  # the same tensor twice, in place
        assert call([(0, 0)] + rest + [(20, 20)]) == INVALID             # views that share elements
        assert call([(0, 400)] + rest + [(800, 400)]) == INVALID         # two outputs on one buffer
        assert call([(0, 400)] + rest + [(400, 800)]) == INVALID         # an output over a later input
        assert call([(400, 800)] + rest + [(0, 436)]) == INVALID   # over an earlier one, by a word
        assert call([(400, 400)] + rest + [(0, 364)]) == INVALID
        assert call([(0, 400)] + rest + [(0, 800), (20, 1200)]) == WORKSPACE        # inputs alone may
        assert call([(0, 0)] + rest + [(40, 40), (80, 120)]) == WORKSPACE           # neighbours


def test_limits_of_the_grids(lib):
    """Workgroups of the walks and of the step are numbered in 32 bits: up to 2^31 / 3 segments, 2^28 heads of a step."""
    one = dict(T=1, H=1, Hk=1, dk=1, dv=1)
    for backward in (0, 1):
        assert size(lib, desc(B=(1 << 31) // 3 - 9, **one), backward)[0] == OK
        assert size(lib, desc(B=(1 << 31) // 3, **one), backward)[0] == UNSUPPORTED
    big = desc(B=1 << 28, **one)
    assert lib.mgs_linattn_step(ctypes.byref(big), fake(0), fake(1), fake(2), fake(3), fake(4), 1 << 28, None, fake(6),
                                None) == UNSUPPORTED
    assert lib.mgs_linattn_fwd(ctypes.byref(desc(B=(1 << 31) // 3, **one)), fake(0), fake(8), fake(16), fake(24), None,
                               None, fake(32), None, fake(64), 1 << 62, None) == UNSUPPORTED
    out = ctypes.c_size_t(0)
    assert lib.mgs_rmsnorm_workspace_size(1 << 30, 64, ctypes.byref(out)) == OK

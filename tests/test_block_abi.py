"""Refusals of the recurrence, norm-and-gate and add-norm entry points, on the
host: every call below is turned down before any launch, so the addresses are
never dereferenced."""
import ctypes

import pytest

import linear_recurrent_sequence_scale_b200 as ret

P = ctypes.c_void_p
MB = 1 << 20
A = [P(0x10000000 + k * 64 * MB) for k in range(12)]   # far apart, 256-byte aligned


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(ret.LIB_PATH):
        from linear_recurrent_sequence_scale_b200 import build
        build.build()
    return ret.load_library()


def off(p, n):
    return P(p.value + n)


def test_constants_match_the_header():
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = open(os.path.join(root, "include", "retention.h")).read()
    assert int(re.search(r"#define RET_SCAN_CHUNK (\d+)", src).group(1)) == ret.SCAN_CHUNK
    assert ret.SCAN_FORMS == {"logit": 0, "log": 1}
    assert ret.NORMS == {None: -1, "layer": 0, "rms": 1}


# --- gated linear recurrence -------------------------------------------------------

def pitches(*pairs):
    flat = [v for p in pairs for v in (p if isinstance(p, tuple) else (p,))]
    return (ctypes.c_longlong * len(flat))(*flat)


DENSE = (300 * 64, 64)


def scan_call(lib, x=A[0], f=A[1], g=None, px=DENSE, pf=DENSE, pg=DENSE, py=DENSE, si=None,
              so=None, cs=None, y=A[2], B=2, N=300, D=64, form=0, dt=1, ws=A[3], wsb=None,
              dense=False):
    need = lib.ret_scan_workspace(B, N, D, dt) if wsb is None else wsb
    return lib.ret_scan(x, f, g, si, so, cs, y, None if dense else pitches(px, pf, pg, py), B, N,
                        D, form, dt, ws, need, None)


def test_scan_refusals(lib):
    bad = lambda **kw: scan_call(lib, **kw)  # noqa: E731
    for kw in (dict(x=None), dict(f=None), dict(y=None), dict(B=0), dict(N=-1), dict(D=0),
               dict(form=2), dict(dt=5), dict(px=(300 * 64, 63)), dict(py=(300 * 64, 0)),
               dict(pf=(300 * 64, -64)), dict(pf=(0, 64)), dict(px=(64 * 200, 64)),
               dict(px=(63, 300 * 64)), dict(g=A[4], pg=(300 * 64, 63)), dict(x=off(A[0], 1)),
               dict(g=off(A[4], 1)), dict(x=off(A[0], 2), dt=0), dict(si=off(A[5], 2)),
               dict(cs=off(A[5], 1)), dict(so=off(A[5], 3))):
        assert bad(**kw) == ret.RET_EINVAL, kw
    assert bad(dense=True, B=1 << 20, D=1 << 12) == ret.RET_EUNSUPPORTED
    assert bad(dense=True, N=1 << 30, D=1 << 12) == ret.RET_EUNSUPPORTED
    assert bad(dense=True, B=1, D=1, N=(1 << 31) - 1) == ret.RET_EUNSUPPORTED
    assert bad(dense=True, B=1, D=(1 << 31) - 1, N=1) == ret.RET_EUNSUPPORTED
    assert bad(px=(1 << 60, 64)) == ret.RET_EUNSUPPORTED
    assert bad(px=(64, 1 << 60)) == ret.RET_EUNSUPPORTED
    # short sequences of few channels need no workspace, long ones 12 bytes for each
    # 64 tokens of a channel (rounded up to pieces of 128 bytes of a row)
    assert lib.ret_scan_workspace(2, 300, 64, 1) == 0
    need = lib.ret_scan_workspace(2, 900, 70, 1)
    assert need == 12 * 15 * 2 * 128
    assert lib.ret_scan_workspace(2, 900, 70, 0) == 12 * 15 * 2 * 96
    long = dict(N=900, D=70, dense=True)
    assert bad(ws=None, **long) == ret.RET_EWORKSPACE
    assert bad(wsb=need - 1, **long) == ret.RET_EWORKSPACE
    assert bad(ws=off(A[3], 8), **long) == ret.RET_EINVAL
    assert bad(y=A[3], **long) == ret.RET_EINVAL             # the workspace over y
    assert lib.ret_scan_workspace(0, 300, 64, 1) == 0
    assert lib.ret_scan_workspace(2, 0, 64, 1) == 0
    # no tokens and no state wanted: nothing to do
    assert bad(N=0, x=None, f=None, y=None, ws=None, wsb=0) == ret.RET_OK


def test_scan_overlaps_are_refused(lib):
    """Sharing is refused; interleaving is not.  What is accepted is shown by the
    refusal that the same call meets later, of a missing workspace or operand."""
    bad = lambda **kw: scan_call(lib, **kw)  # noqa: E731
    wide, time_major = (300 * 192, 192), (64, 128)
    assert bad(y=A[0]) == ret.RET_EINVAL                     # y over x
    assert bad(y=off(A[1], 4096)) == ret.RET_EINVAL          # y inside f
    assert bad(y=off(A[0], 128), px=wide, py=(300 * 128, 128)) == ret.RET_EINVAL
    assert bad(y=off(A[0], 64), px=wide, py=wide) == ret.RET_EINVAL     # half a slice shared
    assert bad(y=off(A[0], 128), px=time_major, py=time_major) == ret.RET_EINVAL
    assert bad(si=A[5], so=off(A[5], 64)) == ret.RET_EINVAL  # state_out partly over state_in
    assert bad(so=A[0]) == ret.RET_EINVAL
    assert bad(cs=A[6], so=A[6]) == ret.RET_EINVAL
    assert bad(N=0, si=A[5], so=off(A[5], 64)) == ret.RET_EINVAL


def test_scan_step_refusals(lib):
    def call(x=A[0], f=A[1], g=None, ldx=64, ldf=64, ldg=64, si=A[2], so=A[2], y=A[3], ldy=64,
             B=4, D=64, form=1, dt=1):
        return lib.ret_scan_step(x, f, g, si, so, y, pitches(ldx, ldf, ldg, ldy), B, D, form, dt,
                                 None)
    for kw in (dict(x=None), dict(si=None), dict(so=None), dict(y=None), dict(ldx=32),
               dict(form=-1), dict(dt=2), dict(D=0), dict(B=-1), dict(y=A[0]), dict(y=A[2]),
               dict(so=off(A[2], 16)), dict(si=off(A[2], 2)), dict(g=A[3]),
               dict(g=A[4], ldg=10)):
        assert call(**kw) == ret.RET_EINVAL, kw


def test_scan_backward_refusals(lib):
    def call(x=A[0], f=A[1], g=None, cs=A[2], dy=A[3], ds=None, gx=A[4], gf=A[5], gg=None,
             dsi=A[6], pgx=DENSE, pgg=DENSE, B=2, N=300, D=64, form=0, dt=1, ws=A[7], wsb=None):
        need = lib.ret_scan_workspace(B, N, D, dt) if wsb is None else wsb
        p = pitches(DENSE, DENSE, DENSE, DENSE, pgx, DENSE, pgg)
        return lib.ret_scan_backward(x, f, g, cs, dy, ds, gx, gf, gg, dsi, p, B, N, D, form, dt,
                                     ws, need, None)
    for kw in (dict(cs=None), dict(dy=None), dict(gx=None), dict(gf=None), dict(g=A[8]),
               dict(pgx=(300 * 64, 32)), dict(gx=A[3]), dict(gx=A[5]), dict(gx=A[0]),
               dict(dsi=A[2]), dict(g=A[8], gg=A[8]), dict(g=A[8], gg=A[9], pgg=(300 * 64, 8)),
               dict(form=9), dict(dt=-1), dict(cs=off(A[2], 1)), dict(ds=off(A[8], 2)),
               dict(ds=off(A[6], 4)), dict(gx=off(A[4], 1))):
        assert call(**kw) == ret.RET_EINVAL, kw
    assert call(N=0, x=None, f=None, cs=None, dy=None, gx=None, gf=None, dsi=None, ws=None,
                wsb=0) == ret.RET_OK


# --- norm and gate -----------------------------------------------------------------

def test_norm_gate_refusals(lib):
    def call(y=A[0], g=A[1], o=A[2], B=2, H=3, N=50, dv=64, norm=0, eps=1e-5, tm=1, ldg=0, ldo=0,
             dt=1):
        return lib.ret_norm_gate(y, g, o, B, H, N, dv, norm, eps, tm, ldg, ldo, dt, None)
    for kw in (dict(y=None), dict(o=None), dict(dv=60), dict(dv=0), dict(H=0), dict(N=-1),
               dict(norm=2), dict(norm=-1), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(dt=3), dict(ldg=100), dict(ldo=196),
               dict(ldg=-8), dict(o=off(A[2], 8)), dict(g=off(A[1], 4)),
               dict(o=A[0]),                              # another layout than y's
               dict(o=A[1], ldg=256, ldo=192),            # the gate's array, another pitch
               dict(o=off(A[0], 64))):
        assert call(**kw) == ret.RET_EINVAL, kw
    assert call(dv=2048) == ret.RET_EUNSUPPORTED
    assert call(B=1000, H=100) == ret.RET_EUNSUPPORTED
    assert call(B=1, H=1, dv=8, N=(1 << 31) - 1) == ret.RET_EUNSUPPORTED
    assert call(N=0, y=None, g=None, o=None) == ret.RET_OK


def test_norm_gate_backward_refusals(lib):
    def call(y=A[0], g=A[1], do=A[2], gy=A[3], gg=A[4], N=50, dv=64, norm=0, eps=1e-5, tm=1,
             ldg=0, lddo=0, ldgg=0, dt=1):
        return lib.ret_norm_gate_backward(y, g, do, gy, gg, 2, 3, N, dv, norm, eps, tm, ldg, lddo,
                                          ldgg, dt, None)
    for kw in (dict(y=None), dict(do=None), dict(gy=None), dict(gg=None), dict(gy=A[2]),
               dict(gg=A[0]), dict(gg=A[3]), dict(dv=4), dict(norm=7), dict(ldgg=8),
               dict(gg=off(A[4], 2)), dict(lddo=193)):
        assert call(**kw) == ret.RET_EINVAL, kw
    assert call(N=0, y=None, g=None, do=None, gy=None, gg=None) == ret.RET_OK


# --- residual and norms ------------------------------------------------------------

def test_add_norm_refusals(lib):
    def call(x=A[0], r=A[1], wp=None, w=A[2], ro=A[3], y=A[4], rows=10, d=100, post=-1, norm=1,
             al=1.0, be=1.0, eps=1e-5, dt=1):
        return lib.ret_add_norm(x, r, wp, w, ro, y, rows, d, post, norm, al, be, eps, dt, None)
    for kw in (dict(x=None), dict(ro=None), dict(y=None), dict(rows=-1), dict(d=0), dict(post=2),
               dict(norm=-1), dict(eps=-1e-9), dict(eps=float("nan")), dict(al=float("inf")),
               dict(be=float("nan")), dict(dt=4), dict(w=off(A[2], 4)), dict(wp=off(A[5], 8)),
               dict(x=off(A[0], 1)), dict(ro=A[4]), dict(ro=off(A[1], 2)), dict(y=A[2])):
        assert call(**kw) == ret.RET_EINVAL, kw
    assert call(d=16385) == ret.RET_EUNSUPPORTED
    assert call(rows=1 << 40) == ret.RET_EUNSUPPORTED
    assert call(rows=0, x=None, r=None, ro=None, y=None) == ret.RET_OK


def test_add_norm_backward_refusals(lib):
    need = lib.ret_add_norm_backward_workspace(10, 100)
    assert need > 0
    assert lib.ret_add_norm_backward_workspace(-1, 100) == 0
    assert lib.ret_add_norm_backward_workspace(10, 1 << 20) == 0

    def call(x=A[0], ro=A[1], wp=None, w=A[2], dy=A[3], dr=A[4], gx=A[5], gr=A[6], gw=A[7],
             gp=None, post=-1, rows=10, dt=1, ws=A[9], wsb=need):
        return lib.ret_add_norm_backward(x, ro, wp, w, dy, dr, gx, gr, gw, gp, rows, 100, post, 0,
                                         1.0, 1.0, 1e-5, dt, ws, wsb, None)
    for kw in (dict(ro=None), dict(dy=None), dict(x=None, post=1), dict(x=None, gp=A[8]),
               dict(gx=A[6]), dict(gw=A[2]), dict(gw=off(A[7], 2)), dict(gp=A[7]),
               dict(gx=off(A[3], 2)), dict(post=5), dict(ws=off(A[9], 4)), dict(ws=A[1]),
               dict(rows=0, gp=A[7])):
        assert call(**kw) == ret.RET_EINVAL, kw
    assert call(ws=None) == ret.RET_EWORKSPACE
    assert call(wsb=need - 1) == ret.RET_EWORKSPACE
    assert call(rows=0, x=None, ro=None, dy=None, dr=None, gx=None, gr=None, gw=None, ws=None,
                wsb=0) == ret.RET_OK


# --- the Python binding's own checks --------------------------------------------------

def test_binding_checks_come_before_the_library():
    import torch
    x = torch.zeros(2, 5, 8)
    with pytest.raises(ValueError, match="CUDA"):
        ret.scan(x, x)
    with pytest.raises(ValueError, match="form"):
        ret.scan(x, x, form="linear")
    with pytest.raises(ValueError, match=r"\[B,N,D\]"):
        ret.scan(x[0], x[0])
    with pytest.raises(TypeError, match="dtype"):
        ret.scan(x.half(), x.half())
    with pytest.raises(ValueError, match=r"\[B,D\]"):
        ret.scan_step(x, x, x)
    with pytest.raises(ValueError, match=r"\[B,H,N,dv\]"):
        ret.norm_gate(x)
    with pytest.raises(ValueError, match="CUDA"):
        ret.add_norm(x, None)

"""Refusals of the Mamba-2 operators over packed sequences that need no GPU: every bad argument is rejected on the host
before anything is launched."""
import pytest

A = 0x10000    # a fake, aligned "device" address: never dereferenced
BIG = 1 << 60  # a workspace size no query exceeds in these cases


def _raw(name, *args):
    from bit_scaffold_int8_amd import dfssm
    return dfssm.raw(name, *args)


def _conv(**kw):
    a = dict(x=A, ldx=64, ti=0, T=12, S=3, ch=64, cu=None, w=A, b=A, win=A, wout=1 << 30, out=A, ldo=64, to=0)
    a.update(kw)
    return _raw("dfssm_mamba2_conv", a["x"], a["ldx"], a["ti"], a["T"], a["S"], a["ch"], a["cu"], a["w"], a["b"], a["win"],
                a["wout"], a["out"], a["ldo"], a["to"], None)


def _conv_backward(**kw):
    a = dict(x=A, ldx=64, ti=0, T=12, S=3, ch=64, cu=None, w=A, b=A, win=A, dout=A, ldd=64, to=0, dwout=A, dx=A, lddx=64,
             dw=A, db=A, dwin=1 << 30, ws=A, n=BIG)
    a.update(kw)
    return _raw("dfssm_mamba2_conv_backward", a["x"], a["ldx"], a["ti"], a["T"], a["S"], a["ch"], a["cu"], a["w"], a["b"],
                a["win"], a["dout"], a["ldd"], a["to"], a["dwout"], a["dx"], a["lddx"], a["dw"], a["db"], a["dwin"], a["ws"],
                a["n"], None)


_CONV = [
    (dict(x=None), 1), (dict(w=None), 1), (dict(b=None), 1), (dict(T=0), 1), (dict(S=0), 1), (dict(ch=0), 1), (dict(T=-1), 1),
    (dict(T=1 << 31, S=1), 1), (dict(S=1 << 31, cu=A), 1), (dict(T=13), 1), (dict(ti=2), 1), (dict(to=-1), 1),
    (dict(ldx=63), 1), (dict(x=A + 2), 1), (dict(x=A + 1, ti=1), 1), (dict(w=A + 8), 1), (dict(b=A + 2), 1),
    (dict(win=A + 8), 1), (dict(cu=A + 2), 1), (dict(T=(1 << 20) + 4, S=4), 2), (dict(S=65536, T=65536), 2),
    (dict(ch=(1 << 18) + 1, ldx=1 << 21, ldo=1 << 21, ldd=1 << 21, lddx=1 << 21), 2), (dict(ldx=1 << 31), 2),
    (dict(T=(1 << 17) + 1, S=1, ch=1 << 17, ldx=1 << 21, ldo=1 << 21, ldd=1 << 21, lddx=1 << 21), 2),   # (a launch of 2^32 threads)
]


def _only(kw, names):
    return {k: v for k, v in kw.items() if k in names}


@pytest.mark.parametrize("kw,want", _CONV + [
    (dict(out=None), 1), (dict(ldo=63), 1), (dict(out=A + 2), 1), (dict(wout=A), 1), (dict(wout=A + 16), 1),
    (dict(wout=A + 8), 1), (dict(ldo=1 << 31), 2),
])
def test_conv_rejects(kw, want):
    assert _conv(**kw) == want


@pytest.mark.parametrize("kw,want", _CONV + [
    (dict(dout=None), 1), (dict(dx=None), 1), (dict(ldd=63), 1), (dict(lddx=63), 1), (dict(dout=A + 2), 1),
    (dict(dx=A + 2), 1), (dict(dw=None), 1), (dict(db=None), 1), (dict(dw=A + 4), 1), (dict(db=A + 1), 1), (dict(ws=None), 1),
    (dict(ws=A + 8), 1), (dict(n=0), 1), (dict(dwin=A), 1), (dict(dwout=A + 4), 1), (dict(ldd=1 << 31), 2),
    (dict(lddx=1 << 31), 2),
])
def test_conv_backward_rejects(kw, want):
    assert _conv_backward(**kw) == want


def _operands(**kw):
    from bit_scaffold_int8_amd import dfssm
    a = dict(x=A, B=A, C=A, dt=A, A_log=A, D=A, dt_bias=A, state_in=A, cu_seqlens=None, ldx=256, ldb=128, ldc=128, lddt=4, T=12,
             S=3, nheads=4, headdim=64, d_state=128, ngroups=1, type=0)
    a.update(kw)
    return dfssm.ScanOperands(*[a[n] for n in dfssm.SCAN_POINTERS + dfssm.SCAN_SIZES], a["type"])


def _scan(y=A, ldy=256, state_out=1 << 40, ws=A, n=BIG, null=False, **kw):
    import ctypes
    op = _operands(**kw)
    return _raw("dfssm_mamba2_scan", None if null else ctypes.addressof(op), y, ldy, state_out, ws, n, None)


_SCAN = [
    (dict(null=True), 1), (dict(x=None), 1), (dict(B=None), 1), (dict(C=None), 1), (dict(dt=None), 1), (dict(A_log=None), 1),
    (dict(D=None), 1), (dict(dt_bias=None), 1), (dict(ws=None), 1), (dict(ws=A + 8), 1), (dict(n=0), 1),
    (dict(T=0), 1), (dict(S=0), 1), (dict(nheads=0), 1), (dict(headdim=0), 1), (dict(d_state=0), 1), (dict(ngroups=0), 1),
    (dict(ngroups=3), 1), (dict(T=13), 1), (dict(T=1 << 31, S=1), 1), (dict(type=2), 1), (dict(ldx=252), 1),
    (dict(ldb=124), 1), (dict(ldc=64), 1), (dict(lddt=3), 1), (dict(x=A + 8), 1), (dict(B=A + 4), 1), (dict(C=A + 8), 1),
    (dict(ldx=258), 1), (dict(ldx=260, type=1), 1), (dict(ldb=130), 1), (dict(ldc=132, type=1), 1), (dict(dt=A + 2), 1), (dict(A_log=A + 1), 1),
    (dict(D=A + 2), 1), (dict(dt_bias=A + 2), 1), (dict(state_in=A + 8), 1), (dict(cu_seqlens=A + 2), 1),
    (dict(headdim=32), 2), (dict(d_state=256, ldb=256, ldc=256), 2),
    (dict(nheads=1025, ngroups=1, ldx=65600, ldy=65600, lddt=1025, lddy=65600, lddx=65600, ldddt=1025), 2),
    (dict(T=(1 << 20) + 4, S=4), 2), (dict(T=65536, S=65536), 2), (dict(lddt=1 << 31), 2), (dict(ldx=1 << 31), 2),
    (dict(T=65535, S=65535, nheads=64, ldx=4096, ldy=4096, lddt=64, lddy=4096, lddx=4096, ldddt=64), 2),
    # a launch of 2^32 threads: 4096 chunks and a sequence of 1024 groups
    (dict(T=4096 * 64, S=1, nheads=1024, ngroups=1024, d_state=64, ldx=65536, ldb=65536, ldc=65536, ldy=65536, lddt=1024,
          lddy=65536, lddx=65536, lddb=65536, lddc=65536, ldddt=1024), 2),
]


@pytest.mark.parametrize("kw,want", _SCAN + [
    (dict(y=None), 1), (dict(y=A + 8), 1), (dict(ldy=252), 1), (dict(ldy=258), 1), (dict(state_out=A + 16), 1),
    (dict(state_out=A + 8), 1), (dict(ldy=1 << 31), 2),
])
def test_scan_rejects(kw, want):
    kw = {k: v for k, v in kw.items() if not k.startswith("ldd") or k == "lddt"}
    assert _scan(**kw) == want


def _scan_backward(ws=A, n=BIG, null=False, no_gradients=False, **kw):
    import ctypes
    from bit_scaffold_int8_amd import dfssm
    g = dict(dy=A, dstate_out=A, dx=A, dB=A, dC=A, ddt=A, dA_log=A, dD=A, ddt_bias_=A, dstate_in=1 << 40, lddy=256, lddx=256,
             lddb=128, lddc=128, ldddt=4)
    g.update({k: v for k, v in kw.items() if k in g})
    op = _operands(**{k: v for k, v in kw.items() if k not in g and k != "ldy"})
    names = [n if n != "ddt_bias" else "ddt_bias_" for n in dfssm.SCAN_GRADIENTS + dfssm.SCAN_GRADIENT_SIZES]
    grad = dfssm.ScanGradients(*[g[n] for n in names])
    return _raw("dfssm_mamba2_scan_backward", None if null else ctypes.addressof(op),
                None if no_gradients else ctypes.addressof(grad), ws, n, None)


@pytest.mark.parametrize("kw,want", _SCAN + [
    (dict(no_gradients=True), 1), (dict(dy=None), 1), (dict(dx=None), 1), (dict(dB=None), 1), (dict(dC=None), 1), (dict(ddt=None), 1),
    (dict(dA_log=None), 1), (dict(dD=None), 1), (dict(ddt_bias_=None), 1), (dict(dy=A + 8), 1), (dict(dx=A + 4), 1),
    (dict(dB=A + 8), 1), (dict(dC=A + 8), 1), (dict(ddt=A + 2), 1), (dict(dA_log=A + 1), 1), (dict(dD=A + 2), 1),
    (dict(ddt_bias_=A + 2), 1), (dict(dstate_out=A + 8), 1), (dict(dstate_in=A + 16), 1), (dict(dstate_in=A), 1),
    (dict(lddy=252), 1), (dict(lddx=258), 1), (dict(lddb=64), 1), (dict(lddc=130), 1), (dict(ldddt=3), 1), (dict(lddy=1 << 31), 2),
    (dict(ldddt=1 << 31), 2),
])
def test_scan_backward_rejects(kw, want):
    assert _scan_backward(**kw) == want


def test_workspace_queries():
    from bit_scaffold_int8_amd import dfssm
    q = dfssm.dfssm_mamba2_scan_workspace_bytes
    assert q(0, 1, 1, 64, 128) == 0 and q(8, 1, 1, 32, 128) == 0 and q(8, 1, 4, 64, 128, 3) == 0
    assert dfssm.dfssm_mamba2_conv_backward_workspace_bytes(0, 1, 4) == 0
    base = (2048, 8, 64, 64, 64, 1)
    b = dfssm.dfssm_mamba2_scan_backward_workspace_bytes
    assert b(0, 1, 1, 64, 128) == 0 and b(*base) > q(*base)
    for i, more in ((0, 2049), (1, 9), (2, 65), (4, 128), (5, 2)):
        bigger = list(base)
        bigger[i] = more
        assert q(*bigger) >= q(*base) > 0 and b(*bigger) >= b(*base)

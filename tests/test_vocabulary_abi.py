"""Refusals of the vocabulary operators (int8 product, cross entropy, embedding gradient) that need no
GPU: every bad argument is rejected on the host before anything is launched."""
import pytest

A = 0x10000   # a fake, aligned "device" address: never dereferenced
BIG = 1 << 40  # a workspace size no query exceeds in these cases


def _raw(name, *args):
    from bit_scaffold_int8_amd import dfssm
    return dfssm.raw(name, *args)


def _gemm(**kw):
    a = dict(x_q=A, ldx=64, s_x=A, M=4, N=8, K=64, w=A, ldw=64, s_w=A, y=A, ldy=8, t=0)
    a.update(kw)
    return _raw("dfssm_int8_gemm", a["x_q"], a["ldx"], a["s_x"], a["M"], a["N"], a["K"], a["w"], a["ldw"], a["s_w"],
                a["y"], a["ldy"], a["t"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(x_q=None), 1), (dict(s_x=None), 1), (dict(w=None), 1), (dict(s_w=None), 1), (dict(y=None), 1),
    (dict(M=0), 1), (dict(N=0), 1), (dict(K=0), 1), (dict(M=-1), 1), (dict(M=1 << 31), 1), (dict(N=1 << 31), 1),
    (dict(ldx=63), 1), (dict(ldw=63), 1), (dict(ldy=7), 1), (dict(t=2), 1), (dict(t=-1), 1),
    (dict(s_x=A + 2), 1), (dict(s_w=A + 1), 1), (dict(y=A + 2), 1), (dict(y=A + 1, t=1), 1),
    (dict(K=131073, ldx=131073, ldw=131073), 2), (dict(ldx=(1 << 22) + 1), 2), (dict(ldw=(1 << 22) + 16), 2),
    (dict(ldy=1 << 40), 2), (dict(M=(1 << 31) - 1, N=(1 << 31) - 1, ldy=1 << 32), 2),
])
def test_int8_gemm_rejects(kw, want):
    assert _gemm(**kw) == want


def _loss(**kw):
    a = dict(x_q=A, s_x=A, M=4, V=8, K=64, e=A, s_e=A, targets=A, loss=A, lse=A, ws=A, n=BIG)
    a.update(kw)
    return _raw("dfssm_cross_entropy", a["x_q"], a["s_x"], a["M"], a["V"], a["K"], a["e"], a["s_e"], a["targets"],
                a["loss"], a["lse"], a["ws"], a["n"], None)


def _backward(**kw):
    a = dict(x_q=A, s_x=A, M=4, V=8, K=64, e=A, s_e=A, targets=A, lse=A, dloss=A, dx=A, de=A, t=0, acc=0, ws=A, n=BIG)
    a.update(kw)
    return _raw("dfssm_cross_entropy_backward", a["x_q"], a["s_x"], a["M"], a["V"], a["K"], a["e"], a["s_e"],
                a["targets"], a["lse"], a["dloss"], a["dx"], a["de"], a["t"], a["acc"], a["ws"], a["n"], None)


_COMMON = [
    (dict(x_q=None), 1), (dict(s_x=None), 1), (dict(e=None), 1), (dict(s_e=None), 1), (dict(targets=None), 1),
    (dict(lse=None), 1), (dict(ws=None), 1), (dict(M=0), 1), (dict(V=0), 1), (dict(K=0), 1), (dict(K=24), 1),
    (dict(M=1 << 31), 1), (dict(V=1 << 31), 1), (dict(x_q=A + 8), 1), (dict(e=A + 4), 1), (dict(ws=A + 8), 1),
    (dict(s_x=A + 2), 1), (dict(s_e=A + 1), 1), (dict(targets=A + 2), 1), (dict(lse=A + 2), 1), (dict(n=0), 1),
    (dict(K=131072 + 16), 2), (dict(M=(1 << 31) - 1, V=(1 << 31) - 1), 2), (dict(M=(1 << 25) + 1), 2),
    (dict(V=(1 << 28) + 1), 2), (dict(M=1 << 24, V=(1 << 14) + 1), 2),
]


@pytest.mark.parametrize("kw,want", _COMMON + [(dict(loss=None), 1), (dict(loss=A + 2), 1)])
def test_cross_entropy_rejects(kw, want):
    assert _loss(**kw) == want


@pytest.mark.parametrize("kw,want", _COMMON + [
    (dict(dloss=None), 1), (dict(dloss=A + 1), 1), (dict(dx=None, de=None), 1), (dict(dx=A + 8), 1),
    (dict(de=A + 4), 1), (dict(t=2), 1), (dict(acc=2), 1), (dict(M=(1 << 18) + 1), 2),
])
def test_cross_entropy_backward_rejects(kw, want):
    assert _backward(**kw) == want


def _lookup(**kw):
    a = dict(tokens=A, T=4, e=A, s_e=A, V=8, K=64, out=A, ldo=64, t=0)
    a.update(kw)
    return _raw("dfssm_embedding_lookup_scaled", a["tokens"], a["T"], a["e"], a["s_e"], a["V"], a["K"], 1.0, a["out"],
                a["ldo"], a["t"], None)


def _embgrad(**kw):
    a = dict(tokens=A, T=4, dout=A, ldd=64, td=0, V=8, K=64, de=A, te=0, acc=0, ws=A, n=BIG)
    a.update(kw)
    return _raw("dfssm_embedding_backward", a["tokens"], a["T"], a["dout"], a["ldd"], a["td"], a["V"], a["K"], 1.0,
                a["de"], a["te"], a["acc"], a["ws"], a["n"], None)


_EMB = [(dict(tokens=None), 1), (dict(T=0), 1), (dict(V=0), 1), (dict(K=0), 1), (dict(T=1 << 31), 1),
        (dict(V=1 << 31), 1), (dict(tokens=A + 2), 1)]


@pytest.mark.parametrize("kw,want", _EMB + [
    (dict(e=None), 1), (dict(s_e=None), 1), (dict(out=None), 1), (dict(s_e=A + 2), 1), (dict(out=A + 2), 1),
    (dict(out=A + 1, t=1), 1), (dict(ldo=63), 1), (dict(t=3), 1), (dict(K=131073, ldo=131073), 2), (dict(ldo=1 << 31), 2),
])
def test_embedding_lookup_scaled_rejects(kw, want):
    assert _lookup(**kw) == want


@pytest.mark.parametrize("kw,want", _EMB + [
    (dict(dout=None), 1), (dict(de=None), 1), (dict(ws=None), 1), (dict(ws=A + 4), 1), (dict(dout=A + 2), 1),
    (dict(dout=A + 1, td=1), 1), (dict(de=A + 2), 1), (dict(ldd=63), 1), (dict(td=2), 1), (dict(te=-1), 1),
    (dict(acc=-1), 1), (dict(n=0), 1), (dict(T=(1 << 24) + 1), 2), (dict(V=(1 << 28) + 1), 2), (dict(K=131073, ldd=131073), 2), (dict(ldd=1 << 31), 2),
])
def test_embedding_backward_rejects(kw, want):
    assert _embgrad(**kw) == want


def test_workspace_queries():
    from bit_scaffold_int8_amd import dfssm
    q = dfssm.raw
    for n in (q("dfssm_cross_entropy_workspace_bytes", 4, 8, 64),
              q("dfssm_cross_entropy_backward_workspace_bytes", 4, 8, 64, 0, 1, 1),
              q("dfssm_embedding_backward_workspace_bytes", 4, 8, 64)):
        assert 0 < n < BIG
    # what the calls refuse has no workspace
    assert q("dfssm_cross_entropy_workspace_bytes", 0, 8, 64) == 0
    assert q("dfssm_cross_entropy_workspace_bytes", 4, 8, 24) == 0
    assert q("dfssm_cross_entropy_backward_workspace_bytes", 4, 8, 64, 2, 1, 1) == 0
    assert q("dfssm_cross_entropy_backward_workspace_bytes", 4, 8, 64, 0, 0, 0) == 0
    assert q("dfssm_cross_entropy_backward_workspace_bytes", (1 << 18) + 1, 8, 64, 0, 1, 1) == 0
    assert q("dfssm_embedding_backward_workspace_bytes", (1 << 24) + 1, 8, 64) == 0
    # one byte short of the query is refused
    for M, V, K in ((1, 1, 16), (300, 5000, 2048), (262144, 50280, 2048)):
        n = q("dfssm_cross_entropy_workspace_bytes", M, V, K)
        assert _loss(M=M, V=V, K=K, n=n - 1) == 1
        for t in (0, 1):
            n = q("dfssm_cross_entropy_backward_workspace_bytes", M, V, K, t, 1, 0)
            assert _backward(M=M, V=V, K=K, t=t, de=None, n=n - 1) == 1
        n = q("dfssm_embedding_backward_workspace_bytes", M, V, K)
        assert _embgrad(T=M, V=V, K=K, ldd=K, n=n - 1) == 1


def test_binding_checks_what_the_abi_cannot_see():
    """Types, shapes, strides and devices of tensors: ValueError before any call."""
    import torch
    from bit_scaffold_int8_amd import dfssm
    x, sx = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    w, sw, y = torch.zeros(8, 64, dtype=torch.int8), torch.zeros(8), torch.zeros(4, 8)
    tok = torch.zeros(4, dtype=torch.int32)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)

    def bad(f, *args):
        with pytest.raises(ValueError):
            f(*args)
    g = dfssm.dfssm_int8_gemm
    bad(g, x, sx, w, sw, y)                                    # on the CPU
    bad(g, x.float(), sx, w, sw, y)
    bad(g, x, sx, w[:, :32], sw, y)
    bad(g, x, sx, w, sw, y.half())
    bad(g, x, sx, w, sw, torch.zeros(8, 4).t())                # columns contiguous instead of rows
    bad(g, x, sx, w, sw, torch.zeros(1, 8).expand(4, 8))       # rows that overlap
    bad(g, x, sx.double(), w, sw, y)
    bad(g, x, sx[:3], w, sw, y)
    bad(dfssm.dfssm_cross_entropy, x, sx, w, sw, tok.long(), sx, sx, ws)
    bad(dfssm.dfssm_cross_entropy, x, sx, w[::2], sw[:4], tok, sx, sx, ws)
    dx, de = torch.zeros(4, 64), torch.zeros(8, 64)
    b = dfssm.dfssm_cross_entropy_backward
    bad(b, x, sx, w, sw, tok, sx, sx, None, None, ws)
    bad(b, x, sx, w, sw, tok, sx, sx, dx, de.bfloat16(), ws)
    bad(b, x, sx, w, sw, tok, sx, sx, dx.t(), de, ws)
    bad(b, x, sx, w, sw, tok, sx, sx, dx, de, ws[::2])
    bad(dfssm.dfssm_embedding_lookup_scaled, tok.long(), w, sw, 1.0, dx)
    bad(dfssm.dfssm_embedding_lookup_scaled, tok, w, sw, 1.0, dx[:, :32])
    bad(dfssm.dfssm_embedding_backward, tok, dx[:3], 1.0, de, ws)
    bad(dfssm.dfssm_embedding_backward, tok, dx, 1.0, de.half(), ws)

"""Refusals of the distillation loss that need no GPU: every bad argument is rejected on the host before anything is launched."""
import pytest

A = 0x10000    # a fake, aligned "device" address: never dereferenced
BIG = 1 << 50  # a workspace size no query exceeds in these cases


def _forward(**kw):
    from bit_scaffold_int8_amd import dfssm
    a = dict(x_q=A, s_x=A, M=4, V=8, K=64, e=A, s_e=A, ids=A, top=A, k=5, T=1.0, loss=A, lse=A, logp=A, ws=A, n=BIG)
    a.update(kw)
    return dfssm.raw("dfssm_distillation", a["x_q"], a["s_x"], a["M"], a["V"], a["K"], a["e"], a["s_e"], a["ids"], a["top"],
                     a["k"], a["T"], a["loss"], a["lse"], a["logp"], a["ws"], a["n"], None)


def _backward(**kw):
    from bit_scaffold_int8_amd import dfssm
    a = dict(x_q=A, s_x=A, M=4, V=8, K=64, e=A, s_e=A, ids=A, top=A, k=5, T=1.0, lse=A, logp=A, dloss=A, dx=A, de=A, t=0,
             acc=0, ws=A, n=BIG)
    a.update(kw)
    return dfssm.raw("dfssm_distillation_backward", a["x_q"], a["s_x"], a["M"], a["V"], a["K"], a["e"], a["s_e"], a["ids"],
                     a["top"], a["k"], a["T"], a["lse"], a["logp"], a["dloss"], a["dx"], a["de"], a["t"], a["acc"],
                     a["ws"], a["n"], None)


_COMMON = [
    (dict(x_q=None), 1), (dict(s_x=None), 1), (dict(e=None), 1), (dict(s_e=None), 1), (dict(ids=None), 1), (dict(top=None), 1),
    (dict(lse=None), 1), (dict(logp=None), 1), (dict(ws=None), 1), (dict(M=0), 1), (dict(V=0), 1), (dict(K=0), 1),
    (dict(K=24), 1), (dict(k=0), 1), (dict(k=-1), 1), (dict(M=1 << 31), 1), (dict(V=1 << 31), 1), (dict(x_q=A + 8), 1),
    (dict(e=A + 4), 1), (dict(ws=A + 8), 1), (dict(s_x=A + 2), 1), (dict(s_e=A + 1), 1), (dict(ids=A + 2), 1), (dict(top=A + 1), 1),
    (dict(lse=A + 2), 1), (dict(logp=A + 2), 1), (dict(n=0), 1), (dict(T=0.0), 1), (dict(T=-1.0), 1), (dict(T=float("nan")), 1),
    (dict(T=float("inf")), 1), (dict(T=1e-30), 1), (dict(k=257), 2), (dict(K=131072 + 16), 2), (dict(V=(1 << 28) + 1), 2),
]


@pytest.mark.parametrize("kw,want", _COMMON + [(dict(loss=None), 1), (dict(loss=A + 2), 1), (dict(M=(1 << 25) + 1), 2),
                                               (dict(M=1 << 22, k=65), 2)])
def test_distillation_rejects(kw, want):
    assert _forward(**kw) == want


@pytest.mark.parametrize("kw,want", _COMMON + [
    (dict(dloss=None), 1), (dict(dloss=A + 1), 1), (dict(dx=None, de=None), 1), (dict(dx=A + 8), 1),
    (dict(de=A + 4), 1), (dict(t=2), 1), (dict(acc=2), 1), (dict(M=(1 << 18) + 1), 2),
])
def test_distillation_backward_rejects(kw, want):
    assert _backward(**kw) == want


def test_workspace_queries():
    from bit_scaffold_int8_amd import dfssm
    f, b = dfssm.lib.dfssm_distillation_workspace_bytes, dfssm.lib.dfssm_distillation_backward_workspace_bytes
    assert f(4, 8, 64, 0) == 0 and f(4, 8, 24, 5) == 0 and f(4, 8, 64, 257) == 0 and f(4, 8, 64, 5) > 0
    assert b(4, 8, 64, 5, 0, 0, 0) == 0 and b(4, 8, 64, 5, 2, 1, 1) == 0
    sizes = [100, 900, 64, 20]
    for i in range(4):
        more = list(sizes)
        more[i] += 16
        assert b(*more, 0, 1, 1) >= b(*sizes, 0, 1, 1) > 0 and f(*more) >= f(*sizes)
    assert b(*sizes, 0, 1, 1) >= b(*sizes, 1, 1, 0)


def test_binding_refuses_other_shapes_and_types():
    import torch
    from bit_scaffold_int8_amd import dfssm
    x_q, s_x, e, s_e = torch.zeros(3, 16, dtype=torch.int8), torch.zeros(3), torch.zeros(7, 16, dtype=torch.int8), torch.zeros(7)
    ids, top, out, ws = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2), torch.zeros(3), torch.zeros(64)

    def call(**kw):
        a = dict(x_q=x_q, s_x=s_x, e=e, s_e=s_e, ids=ids, top=top, loss=out, lse=out.clone(), logp=top.clone())
        a.update(kw)
        dfssm.dfssm_distillation(a["x_q"], a["s_x"], a["e"], a["s_e"], a["ids"], a["top"], 1.0, a["loss"], a["lse"], a["logp"], ws)
    for kw in (dict(ids=ids.long()), dict(top=top.double()), dict(top=top[:, :1]), dict(ids=ids.t()), dict(loss=out[:2]),
               dict(logp=top.t()), dict(x_q=x_q.float()), dict(s_e=s_e[:3]), {}):   # (the last: not on a GPU)
        with pytest.raises(ValueError):
            call(**kw)

"""A teacher whose logits are broken: what a NaN or +infinity among a token's entries reaches, and what it does not."""
import pytest
import torch

import vocabulary_reference as ref
from test_gpu_distillation import backward, forward, teacher

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")

# what the entries of a token hold: the first ones, then (None) its finite logits, or -infinity, or no entries
BROKEN = {
    "a NaN beside finite logits": ([NAN], None),
    "+infinity beside finite logits": ([INF], None),
    "a NaN beside -infinity": ([NAN], -INF),
    "+infinity beside -infinity": ([INF], -INF),
    "a NaN alone": ([NAN], "none"),
    "+infinity alone": ([INF], "none"),
    "NaN everywhere": ([NAN], NAN),
    "both": ([NAN, INF], None),
}


@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind", BROKEN)
def test_a_broken_teacher_shows(kind, bf16):
    """The softmax over entries of which one is NaN or +infinity is NaN: so are the token's loss, its row of dx and the rows
    of de that its entries name.  Everything else has the bits of the call with a sound teacher."""
    M, V, K, k, T, m = 9, 700, 64, 70, 1.5, 4
    ops = ref.head(M, V, K, seed=21)[:4]
    ids, top = teacher(M, V, k, seed=21, padded=False)
    ids[m, 66] = ids[m, 2]                     # an id twice, in two entries of the wave's lanes
    first, rest = BROKEN[kind]
    if rest == "none":
        ids[m, len(first):] = -1
    bad = top.clone()
    if isinstance(rest, float):
        bad[m] = rest
    for at, value in zip((2, 67), first):
        bad[m, 0 if rest == "none" else at] = value
    dloss = torch.rand(M, device="cuda") + 0.5
    sound, broken = [], []
    for logits, out in ((top, sound), (bad, broken)):
        loss, lse, logp = forward(ops, ids, logits, T)
        out += [loss, lse, logp, *backward(ops, ids, logits, T, lse, logp, dloss, bf16)]
    assert all(bool(torch.isfinite(t).all()) for t in sound)
    others = torch.arange(M, device="cuda") != m
    named = torch.zeros(V, dtype=torch.bool, device="cuda")
    named[ids[m][ids[m] >= 0].long()] = True
    loss, lse, logp, dx, de = broken
    assert not bool(torch.isfinite(loss[m])), float(loss[m])
    assert torch.equal(loss[others], sound[0][others])
    assert torch.equal(lse, sound[1]) and torch.equal(logp, sound[2])     # (the student's alone)
    assert not bool(torch.isfinite(dx[m]).any())
    assert torch.equal(dx[others], sound[3][others])
    assert not bool(torch.isfinite(de[named]).any())
    assert torch.equal(de[~named], sound[4][~named])


def test_what_is_no_entry_may_be_broken():
    """NaN and infinities where the id is none, and -infinity where it is one, change nothing."""
    M, V, K, k, T = 6, 300, 32, 12, 1.0
    ops = ref.head(M, V, K, seed=22)[:4]
    ids, top = teacher(M, V, k, seed=22, padded=False)
    ids[:, 5:8] = torch.tensor([-1, V, -100], dtype=torch.int32, device="cuda")
    ids[3] = -1
    top[4, 9] = -INF
    other = top.clone()
    other[:, 5:8] = torch.tensor([NAN, INF, -INF], device="cuda")
    other[3] = NAN
    dloss = torch.ones(M, device="cuda")
    outs = []
    for logits in (top, other):
        loss, lse, logp = forward(ops, ids, logits, T)
        outs.append([loss, lse, logp, *backward(ops, ids, logits, T, lse, logp, dloss, False)])
    for a, b in zip(*outs):
        assert bool(torch.isfinite(a).all()) and torch.equal(a, b)
    assert float(outs[0][0][3]) == 0.0 and bool((outs[0][3][3] == 0).all())

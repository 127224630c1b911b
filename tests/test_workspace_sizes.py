"""The workspace queries never fall as a size grows: what a program allocates for its longest batch serves every shorter
one.  (On the CPU: the queries, and calls refused for one byte less.)"""
import random

import pytest

A = 0x10000


def _q(name, *args):
    from bit_scaffold_int8_amd import dfssm
    return dfssm.raw(name, *args)


def _lengths(rng, most):
    """Lengths around where plans change, and random ones, in order."""
    out = {1, most}
    for p in (16, 32, 64, 96, 128, 192, 256, 300, 512, 1024, 1500, 2048, 3000, 4096, 5400, 8192, 11100, 16384, 20300, 23900,
              32768, 65536, 131072, 262144, 1 << 20, 1 << 22, 1 << 24):
        out.update((p - 1, p, p + 1))
    out.update(int(2 ** rng.uniform(0, 24)) for _ in range(400))
    return sorted(n for n in out if 1 <= n <= most)


MATRICES = [(50280, 2048), (11898, 2480), (1000, 64), (300, 512), (310, 16), (1, 16), (60001, 4096), (1 << 18, 16),
            (33, 131072)]


@pytest.mark.parametrize("V,K", MATRICES)
def test_cross_entropy_sizes_do_not_fall(V, K):
    rng = random.Random(V)
    last = 0
    for M in _lengths(rng, min(1 << 24, (1 << 38) // V)):
        n = _q("dfssm_cross_entropy_workspace_bytes", M, V, K)
        assert n >= last > -1 and n >= M * 8
        last = n
    for t in (0, 1):
        for dx, de in ((1, 1), (1, 0), (0, 1)):
            last = 0
            for M in _lengths(rng, 1 << 18):
                n = _q("dfssm_cross_entropy_backward_workspace_bytes", M, V, K, t, dx, de)
                assert n >= last and n > 0, (M, t, dx, de)
                last = n
                # one gradient takes no more than both, bf16 no more than fp32
                assert n <= _q("dfssm_cross_entropy_backward_workspace_bytes", M, V, K, 0, 1, 1)


@pytest.mark.parametrize("M", [1, 5, 65, 300, 1500, 2048, 8192, 100000])
def test_cross_entropy_sizes_do_not_fall_with_the_matrix(M):
    for Ks, V in ((range(16, 4096, 208), 50280), (range(16, 300, 16), 700)):
        last = [0] * 3
        for K in Ks:
            n = [_q("dfssm_cross_entropy_workspace_bytes", M, V, K)]
            n += [_q("dfssm_cross_entropy_backward_workspace_bytes", M, V, K, 0, 1, de) for de in (0, 1)]
            assert all(a >= b for a, b in zip(n, last)), (V, K)
            last = n
    last = [0] * 3
    for V in sorted(set(list(range(1, 700, 31)) + [1000, 1024, 8192, 11898, 20001, 50280, 60001, 100000, 1 << 18])):
        n = [_q("dfssm_cross_entropy_workspace_bytes", M, V, 2048)]
        n += [_q("dfssm_cross_entropy_backward_workspace_bytes", M, V, 2048, 0, 1, de) for de in (0, 1)]
        assert all(a >= b for a, b in zip(n, last)), V
        last = n


@pytest.mark.parametrize("V,K", MATRICES)
def test_embedding_sizes_do_not_fall(V, K):
    rng = random.Random(K)
    last = 0
    for T in _lengths(rng, 1 << 24):
        n = _q("dfssm_embedding_backward_workspace_bytes", T, V, K)
        assert n >= last and n >= T * 16
        last = n


def test_the_longest_batch_size_serves_shorter_ones():
    """A call checks the size of its own query: what a longer batch's query gave is enough."""
    def refused(M, n):
        return _q("dfssm_cross_entropy", A, A, M, 50280, 2048, A, A, A, A, A, A, n, None) == 1
    for short, long in ((1500, 2048), (65, 128), (8192, 8193)):
        own = _q("dfssm_cross_entropy_workspace_bytes", short, 50280, 2048)
        assert refused(short, own - 1)
        assert _q("dfssm_cross_entropy_workspace_bytes", long, 50280, 2048) >= own
        n = _q("dfssm_embedding_backward_workspace_bytes", short, 50280, 2048)
        assert _q("dfssm_embedding_backward", A, short, A, 2048, 0, 50280, 2048, 1.0, A, 0, 0, A, n - 1, None) == 1
        assert _q("dfssm_embedding_backward_workspace_bytes", long, 50280, 2048) >= n

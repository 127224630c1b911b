"""The scan's workspace queries (on the CPU): small calls take little, and no size falls as another argument grows."""
import random


def _queries():
    from bit_scaffold_int8_amd import dfssm
    return dfssm.dfssm_mamba2_scan_workspace_bytes, dfssm.dfssm_mamba2_scan_backward_workspace_bytes


def test_small_calls_take_little():
    """Forward: per chunk its products, pieces (160 KB a group) and decays (1792 bytes a head), and a state (32 KB a head) for each
    possible segment, of which there are at most a chunk's and a sequence's.  Backward: one more set of pieces (48 KB), two states
    and 64 KB of shares a chunk and head."""
    forward, backward = _queries()
    for T, S, H, G in ((1, 1, 1, 1), (1, 1, 64, 1), (64, 1, 1, 1), (300, 3, 3, 1), (64, 64, 8, 2), (1000, 1, 24, 1)):
        chunks = T // 64 + S
        most = chunks * (G * 160 * 1024 + H * 1792 + 32) + (chunks + S) * H * (32768 + 4) + 4096
        assert 0 < forward(T, S, H, 64, 128, G) <= most + 16 * (S + 1) + chunks * 32
        more = chunks * (G * 48 * 1024 + H * (2 * 32768 + 65536 + 16))
        assert forward(T, S, H, 64, 128, G) < backward(T, S, H, 64, 128, G) <= most + more + 16 * (S + 1) + chunks * 32 + 4096


def test_sizes_do_not_fall():
    rng = random.Random(5)
    for _ in range(3000):
        T, S, H, G = (int(2 ** rng.uniform(0, top)) for top in (14, 8, 7, 2))
        H *= G
        for query in _queries():
            n = query(T, S, H, 64, 64, G)
            assert n > 0
            assert query(T, S, H, 64, 128, G) >= n
            assert query(T + rng.randrange(1, 200), S, H, 64, 64, G) >= n
            assert query(T, S + rng.randrange(1, 20), H, 64, 64, G) >= n
            assert query(T, S, H + G * rng.randrange(1, 9), 64, 64, G) >= n
            assert query(T, S, 2 * H, 64, 64, 2 * G) >= n

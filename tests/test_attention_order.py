"""The waits of the tensor-core attention forward end, for every group size, window, sink count and split."""
import pytest

from attention_order import blocks, completes

SIZES = [(256, 256), (512, 512), (700, 700), (1100, 1100), (300, 1000), (129, 4000)]
WINDOWS = [0, 1, 64, 65, 100, 128, 129, 191, 193, 300, 512]


@pytest.mark.parametrize("G", [1, 2, 3, 4, 7, 16, 64])
@pytest.mark.parametrize("nq,kv", SIZES)
def test_every_block_ends(G, nq, kv):
    tried = set()
    for window in WINDOWS:
        for sinks in (0, 4, 65, 300) if window else (0,):
            for paged, splits in ((False, 1), (True, 1), (True, 2), (True, 5)):
                for n, act, ntiles in blocks(nq, kv, G, window, sinks, splits):
                    case = n, tuple(map(tuple, act)), ntiles, paged
                    if case not in tried:
                        tried.add(case)
                        assert completes(n, act, ntiles, paged, True), (window, sinks, splits, n, act)


@pytest.mark.parametrize("nq,kv,window,sinks", [(512, 512, 100, 0), (2048, 2048, 512, 4), (300, 1000, 150, 4)])
def test_a_wait_for_both_tiles_would_not(nq, kv, window, sinks):
    """With one query head per key/value head the second tile's window starts two steps behind the first's. A row
    of it that waits for the ring's unit, which the first tile's issuer lets go of two steps later, holds the
    turn that this issuer's rows are waiting for."""
    stuck = [not completes(n, act, t, False, False) for n, act, t in blocks(nq, kv, 1, window, sinks)]
    assert any(stuck)
    for G in (2, 4):
        assert all(completes(n, act, t, False, False) for n, act, t in blocks(nq, kv, G, window, sinks))
    assert all(completes(n, act, t, False, False) for n, act, t in blocks(nq, kv, 1, nq + kv, sinks))

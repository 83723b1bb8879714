"""The shapes of tile_cases.py reach every kernel of the 8-bit products, plain and gated, with more than
twice as many steps as its ring has stages: each buffer is refilled and read again at least once.
A change of the table that chooses the tile fails here where it takes that away."""
import pytest

import tile_cases as tc


@pytest.mark.parametrize("gated,cases", [(False, tc.PLAIN), (True, tc.GATED)])
def test_every_ring_wraps_twice(gated, cases):
    assert len(tc.KERNELS) == len(tc.TILES) and all(k[:2] == t[:2] for k, t in zip(tc.KERNELS, tc.TILES))
    wanted = {("few", tt) for tt in (1, 2, 3, 4)} | {("tile", i) for i in range(len(tc.TILES))}
    seen = {}
    for T, N, K, bf16, pieces in cases:
        kernel, steps, stages = tc.kernel_of(T, N, K, gated)
        assert steps >= 2 * stages + 1, (T, N, K, kernel, steps, stages)
        seen.setdefault(kernel, set()).add((bf16, pieces))
    assert set(seen) == wanted, wanted - set(seen)
    # both output types of each tile, and rows stored in pieces and by elements
    for kernel, ways in seen.items():
        if kernel[0] == "tile":
            assert {b for b, _ in ways} == {p for _, p in ways} == {False, True}, (kernel, ways)

"""Every tile of the bfloat16 products has a shape in bf16_cases.py that reaches it and runs its ring of stages around
twice.  A change of a table fails here where it takes that away."""
import pytest

import bf16_cases as bc


@pytest.mark.parametrize("kind,adapters", [("MAT_NT", False), ("MAT_NT", True), ("MAT_GATED", False), ("MAT_GATED", True),
                                           ("MAT_NN", False), ("MAT_TN", False)])
def test_every_tile_has_a_shape(kind, adapters):
    tiles = bc.TILES[kind][:11] if adapters else bc.TILES[kind]
    assert len(bc.RINGS) == 12 and len(tiles) == (11 if adapters else 12)
    built = {i for i, t in enumerate(tiles) if t[2] < 9}     # (a row of nines: not built for this kind)
    assert len(built) >= len(tiles) - 1 and set(bc.shapes(kind, adapters)) == built


def test_every_pair_has_a_shape():
    assert set(bc.pair_shapes()) == {-1} | {i for i, _ in bc.PAIR}

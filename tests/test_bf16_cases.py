"""Every tile of the bfloat16 products has a shape in bf16_cases.py that reaches it and runs its ring of stages around
twice.  A change of a table fails here where it takes that away."""
import pytest

import bf16_cases as bc


@pytest.mark.parametrize("kind,adapters", [("MAT_NT", False), ("MAT_NT", True), ("MAT_GATED", False), ("MAT_GATED", True),
                                           ("MAT_NN", False), ("MAT_TN", False)])
def test_every_tile_has_a_shape(kind, adapters):
    tiles = bc.TILES[kind][:9] if adapters else bc.TILES[kind]
    assert len(bc.RINGS) == 10 and len(tiles) == (9 if adapters or kind == "MAT_GATED" else 10)
    assert set(bc.shapes(kind, adapters)) == set(range(len(tiles)))


def test_every_pair_has_a_shape():
    assert set(bc.pair_shapes()) == {-1} | {i for i, _ in bc.PAIR}

"""The sizes that send blocks of the bf16 expert products through several tiles do so,
for each tile that the products choose from."""
import pytest

import _grouped_rule as rule


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("name,counts,N", rule.ROUNDS, ids=[r[0] for r in rule.ROUNDS])
def test_blocks_take_several_tiles(name, counts, N, trans):
    taken, tiles, slots = rule.choice(counts, N, trans)
    assert taken == name and tiles > 1.5 * slots
    assert min(counts) == 0 and sum(counts) % 2 == 0


def test_every_tile_is_covered():
    assert {r[0] for r in rule.ROUNDS} == set(rule.tiles()[0])


def test_the_measured_choices():
    """Choices of the tables beside the rule: rows per expert, even."""
    def even(rows, E, N, trans):
        return rule.choice([rows] * E, N, trans)[0]
    assert even(1, 128, 1536, False) == even(8, 128, 1536, False) == "rows"
    assert even(16, 128, 1536, False) == even(8, 128, 768, True) == "Low"
    assert even(32, 128, 1536, False) == "Half"
    assert even(150, 128, 1536, False) == "Wide"
    assert even(150, 128, 768, True) == "Broad"
    assert rule.choice([256] * 8, 1536, False)[0] == "Half"  # (few tiles)

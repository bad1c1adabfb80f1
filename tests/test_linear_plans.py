"""flux_linear's choice of kernel, form and tile, on the CPU."""
import itertools

from tests.linear_plans import PAIR_X, plans


def test_every_size_has_a_plan():
    """Also where the tokens of many batch elements, which do not follow one
    another and are rounded up one by one, are too many columns for the forms
    with W's rows as tiles, and too few to fill tiles of token rows."""
    few = [(B, S, K, N, dict(act=act)) for (B, S), K, N, act in itertools.product(
        [(20, 3), (31, 2), (17, 2), (32, 2), (63, 1), (9, 7), (100, 2), (1, 1), (4, 16), (8, 8),
         (5, 9), (2, 31), (60, 1), (3000, 1), (300, 300)], (8, 64, 4096), (8, 4096),
        (None, "swiglu"))]
    for problem, plan in zip(few, plans(few)):
        assert 1e3 < plan.ns < 1e9, (problem, plan)
        assert plan.tile >= 16 and plan.parts >= 1, (problem, plan)
    assert plans([(20, 3, 4096, 4096, {})])[0].form == PAIR_X

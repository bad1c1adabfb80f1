"""flux_linear's choice of kernel, form and tile, on the CPU."""
import itertools

from tests import linear_cases as C
from tests.linear_plans import PAIR_W, PAIR_X, SINGLE, plans


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


def _problem(case):
    kw = dict(case[-1], residual=True)
    return (*((1,) if len(case) == 4 else ()), *case[:-1], kw)


def test_the_gpu_cases_take_the_classes_they_name():
    cases = C.CLASSES + C.WIDE_VIEWS
    for (want, case), plan in zip(cases, plans([_problem(c) for _, c in cases])):
        assert C.class_of(plan) == want, (case, plan)


def test_the_gpu_cases_take_every_class():
    """Every kernel that is compiled, and every tile width of linear_pair, with and
    without SwiGLU."""
    want = {("split", SINGLE, c, glu) for c in (1, 2, 3, 4, 6, 8) for glu in (False, True)}
    want |= {("split", form, c, glu) for form in (PAIR_W, PAIR_X) for c in (1, 2, 3, 4)
             for glu in (False, True)}
    want |= {("pair", 0, tn, False) for tn in range(32, 257, 32)}
    want |= {("pair", 0, tn, True) for tn in range(64, 257, 64)}
    have = {(*cls, case[-1].get("act") == "swiglu") for cls, case in C.CLASSES}
    assert have == want

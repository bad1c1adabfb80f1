"""The choice of kernel, form and tile of flux_linear_fp8 and
flux_cross_attention, on the CPU."""
import itertools

from tests import operator_cases as C
from tests import operator_plans as P


def test_every_size_has_a_plan():
    few = [P.linear(B, S, K, N, act) for (B, S), K, N, act in itertools.product(
        [(1, 1), (20, 3), (63, 1), (3, 100), (300, 300), (2, 4097), (1, 1 << 20)],
        (16, 128, 4096, 1 << 22), (128, 4096, 1 << 20), (None, "swiglu"))]
    few += [P.linear(1, 5, 144, 8), P.linear(2, 700, 16, 40)]
    for line, (form, tile, parts, ns) in zip(few, P.plans(few)):
        assert 1e3 < ns < 1e13 and tile >= 16 and 1 <= parts <= 8, line
    few = [P.cross(B, Sq, Sk, H, Hk, D) for B, Sq, Sk, (H, Hk), D in itertools.product(
        (1, 3), (1, 130, 70000), (1, 129, 70000), ((1, 1), (128, 1), (6, 2), (48, 48)), (64, 128))]
    for line, (form, parts, _, ns) in zip(few, P.plans(few)):
        assert 1e3 < ns < 1e11 and (form == "wide" or 1 <= parts <= 16), line


def test_the_gpu_cases_take_every_form_and_tile():
    for cases, act in ((C.LINEAR, None), (C.GLU, "swiglu")):
        lines = [P.linear(*c[:4], act=c[4].get("act", act), residual=c[4].get("residual", False))
                 for c in cases.values()]
        assert [p[:2] for p in P.plans(lines)] == list(cases)
    assert {t for f, t in C.LINEAR if f == "split"} == {16, 32, 64, 96, 128}
    assert {t for f, t in C.LINEAR if f == "pair"} == {64, 128, 192, 256}
    got = P.plans([P.cross(*c) for c in C.CROSS.values()])
    assert [p[:2] for p in got] == list(C.CROSS)

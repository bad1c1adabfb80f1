"""Problems for binding.linear that between them take every kernel, form, split of
the channels and tile width that the plan has; tests/test_linear_plans.py checks
on the CPU that they still do, so that new constants of the plan cannot move the
GPU tests off a kernel unseen."""
from tests.linear_plans import PAIR_W, PAIR_X, SINGLE

GLU = dict(act="swiglu")

# (kernel, form, tile of linear_pair or parts of linear_split) and a problem
# (S, K, N, kw) of one batch element with bias, gate and residual. Ragged channels
# (no multiple of 64) and features (no multiple of 32) wherever they fit.
CLASSES = [
    (("split", SINGLE, 1), (10, 72, 9912, {})),
    (("split", SINGLE, 2), (23, 72, 296, {})),
    (("split", SINGLE, 3), (10, 88, 304, dict(K2=16))),
    (("split", SINGLE, 4), (61, 80, 280, dict(K2=80, act="silu"))),
    (("split", SINGLE, 6), (10, 328, 280, {})),
    (("split", SINGLE, 8), (39, 472, 304, dict(act="gelu_tanh"))),
    (("split", SINGLE, 1), (10, 80, 5088, GLU)),
    (("split", SINGLE, 2), (33, 72, 280, GLU)),
    (("split", SINGLE, 3), (10, 88, 312, dict(GLU, K2=16))),
    (("split", SINGLE, 4), (10, 152, 288, dict(GLU, K2=8))),
    (("split", SINGLE, 6), (17, 336, 312, GLU)),
    (("split", SINGLE, 8), (10, 184, 288, dict(GLU, K2=312))),
    (("split", PAIR_W, 1), (77, 72, 9616, {})),
    (("split", PAIR_W, 2), (71, 72, 5024, dict(act="silu"))),
    (("split", PAIR_W, 3), (112, 72, 5272, dict(K2=8))),
    (("split", PAIR_W, 4), (68, 136, 1512, dict(K2=136))),
    (("split", PAIR_W, 1), (66, 72, 2808, GLU)),
    (("split", PAIR_W, 2), (66, 200, 2712, GLU)),
    (("split", PAIR_W, 3), (77, 80, 2664, dict(GLU, K2=8))),
    (("split", PAIR_W, 4), (69, 416, 496, GLU)),
    (("split", PAIR_X, 1), (268, 440, 9480, dict(K2=24))),
    (("split", PAIR_X, 2), (265, 776, 1432, {})),
    (("split", PAIR_X, 3), (272, 560, 280, dict(act="gelu_tanh"))),
    (("split", PAIR_X, 4), (261, 136, 360, dict(K2=424))),
    (("split", PAIR_X, 1), (262, 72, 1456, GLU)),
    (("split", PAIR_X, 2), (289, 288, 280, dict(GLU, K2=64))),
    (("split", PAIR_X, 3), (280, 80, 296, dict(GLU, K2=240))),
    (("split", PAIR_X, 4), (287, 144, 304, dict(GLU, K2=224))),
    (("pair", 0, 32), (135, 72, 72, dict(K2=256))),
    (("pair", 0, 64), (129, 272, 2616, dict(K2=40, act="silu"))),
    (("pair", 0, 96), (137, 208, 5288, {})),
    (("pair", 0, 128), (2180, 344, 3080, {})),
    (("pair", 0, 160), (4408, 304, 1800, {})),
    (("pair", 0, 192), (4868, 328, 1848, dict(act="gelu_tanh"))),
    (("pair", 0, 224), (2580, 304, 3976, {})),
    (("pair", 0, 256), (3208, 224, 4024, dict(K2=80))),
    (("pair", 0, 64), (291, 304, 184, GLU)),
    (("pair", 0, 128), (1298, 328, 2416, GLU)),
    (("pair", 0, 192), (1284, 152, 3248, dict(GLU, K2=176))),
    (("pair", 0, 256), (1577, 328, 3096, GLU)),
]

# Batch elements that do not follow one another, in place, at wide tiles of
# linear_pair: (kernel, form, tile) and (B, S, K, N, kw).
WIDE_VIEWS = [
    (("pair", 0, 224), (2, 2305, 520, 4104, dict(K2=136))),
    (("pair", 0, 256), (3, 1100, 264, 3096, GLU)),
]

# Products of the FLUX.2 workloads' blocks, compared at sampled rows: (B, S, K, N, kw).
WORKLOADS = {
    "modulation": (2, 1, 4096, 24576, dict(bias=True)),
    "text attention out": (1, 512, 4096, 4096, dict(gate=True, residual=True)),
    "text feed-forward in": (1, 512, 4096, 12288, GLU),
    "text feed-forward out": (2, 77, 12288, 4096, dict(gate=True, residual=True)),
    "image attention out, 1200 tokens": (1, 1200, 4096, 4096, dict(gate=True, residual=True)),
    "image attention out": (1, 4096, 4096, 4096, dict(gate=True, residual=True)),
    "image feed-forward in": (1, 4096, 4096, 12288, GLU),
    "image feed-forward out": (1, 4096, 12288, 4096, dict(gate=True, residual=True)),
    "single-stream out": (1, 4608, 4096, 4096, dict(K2=12288, gate=True, residual=True)),
    "final projection": (1, 4056, 4096, 128, dict(bias=True)),
}


def class_of(plan):
    return (plan.kernel, plan.form, plan.tile if plan.kernel == "pair" else plan.parts)

"""Problems of flux_linear_fp8 that take every kernel and tile that its plan has,
and of flux_cross_attention for every form: tests/test_operator_plans.py checks on
the CPU that they still do, the GPU tests run them."""

# (form, tile): (B, S, K, N, options)
LINEAR = {
    ("split", 16): (1, 3, 2048, 512, dict(bias=True, gate=True, residual=True)),
    ("split", 32): (1, 30, 4096, 24576, dict(bias=True)),
    ("split", 64): (1, 61, 4096, 8192, dict(gate=True, residual=True)),
    ("split", 96): (1, 90, 4096, 8192, dict(bias=True, act="silu")),
    ("split", 128): (1, 120, 8192, 4096, dict(bias=True, gate=True, residual=True)),
    ("pair", 64): (1, 500, 512, 2048, dict(bias=True, residual=True)),
    ("pair", 128): (1, 500, 2048, 4096, dict(bias=True, gate=True, residual=True)),
    ("pair", 192): (1, 1200, 512, 4096, dict(gate=True, residual=True)),
    ("pair", 256): (1, 2304, 1024, 4096, dict(bias=True, gate=True, residual=True)),
}
GLU = {
    ("split", 16): (1, 3, 2048, 512, dict(bias=True, gate=True, residual=True)),
    ("split", 32): (1, 30, 4096, 12288, dict(bias=True)),
    ("split", 64): (1, 61, 4096, 4096, dict(gate=True, residual=True)),
    ("split", 96): (1, 90, 4096, 4096, dict(bias=True)),
    ("split", 128): (3, 195, 12032, 512, dict(residual=True)),
    ("pair", 128): (1, 500, 2048, 2048, dict(bias=True, gate=True, residual=True)),
    ("pair", 256): (1, 2304, 512, 2048, dict(bias=True, gate=True, residual=True)),
}
# (form, parts): (B, Sq, Sk, H, Hk, D)
CROSS = {
    ("narrow", 1): (2, 40, 100, 8, 8, 128),
    ("narrow", 2): (2, 73, 1950, 32, 32, 64),
    ("narrow", 4): (1, 5, 1750, 16, 16, 128),
    ("narrow", 8): (1, 39, 1155, 16, 8, 128),
    ("narrow", 12): (1, 7, 6000, 24, 8, 128),
    ("narrow", 16): (1, 2, 5000, 8, 2, 64),
    ("wide", 1): (1, 3000, 300, 16, 8, 128),
}

"""Shapes of grouped products, each with the form that it is there to reach (tests/test_moe_cpu.py asks the
selection about every one): rows, groups, outputs, K, activations, form."""

_BOTH = [
    (5, 8, 333, 416, "few 16 x 2"), (16, 64, 4100, 160, "few 16 x 2"), (8, 3, 40, 4128, "few 16 x 2"),
    (40, 6, 333, 1184, "few 16 x 2"), (100, 10, 72, 96, "few 16 x 2"), (500, 3, 333, 352, "few 16 x 2"),
    (200, 33, 1000, 288, "few 16 x 2"), (600, 6, 200, 1184, "few 16 x 2"),
    (333, 4, 1001, 2080, "64"), (100, 8, 2050, 544, "64"), (900, 5, 1000, 416, "64"), (50, 3, 4112, 1024, "64"),
    (2000, 6, 2054, 800, "128"), (2000, 4, 1030, 4128, "128"), (2100, 3, 4100, 1056, "128"),
    (4096, 2, 8196, 1184, "256"), (3000, 3, 8209, 800, "256"), (4096, 4, 4100, 1184, "256"), (2500, 3, 8192, 1024, "256"),
    (3500, 3, 8200, 416, "256"),
]
GROUPED = [(M, E, N, K, fmt, form) for M, E, N, K, form in _BOTH for fmt in ("fp8", "fp4")]

"""Shapes of products with an epilogue whose result is quantized (whole blocks of 32 outputs), each with the form of
the product that it is there to reach (tests/test_linear_forms_cpu.py asks the selection about every one).  The kernel
for few tokens then takes two tiles of 16 outputs, and 32 LDS rows for 24."""

_BOTH = [
    (1, 352, 4128, "few 4 x 1"), (4, 8224, 160, "few 4 x 1"),
    (7, 2048, 1184, "few 16 x 1"), (16, 4096, 2080, "few 16 x 1"),
    (5, 8224, 544, "few 16 x 2"), (16, 4128, 4640, "few 16 x 2"),
    (30, 320, 416, "few 32 x 1"), (64, 96, 352, "few 32 x 1"),
    (40, 4128, 352, "few 32 x 2"), (1000, 2080, 288, "few 32 x 2"),
    (130, 544, 1024, "64, 3 slots"), (513, 992, 1184, "64, 3 slots"),
    (333, 992, 2080, "64, 6 slots"), (65, 64, 2080, "64, 6 slots"),
    (200, 544, 4096, "64, ranges, 3 slots"), (130, 64, 4640, "64, ranges, 3 slots"),
    (512, 992, 12288, "64, ranges, 6 slots"),
    (1500, 2080, 544, "128"), (333, 12256, 768, "128"),
    (200, 2080, 12288, "128, ranges"), (513, 992, 12256, "128, ranges"),
    # rows and outputs that fill no tile; more than 256 tiles, so that a persistent block has several
    (1024, 16032, 768, "largest"), (1500, 8224, 1184, "largest"), (2100, 12256, 1088, "largest"),
    (4000, 16032, 416, "largest"),
]
QUANTIZED = [(M, N, K, fmt, form) for M, N, K, form in _BOTH for fmt in ("fp8", "fp4")]
QUANTIZED += [(20, 512, 1184, "fp8", "few 24 x 1"), (24, 4096, 4128, "fp8", "few 24 x 1")]

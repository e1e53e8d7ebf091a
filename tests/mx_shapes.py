"""Shapes of microscaled products, each with the form that it is there to reach.  The
selection refuses nothing, so a change of its estimates could move a shape to another
form: tests/test_mx_tiling_cpu.py asks it about every one of them."""

# kind, then LDS rows and 16-output tiles (few tokens) or more than one K range and LDS slots (tiles of 64)
FORMS = {
    "few 4 x 1": ("few", 4, 1), "few 16 x 1": ("few", 16, 1), "few 16 x 2": ("few", 16, 2),
    "few 24 x 1": ("few", 24, 1), "few 32 x 1": ("few", 32, 1), "few 32 x 2": ("few", 32, 2),
    "64, 3 slots": ("tile 64", False, 3), "64, 6 slots": ("tile 64", False, 6),
    "64, ranges, 3 slots": ("tile 64", True, 3), "64, ranges, 6 slots": ("tile 64", True, 6),
    "128": ("tile 128", False, 0), "128, ranges": ("tile 128", True, 0), "largest": ("largest", False, 0),
}

_BOTH = [
    (1, 333, 4128, "few 4 x 1"), (4, 8208, 160, "few 4 x 1"),
    (7, 2050, 1184, "few 16 x 1"), (16, 4096, 2080, "few 16 x 1"),
    (5, 8209, 544, "few 16 x 2"), (16, 4112, 4640, "few 16 x 2"),
    (30, 333, 416, "few 32 x 1"), (64, 72, 352, "few 32 x 1"),
    (40, 4099, 352, "few 32 x 2"), (300, 4096, 96, "few 32 x 2"), (1000, 2050, 288, "few 32 x 2"),
    (100, 333, 384, "64, 3 slots"), (130, 520, 1024, "64, 3 slots"), (513, 1001, 1184, "64, 3 slots"),
    (65, 48, 2080, "64, 6 slots"), (333, 1000, 2080, "64, 6 slots"), (257, 520, 2176, "64, 6 slots"),
    (200, 520, 4096, "64, ranges, 3 slots"), (130, 49, 4640, "64, ranges, 3 slots"),
    (100, 333, 12288, "64, ranges, 6 slots"), (512, 1000, 12288, "64, ranges, 6 slots"),
    (1500, 2051, 544, "128"), (1024, 4096, 1024, "128"), (333, 12250, 768, "128"),
    (200, 2050, 12288, "128, ranges"), (513, 1001, 12256, "128, ranges"), (512, 4096, 12288, "128, ranges"),
    (1024, 16001, 768, "largest"), (4096, 4096, 1024, "largest"), (1500, 8209, 1184, "largest"),
    (4000, 16001, 416, "largest"), (2100, 12250, 1088, "largest"),
]
PRODUCTS = [(M, N, K, fmt, form) for M, N, K, form in _BOTH for fmt in ("fp8", "fp4")]
PRODUCTS += [(20, 520, 1184, "fp8", "few 24 x 1"), (24, 4096, 4128, "fp8", "few 24 x 1"),
             (17, 49, 352, "fp8", "few 24 x 1"),
             (4096, 16001, 512, "fp4", "largest"), (1024, 16001, 2048, "fp4", "largest")]

# products run side by side: kind, more than one K range
REACHED = [(200, 520, 4096, "fp8", ("tile 64", True)), (200, 2050, 12288, "fp8", ("tile 128", True)),
           (1024, 16001, 768, "fp8", ("largest", False)), (1024, 16001, 768, "fp4", ("largest", False)),
           (200, 520, 4640, "fp8", ("tile 64", True)), (200, 520, 4640, "fp4", ("tile 64", True))]

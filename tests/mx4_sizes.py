"""Sizes at which the 4-bit product takes each of its kernels, odd in every direction. The host test
asks the plan (csrc/sffn_mx4_host.h) that they do, the GPU test runs them."""

# (kernel of the first channels, kernel of the rest or None, M, K, N)
FORMS = [
    ("Few", None, 3, 1000, 333),
    ("Short", None, 39, 347, 3471),
    ("Split16", None, 21, 3561, 333),
    ("Split16x32", None, 61, 3561, 3001),
    ("Split32", None, 11, 1001, 8599),
    ("Split64", None, 61, 1543, 9001),
    ("Tile64", None, 67, 1223, 16517),
    ("Tile64x128", None, 1001, 2001, 3333),
    ("Tile128", None, 201, 711, 16717),
    ("Tile256", None, 391, 455, 18985),
    ("Tile256", "Split16", 1919, 219, 16437),
    ("Tile256", "Split32", 3741, 295, 4461),
    ("Tile256", "Split64", 4292, 449, 3991),
    ("Tile256", "Tile64", 842, 300, 19141),
    ("Tile256", "Tile128", 1345, 227, 14868),
]

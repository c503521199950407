"""Shapes of the unquantised products that reach the kernels for large batches, each with the
kernel that the library takes for it.  test_matmul_choice.py holds the library to that
on the CPU, test_gpu_matmul_tiles.py runs them, so a change of the rule cannot move a kernel
out of the tests unseen.

A kernel is (name, mt, nt, splits) as the rule has it: tiles of 32 mt rows of x by 32 nt rows of
w; "any" is the 64 x 64 tile for rows at any address."""

BIG, MIDDLE, ANY = ("tile", 8, 8, 1), ("tile", 4, 4, 1), ("any", 2, 2, 1)

# dtype, gated, rows, K, N, kernel.  Ends inside a row tile, a column tile and a step (K not a
# multiple of 64 16-bit or 32 fp32 inputs), odd and even counts of whole steps.
DENSE = [
    ("bf16", False, 4090, 576, 4000, BIG),
    ("fp16", False, 3900, 4160, 4000, BIG),
    ("bf16", False, 8000, 1032, 2000, BIG),
    ("fp16", False, 9001, 4168, 1000, BIG),
    ("bf16", True, 4090, 320, 2000, BIG),
    ("fp16", True, 2990, 2112, 2000, BIG),
    ("bf16", True, 8000, 264, 1000, BIG),
    ("bf16", False, 4100, 576, 4104, MIDDLE),
    ("fp16", True, 4100, 584, 2056, MIDDLE),
    ("fp32", False, 2048, 2048, 2048, MIDDLE),
    ("fp32", False, 2001, 1004, 2000, MIDDLE),
    ("fp32", False, 4090, 2016, 1000, MIDDLE),
    ("fp32", True, 2001, 1000, 1000, MIDDLE),
    ("fp32", True, 2048, 1004, 1001, MIDDLE),
    ("fp32", False, 2001, 2047, 2048, ANY),
    ("fp32", True, 1001, 1003, 1000, ANY),
    ("bf16", False, 4096, 1003, 1357, ANY),
    ("fp16", True, 2049, 515, 1357, ANY),
]

# dtype, out dtype, gated, experts, tokens, top_k, K, N, kernel
GROUPED = [
    ("bf16", "bf16", False, 3, 3050, 2, 576, 2000, BIG),
    ("fp16", "fp16", False, 3, 3050, 2, 2120, 2000, BIG),
    ("bf16", "bf16", True, 3, 3050, 2, 320, 1000, BIG),
    ("fp16", "fp16", True, 4, 8000, 1, 2112, 500, BIG),
    ("bf16", "fp32", True, 3, 3000, 2, 520, 1000, BIG),
    ("bf16", "fp32", False, 4, 16000, 4, 1032, 1024, BIG),
    ("fp32", "fp32", False, 8, 6000, 2, 520, 500, MIDDLE),
    ("fp32", "bf16", True, 8, 4001, 3, 516, 500, MIDDLE),
    ("fp32", "fp32", False, 4, 3000, 1, 1003, 1000, ANY),
    ("bf16", "bf16", True, 4, 1500, 2, 1003, 1000, ANY),
]

# Rows far apart, as the packed shapes have them: rows, K, N, elements between the rows
# (bf16), kernel.  A tile's rows of x or of w reach to the last offset below 4 GiB.
FAR_X = (512, 576, 60000, (1 << 23) - 8, BIG)
FAR_W = (60000, 576, 512, (1 << 23) - 8, BIG)
# experts, slots, K, N, elements between the rows of x: gathered rows just below 4 GiB
FAR_GATHERED = [(3, 6000, 576, 2000, 357904, BIG), (2, 511, 576, 200, 1 << 22, ("deep", 1, 2, 1))]

# Few tiles over a long K, whose K goes in stretches: rows, K, N, then the kernel of the 16-bit
# plain, 16-bit gated, fp32 plain and fp32 gated product (None: any, these shapes are on the edge)
LONG = [
    (1, 16384, 64, ("deep", 1, 2, 16), ("deep", 1, 2, 16), ("deep", 1, 2, 16), ("deep", 1, 2, 16)),
    (20, 8192, 96, ("deep", 1, 2, 16), ("deep", 1, 2, 16), ("deep", 1, 2, 16), ("deep", 1, 2, 16)),
    (64, 8192, 512, ("deep", 2, 2, 16), ("deep", 2, 4, 16), ("deep", 2, 2, 16), ("deep", 2, 4, 16)),
    (100, 4104, 130, None, None, ("deep", 2, 2, 16), None),
    (200, 8192, 300, ("deep", 2, 4, 8), ("deep", 2, 4, 4), None, None),
    (300, 16392, 64, ("deep", 2, 2, 16), ("deep", 2, 4, 16), ("deep", 2, 2, 16), ("deep", 2, 4, 16)),
]

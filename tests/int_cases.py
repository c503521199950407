"""Shapes for the integer products that reach every kernel in both forms, dense and per expert.  The GPU
tests run them and the CPU tests check which kernel the library takes for each."""

# Integers at an odd address, and rows that are no whole chunks, are copied into the workspace where there are many of them;
# SMALL is a workspace without room for that.
SMALL = 256

# x, out, gated, experts (0 = dense), tokens, top_k, K, N, offset of x in elements, workspace (-1 = as asked for),
# (kernel, mt, nt, splits, quantised or copied first)
CASES = [
    # rows of x at odd addresses, from where they are
    ("int8", "bf16", False, 0, 549, 1, 71, 1331, 1, SMALL, ("any", 2, 2, 1, 0)),
    ("int8", "fp32", True, 0, 287, 1, 80, 948, 1, SMALL, ("any", 2, 2, 1, 0)),
    ("int8", "fp16", False, 3, 40, 2, 155, 66, 1, SMALL, ("any", 2, 2, 1, 0)),
    ("int8", "bf16", True, 3, 25, 1, 816, 30, 1, SMALL, ("any", 2, 2, 1, 0)),
    # one launch that quantises x itself
    ("bf16", "fp32", False, 0, 1, 1, 522, 60, 0, -1, ("int_few", 1, 1, 1, 0)),
    ("bf16", "fp16", True, 0, 2, 1, 282, 44, 3, -1, ("int_few", 1, 1, 1, 0)),
    ("fp32", "bf16", False, 0, 16, 1, 1003, 285, 1, -1, ("int_few", 1, 1, 1, 0)),
    ("fp32", "bf16", False, 0, 247, 1, 16, 285, 0, -1, ("int_few", 1, 2, 1, 0)),
    ("bf16", "fp32", True, 0, 306, 1, 26, 109, 0, -1, ("int_few", 1, 2, 1, 0)),
    ("fp32", "bf16", False, 0, 577, 1, 29, 235, 0, -1, ("int_few", 1, 4, 1, 0)),
    ("fp32", "fp32", True, 0, 339, 1, 24, 222, 0, -1, ("int_few", 1, 4, 1, 0)),
    ("fp32", "fp16", False, 5, 3, 2, 1602, 81, 1, -1, ("int_few", 1, 4, 1, 0)),
    ("fp16", "fp32", True, 8, 1, 2, 228, 15, 0, -1, ("int_few", 1, 4, 1, 0)),
    ("bf16", "bf16", True, 200, 30, 6, 40, 21, 0, -1, ("int_few", 1, 4, 1, 0)),
    # few rows, K split over waves
    ("int8", "fp16", False, 0, 2, 1, 1408, 19, 0, -1, ("few", 1, 0, 1, 0)),
    ("int8", "fp32", True, 0, 3, 1, 1408, 33, 0, -1, ("few", 1, 0, 1, 0)),
    ("bf16", "fp16", False, 0, 9, 1, 4293, 23, 0, -1, ("few", 1, 0, 1, 1)),
    ("int8", "bf16", True, 0, 275, 1, 16, 58, 1, -1, ("few", 1, 0, 1, 1)),
    ("int8", "fp32", False, 0, 444, 1, 12, 179, 0, -1, ("few", 2, 0, 1, 0)),
    ("fp32", "fp16", True, 0, 476, 1, 13, 219, 0, -1, ("few", 2, 0, 1, 1)),
    # small tiles
    ("int8", "bf16", False, 0, 487, 1, 272, 589, 0, -1, ("deep", 1, 2, 1, 0)),
    ("bf16", "bf16", True, 0, 350, 1, 257, 377, 0, -1, ("deep", 1, 2, 1, 1)),
    ("int8", "fp32", False, 2, 131, 2, 150, 35, 1, -1, ("deep", 1, 2, 1, 1)),
    ("fp32", "fp32", True, 2, 32, 1, 198, 70, 0, -1, ("deep", 1, 2, 1, 1)),
    ("fp32", "fp16", False, 0, 555, 1, 17, 1583, 0, -1, ("deep", 2, 2, 1, 1)),
    ("int8", "bf16", True, 0, 568, 1, 21, 2092, 1, -1, ("deep", 2, 2, 1, 1)),
    ("bf16", "fp16", False, 2, 392, 2, 27, 682, 0, -1, ("deep", 2, 2, 1, 1)),
    ("bf16", "fp16", True, 8, 749, 1, 20, 298, 0, -1, ("deep", 2, 2, 1, 1)),
    ("int8", "bf16", False, 0, 591, 1, 52, 1838, 1, -1, ("deep", 2, 4, 1, 1)),
    ("int8", "fp32", True, 0, 543, 1, 21, 1685, 1, -1, ("deep", 2, 4, 1, 1)),
    ("bf16", "fp32", False, 3, 326, 3, 23, 1261, 0, -1, ("deep", 2, 4, 1, 1)),
    ("int8", "fp16", True, 100, 381, 2, 66, 209, 1, -1, ("deep", 2, 4, 1, 1)),
    # the same with K in stretches
    ("int8", "bf16", False, 0, 6, 1, 16400, 37, 0, -1, ("deep", 1, 2, 16, 0)),
    ("int8", "fp32", True, 0, 11, 1, 32784, 21, 0, -1, ("deep", 1, 2, 16, 0)),
    ("bf16", "bf16", False, 24, 11, 1, 16400, 20, 0, -1, ("deep", 1, 2, 8, 1)),
    ("int8", "fp16", True, 2, 4, 2, 16400, 46, 0, -1, ("deep", 1, 2, 16, 0)),
    ("int8", "fp32", False, 0, 261, 1, 16400, 29, 1, -1, ("deep", 2, 2, 16, 1)),
    ("bf16", "bf16", True, 0, 355, 1, 16400, 17, 0, -1, ("deep", 2, 2, 16, 1)),
    ("bf16", "fp16", False, 8, 33, 2, 32784, 27, 0, -1, ("deep", 2, 2, 16, 1)),
    ("int8", "fp16", True, 3, 252, 2, 8208, 19, 0, -1, ("deep", 2, 2, 8, 0)),
    ("int8", "fp32", False, 0, 5, 1, 16400, 779, 0, -1, ("deep", 2, 4, 16, 0)),
    ("fp32", "bf16", True, 0, 6, 1, 16400, 279, 0, -1, ("deep", 2, 4, 16, 1)),
    ("int8", "fp32", False, 8, 9, 1, 8208, 146, 0, -1, ("deep", 2, 4, 8, 0)),
    ("fp32", "fp32", True, 8, 2, 5, 8208, 94, 0, -1, ("deep", 2, 4, 8, 1)),
    # large tiles
    ("int8", "fp16", False, 0, 4486, 1, 176, 876, 0, -1, ("tile", 4, 4, 1, 0)),
    ("bf16", "fp16", True, 0, 2210, 1, 38, 1577, 0, -1, ("tile", 4, 4, 1, 1)),
    ("int8", "fp32", False, 8, 2563, 3, 160, 487, 0, -1, ("tile", 4, 4, 1, 0)),
    ("int8", "bf16", True, 5, 239, 4, 143, 1431, 1, -1, ("tile", 4, 4, 1, 1)),
    ("fp16", "fp32", False, 0, 5986, 1, 1088, 2094, 0, -1, ("tile", 8, 8, 1, 1)),
    ("int8", "fp16", True, 0, 3918, 1, 518, 1859, 1, -1, ("tile", 8, 8, 1, 1)),
    ("bf16", "fp16", False, 8, 1688, 5, 800, 1525, 0, -1, ("tile", 8, 8, 1, 1)),
    ("int8", "bf16", True, 3, 2517, 3, 525, 794, 1, -1, ("tile", 8, 8, 1, 1)),
]

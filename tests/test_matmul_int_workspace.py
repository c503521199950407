"""What workspace a call of the integer products asks for, as the header has it (CPU only: every call here
ends in the host's checks)."""

import int_cases
import quantized_expert_gemv_moe_amd as moe
from test_matmul_int_choice import choose  # noqa: F401
from test_matmul_int_host import I, W, call, gcall, linear


def test_floating_rows_ask_for_all_of_it(choose):  # noqa: F811
    """Codes and scales of the rows whatever the kernel, the one that quantises into LDS among them."""
    for x, o, g, e, t, top, k, n, off, ws, kernel in int_cases.CASES:
        if x != "int8":
            codes = t * top * ((k + 15) // 16 * 16)
            for short in (0, codes // 2, codes):  # no room for the scales
                assert choose([(x, o, g, e, t * top, k, n, 1, off, short)])[0][0] == f"status{W}", (x, e, t, k, n, kernel)
    for rows in (1, 8, 64):  # the kernel for few rows and others
        for xd in (0, 1):
            assert call(xd=xd, rows=rows, ws=None) == I and call(xd=xd, rows=rows, wb=0) == W
            assert gcall(xd=xd, slots=rows, ws=None) == I and gcall(xd=xd, slots=rows, wb=0) == W


def test_integers_take_less(choose):  # noqa: F811
    """None at all where K is whole; rows at odd addresses are then not copied."""
    seen = 0
    for x, o, g, e, t, top, k, n, off, ws, kernel in int_cases.CASES:
        if x == "int8":
            got = choose([(x, o, g, e, t * top, k, n, 1, off, 0)])[0]
            assert got[0] == f"status{W}" if got[0].startswith("status") else got[3:] == (1, 0), (t, k, n, got)
            seen += not got[0].startswith("status")
    assert seen > 10
    # a stretch of K per workgroup needs its sums' place, and a NULL is no place
    long = linear(in_features=16400, out_features=32, row_stride=16400)
    assert call(lin=long, rows=6, ws=None) == I and call(lin=long, rows=6, wb=0) == W
    assert call(rows=0, ws=None) == moe.MOE_OK

"""Problems that reach every kernel of the products by expert of microscaled FP4 rows on 256 CUs
(moe_grouped_gemm_mxfp4): each with and without the activation, with rows as they lie, gathered
through a list in LDS and gathered from row_idx itself.  tests/test_mxfp4_rule.py asks the launch
rule whether they do."""

CUS = 256

# (rows, wavefronts, workgroups a CU, 64-bit addresses, how rows come): R, E, N without the
# activation, N with it, K
PROBLEMS = {
    (256, 4, 1, False, "plain"): (9000, 3, 2600, 1300, 416),
    (256, 4, 1, False, "gathered"): (9000, 3, 2603, 1301, 800),
    (128, 8, 1, False, "plain"): (2000, 8, 2300, 1157, 288),
    (128, 8, 1, False, "list"): (1300, 16, 2300, 1157, 288),
    (128, 8, 1, False, "direct"): (12000, 65, 1030, 515, 160),
    (64, 8, 1, False, "plain"): (5000, 600, 300, 140, 288),
    (64, 8, 1, False, "list"): (2000, 100, 300, 150, 544),
    (64, 8, 1, False, "direct"): (5000, 600, 300, 141, 160),
    (64, 4, 2, False, "plain"): (1000, 1, 2001, 1000, 672),
    (64, 4, 2, False, "list"): (1000, 1, 2001, 1000, 672),
    (64, 4, 2, False, "direct"): (75000, 8200, 40, 20, 96),
    (32, 2, 4, False, "plain"): (300, 1, 1000, 500, 544),
    (32, 2, 4, False, "list"): (300, 1, 1000, 500, 4128),
    (32, 2, 4, False, "direct"): (2500, 1, 400, 200, 288),
    (16, 2, 4, False, "plain"): (40, 4, 300, 150, 544),
    (16, 2, 4, False, "list"): (40, 4, 301, 151, 1056),
    (16, 2, 4, False, "direct"): (2200, 300, 40, 20, 288),
    (64, 4, 2, True, "list"): (600, 2, 90, 45, 16384),
    (64, 4, 2, True, "direct"): (2500, 3, 50, 26, 16384),
    (16, 2, 4, True, "list"): (50, 8, 90, 45, 16384),
    (16, 2, 4, True, "direct"): (2100, 300, 40, 20, 16384),
}
# of the widest weights' kernels without gathered rows (one expert's weights past 4 GB):
# R, E, N with the activation, K
WIDE_WEIGHTS = {(64, 4, 2, True, "plain"): (200, 1, 65536, 65536),
                (16, 2, 4, True, "plain"): (3, 1, 65536, 65536)}
WIDE_ROWS = 530000                     # rows of 8192 code bytes: past 4 GB
ROW_DIV = 3


def sizes(kernel, situ):
    """(R, E, N, K, x_rows) of a problem."""
    R, E, plain, half, K = PROBLEMS[kernel]
    gathered = kernel[4] != "plain"
    x_rows = WIDE_ROWS if kernel[3] else (R + ROW_DIV - 1) // ROW_DIV if gathered else R
    return R, E, half if situ else plain, K, x_rows

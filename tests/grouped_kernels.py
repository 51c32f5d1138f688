"""Calls of the products beside the layer that reach each of their kernels, and
the query of which kernel a call is given to.

A case: the product, the type of its output (None: both, whose kernel is the
same), the kernel, rows per group (a number: no offsets), n, k and, for the
weight gradients, which sides are looked up through pairs.
"""

import block_scaled_mxfp4_amd as B

ADDRESS = 1 << 20          # a stand-in: the query follows no address

RAGGED = [0, 1, 63, 64, 65, 128, 129, 190, 320, 0, 7, 0, 500, 2, 0, 33]     # 0, 1, 2, 3 and more steps of 64 rows
FEW = [1, 0, 9, 3, 0, 2, 17, 0, 0, 1, 4, 8, 0, 6, 0, 5]
SMALL = [9, 0, 17, 30, 1, 0, 0, 8, 2, 33, 5, 3, 0, 16, 4, 2]
MIDDLE = [70, 0, 65, 200, 1, 0, 129, 64, 33, 90, 100, 7, 0, 128, 201, 12]

CASES = [
    ("fwd", None, "grouped_few_kernel 16", [2, 0, 5], 77, 136),
    ("fwd", None, "grouped_few_kernel 16", 7, 520, 1032),
    ("fwd", None, "grouped_few_kernel 32", FEW, 1034, 264),
    ("fwd", None, "grouped_thin_kernel", [700, 33, 0, 290], 783, 40),
    ("fwd", None, "grouped_thin_kernel", 300, 136, 64),
    ("fwd", None, "grouped_kernel 64x128 short", [700, 33, 0, 290], 785, 104),
    ("fwd", None, "grouped_kernel 64x128 short", 300, 136, 128),
    ("fwd", None, "grouped_kernel 64x64", [60, 0, 33], 265, 328),
    ("fwd", None, "grouped_kernel 64x64", 300, 520, 264),
    ("fwd", None, "grouped_kernel 64x128", SMALL, 2057, 264),
    ("fwd", None, "grouped_kernel 64x128", 300, 8200, 264),
    ("fwd", None, "grouped_kernel 128x128", MIDDLE, 3208, 264),
    ("fwd", None, "grouped_kernel 128x128", 520, 8201, 264),
    ("fwd", None, "grouped_pair_kernel", 2100, 4104, 264),
    ("fwd", None, "grouped_pair_kernel", [2 * c for c in MIDDLE], 3205, 264),
    ("fwd", None, "grouped_split_kernel 64x32", [60, 0, 45], 521, 1800),
    ("fwd", None, "grouped_split_kernel 64x32", 60, 72, 1032),
    ("fwd", None, "grouped_split_kernel 64x64", SMALL, 520, 1544),
    ("fwd", None, "grouped_split_kernel 64x64", 128, 8190, 1800),
]
for f32 in (False, True):
    CASES += [
        ("fp8", f32, "grouped_few_kernel 16", [2, 0, 5], 77, 144),
        ("fp8", f32, "grouped_few_kernel 16", 7, 520, 1040),
        ("fp8", f32, "grouped_few_kernel 32", FEW, 1034, 272),
        ("fp8", f32, "grouped_kernel 64x128 short", [700, 33, 0, 290], 785, 208),
        ("fp8", f32, "grouped_kernel 64x128 short", 300, 136, 48),
        ("fp8", f32, "grouped_kernel 64x64", [60, 0, 33], 265, 336),
        ("fp8", f32, "grouped_kernel 64x64", 300, 520, 272),
        ("fp8", f32, "grouped_kernel 64x128", SMALL, 2057, 272),
        ("fp8", f32, "grouped_kernel 64x128", 300, 8200, 272),
        ("fp8", f32, "grouped_kernel 128x128", MIDDLE, 3208, 272),
        ("fp8", f32, "grouped_kernel 128x128", 520, 8201, 272),
        ("fp8", f32, "grouped_split_kernel 64x32", [60, 0, 45], 521, 1808),
        ("fp8", f32, "grouped_split_kernel 64x32", 60, 72, 1552),
        ("fp8", f32, "grouped_split_kernel 64x64", SMALL, 776, 4112),
        ("fp8", f32, "grouped_split_kernel 64x64", 128, 8190, 4112),
    ]
CASES += [
    ("fp8", False, "grouped_pair_kernel", 2100, 4104, 272),
    ("fp8", False, "grouped_pair_kernel", [2 * c for c in MIDDLE], 3205, 272),
    ("fp8", False, "grouped_pair_kernel", [3000, 0, 2500, 1], 4099, 1168),
]
# dx: the contraction is n, the columns are k
CASES += [("dgrad", out, kernel, counts, k, (n + 7) // 8 * 8) for p, out, kernel, counts, n, k in CASES
          if p == "fwd" and "few" not in kernel]
for sides in ("", "x", "y", "xy"):
    at = " indexed" if sides else ""
    CASES += [
        ("wgrad", None, "grouped_kernel 64x64" + at, [60, 0, 33, 190], 72, 136, sides),
        ("wgrad", None, "grouped_kernel 64x128" + at, SMALL, 72, 1040, sides),
        ("wgrad", None, "grouped_kernel 64x128" + at, RAGGED, 520, 1544, sides),
        ("wgrad", None, "grouped_kernel 128x128" + at, RAGGED, 264, 1032, sides),
        ("wgrad", None, "grouped_kernel 128x128" + at, 500, 2056, 2056, sides),
        ("wgrad", None, "grouped_pair_kernel" + at, RAGGED, 264, 1544, sides),
        ("wgrad", None, "grouped_pair_kernel" + at, [0, 700, 130, 1, 0, 1200], 2568, 2312, sides),
        ("wgrad", None, "grouped_pair_kernel" + at, 2500, 4104, 2056, sides),
    ]
CASES += [
    ("wgrad", None, "grouped_split_kernel 64x32", [2500, 0, 3300], 72, 136, ""),
    ("wgrad", None, "grouped_split_kernel 64x32", 1100, 264, 136, ""),
    ("wgrad", None, "grouped_split_kernel 64x64", 2100, 72, 4104, ""),
    ("wgrad", None, "grouped_split_kernel 64x64", [2500, 0, 3300], 72, 1544, ""),
]
CASES = [c if len(c) == 7 else c + ("",) for c in CASES]

KERNELS = {
    "fwd": ["few_kernel 16", "few_kernel 32", "thin_kernel", "kernel 64x128 short", "kernel 64x64", "kernel 64x128",
            "kernel 128x128", "pair_kernel", "split_kernel 64x32", "split_kernel 64x64"],
    "fp8": ["few_kernel 16", "few_kernel 32", "kernel 64x128 short", "kernel 64x64", "kernel 64x128", "kernel 128x128",
            "pair_kernel", "split_kernel 64x32", "split_kernel 64x64"],
    "dgrad": ["thin_kernel", "kernel 64x128 short", "kernel 64x64", "kernel 64x128", "kernel 128x128", "pair_kernel",
              "split_kernel 64x32", "split_kernel 64x64"],
    "wgrad": ["kernel 64x64", "kernel 64x128", "kernel 128x128", "pair_kernel", "split_kernel 64x32",
              "split_kernel 64x64", "kernel 64x64 indexed", "kernel 64x128 indexed", "kernel 128x128 indexed",
              "pair_kernel indexed"],
}


def rows_of(counts):
    """Rows and groups of a case; with offsets three rows belong to no group."""
    return (counts, 1) if isinstance(counts, int) else (sum(counts) + 3, len(counts))


def case_id(c):
    p, f32, kernel, counts, n, k, sides = c
    return "-".join(filter(None, (p, {None: "", False: "bf16", True: "f32"}[f32], kernel.replace(" ", "_"), sides,
                                  str(rows_of(counts)[0]) + ("" if isinstance(counts, int) else f"in{len(counts)}"),
                                  str(n), str(k))))


def kernel_of(product, rows, experts, n, k, *, f32=False, offsets=True, sides="", x_rows=None, x_div=1, cus=256):
    """The kernel of a call with these sizes."""
    off = ADDRESS if offsets else None
    if product == "fp8":
        a = B.SituMoeFp8Matmul(rows=rows, n=n, k=k, experts=experts, out_dtype=B.OUT_F32 if f32 else B.OUT_BF16,
                               a_stride=k, a_scale_stride=-(-k // 128), out_stride=n, a=ADDRESS, a_scale=ADDRESS,
                               w=ADDRESS, w_scale=ADDRESS, offsets=off, out=ADDRESS)
        return B.situ_moe_matmul_fp8_block128_kernel(a, cus)
    a = B.SituMoeGrouped(rows=rows, n=n, k=k, experts=experts, x_rows=x_rows or rows, y_rows=2 * rows,
                         x_div=x_div if "x" in sides else 0, y_div=1 if "y" in sides else 0,
                         out_dtype=B.OUT_F32 if f32 else B.OUT_BF16, x_stride=k, y_stride=n, offsets=off,
                         pairs=ADDRESS if sides else None, x=ADDRESS, y=ADDRESS, w=ADDRESS)
    return B.situ_moe_grouped_matmul_kernel(("fwd", "dgrad", "wgrad").index(product), a, cus)

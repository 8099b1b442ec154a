"""16-bit products whose sizes reach each kernel, tile shape and store policy that the
library's plan can choose: what the plan is asserted to be on the CPU
(test_half_plans.py), run on the GPU (test_gpu_half_plans.py).

A plan reads: tile, p1 results that leave past the caches, p0 others.  Every size is run
with BF16 and FP16 operands and results in their type, FP32 and accumulated FP32."""

#: (operands' type, results': None for the same, "f32", "add")
KINDS = [(t, out) for t in ("bf16", "fp16") for out in (None, "f32", "add")]

# (rows of each group, rows past the last one, n, k, weights [k, n], tile, results past the caches)
_ROWS = [
    ([2100, 0, 1700, 63, 3], 5, 2056, 328, False, "256x256", False),
    ([2100, 0, 1700, 63, 3], 5, 2056, 328, True, "256x256", False),
    ([3001, 129, 0, 2890, 460], 20, 4096, 200, False, "256x256", True),
    ([3001, 129, 0, 2890, 460], 20, 4096, 200, True, "256x256", True),
    ([301, 0, 255, 400], 3, 4192, 328, False, "128x256", False),
    ([301, 0, 255, 400], 3, 4192, 328, True, "128x256", False),
    ([4300, 1, 1199], 0, 4096, 264, False, "128x256", True),
    ([4300, 1, 1199], 0, 4096, 264, True, "128x256", True),
    ([300, 130, 0, 70], 9, 520, 328, False, "128x128", False),
    ([300, 130, 0, 70], 9, 520, 328, True, "128x128", False),
    ([40, 0, 61, 90] * 30, 1, 3200, 200, False, "128x128", True),
    ([40, 0, 61, 90] * 30, 1, 3200, 200, True, "128x128", True),
    ([30, 0, 41, 7], 2, 520, 328, False, "64x128", False),
    ([30, 0, 41, 7], 2, 520, 328, True, "64x128", False),
    ([30, 0, 41, 7] * 50, 2, 4608, 200, False, "64x128", True),
    ([30, 0, 41, 7] * 50, 2, 4608, 200, True, "64x128", True),
    ([15, 0, 9, 33], 2, 520, 1096, False, "32x64", False),
    ([15, 0, 9, 33], 2, 520, 1096, True, "32x64", False),
    ([15, 0, 9, 33] * 25, 2, 12864, 72, False, "32x64", True),
    ([1, 0, 2, 0, 1], 1, 24, 1096, False, "direct", None),
]
CONTIGUOUS = [(c, spare, n, k, t, out, tr, tile if p is None else f"{tile} p{int(p and out != 'add')}")
              for c, spare, n, k, tr, tile, p in _ROWS for t, out in KINDS]

# (valid rows of each slot, rows of a slot, n, k, weights [k, n], tile, results past the caches)
_SLOTS = [
    ([132, 0, 129, 1] * 4, 132, 2056, 328, False, "256x256", False),
    ([132, 0, 129, 1] * 4, 132, 2056, 328, True, "256x256", False),
    ([520, 0, 257, 1] * 2, 520, 4096, 200, False, "256x256", True),
    ([520, 0, 257, 1] * 2, 520, 4096, 200, True, "256x256", True),
    ([132, 0, 129, 1] * 2, 132, 2056, 328, False, "128x256", False),
    ([132, 0, 129, 1] * 2, 132, 2056, 328, True, "128x256", False),
    ([260, 0, 129, 1] * 4, 260, 4096, 200, False, "128x256", True),
    ([260, 0, 129, 1] * 4, 260, 4096, 200, True, "128x256", True),
    ([140, 0, 129, 1], 140, 520, 328, False, "128x128", False),
    ([140, 0, 129, 1], 140, 520, 328, True, "128x128", False),
    ([260, 0, 129, 1] * 2, 260, 8256, 200, False, "128x128", True),
    ([260, 0, 129, 1] * 2, 260, 8256, 200, True, "128x128", True),
    ([40, 0, 33, 1], 40, 520, 328, False, "64x128", False),
    ([40, 0, 33, 1], 40, 520, 328, True, "64x128", False),
    ([64, 0, 33, 1] * 10, 64, 8256, 200, False, "64x128", True),
    ([64, 0, 33, 1] * 10, 64, 8256, 200, True, "64x128", True),
    ([20, 0, 9, 1], 20, 520, 1096, False, "32x64", False),
    ([20, 0, 9, 1], 20, 520, 1096, True, "32x64", False),
    ([32, 0, 9, 1] * 20, 32, 6592, 72, False, "32x64", True),
    ([8, 0, 3, 1], 8, 24, 1096, False, "direct", None),
]
MASKED = [(c, slot, n, k, t, out, tr, tile if p is None else f"{tile} p{int(p and out != 'add')}")
          for c, slot, n, k, tr, tile, p in _SLOTS for t, out in KINDS]

# (rows of each group, rows past the last one, m, n, tile, results past the caches); more than 128 groups are taken
# as they come, fewer longest first
_SUMS = [
    ([0, 63, 65, 200, 0, 1, 640, 130], 3, 1032, 1528, "256x256", False),
    ([0, 63, 65, 200, 0, 1, 640, 130] * 2, 3, 1032, 1536, "256x256", True),
    ([0, 63, 65, 200, 0, 1, 130] * 19, 0, 136, 1544, "256x256", False),
    ([0, 63, 65, 200, 0, 1, 130] * 19, 0, 136, 1536, "256x256", True),
    ([0, 63, 65, 200, 0, 1, 130], 3, 136, 264, "128x128", False),
    ([0, 63, 65, 200, 0, 1, 640, 130], 3, 1536, 1536, "128x128", True),
    ([0, 63, 65, 200, 0, 1, 130] * 27, 3, 72, 1544, "128x128", False),
    ([0, 63, 65, 200, 0, 1, 130] * 27, 0, 72, 1536, "128x128", True),
]
GROUP_K = [(c, spare, m, n, t, out, f"{tile} p{int(p and out != 'add')}")
           for c, spare, m, n, tile, p in _SUMS for t, out in KINDS]

# groups of many thousands of rows, the last of them past 2^31 elements of a
GROUP_K += [([450000, 0, 449999, 70001], 7, 2560, 1536, t, out, "256x256 " + ("p0" if out == "add" else "p1"))
            for t, out in (("bf16", "f32"), ("fp16", "add"))]

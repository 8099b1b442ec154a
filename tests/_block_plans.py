"""Block-128 products whose sizes reach each kernel, tile shape, K split and
store policy that the library's plan can choose: what the plan is asserted to be
on the CPU (test_block_plans.py), run on the GPU (test_gpu_block_plans.py).

A plan reads: operand path, tile, sN for N slices of K, p0 stores kept in the
caches, p1 streamed, p2 with streamed weights too; "+" joins the launch over the
first `head` columns and the one over the rest."""
import torch

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
FULL = 64 << 20

#: (m, n, k, result type, workspace bytes, plan)
DENSE = [
    # whole rounds of 256 x 256 tiles, then the other columns
    (3611, 9272, 672, BF16, FULL, "fp8 256x256 s1 p1 + fp8 128x128 s1 p0 head 8704"),
    (3471, 9496, 4096, BF16, FULL, "fp8 256x256 s1 p1 + fp8 128x128 s3 p0 head 9216"),
    (5960, 6048, 640, BF16, 0, "fp8 256x256 s1 p1 + fp8 128x256 s1 p0 head 5376"),
    (3313, 10528, 5056, BF16, FULL, "fp8 256x256 s1 p1 + fp8 128x256 s3 p0 head 9984"),
    (5525, 9408, 5248, BF16, FULL, "fp8 256x256 s1 p1 + fp8 256x256 s3 p0 head 8704"),
    (3983, 8256, 416, BF16, FULL, "fp8 256x256 s1 p1 + fp8 64x128 s1 p0 head 8192"),
    (2961, 10872, 4384, BF16, FULL, "fp8 256x256 s1 p1 + fp8 64x128 s5 p0 head 10752"),
    (5797, 4208, 4992, BF16, 0, "fp8 256x256 s1 p0 + fp8 128x128 s1 p0 head 2816"),
    # one launch
    (4277, 2032, 448, BF16, FULL, "fp8 256x256 s1 p0"),
    (5570, 4560, 416, BF16, FULL, "fp8 256x256 s1 p1"),
    (3342, 1256, 5984, BF16, FULL, "fp8 256x256 s3 p0"),
    (1548, 2448, 448, BF16, FULL, "fp8 128x256 s1 p0"),
    (2405, 7040, 416, BF16, 0, "fp8 128x256 s1 p1"),
    (1168, 1064, 5728, BF16, FULL, "fp8 128x256 s5 p0"),
    (1245, 1568, 416, BF16, FULL, "fp8 128x128 s1 p0"),
    (1238, 520, 2080, BF16, FULL, "fp8 128x128 s3 p0"),
    (77, 5120, 17408, BF16, FULL, "fp8 128x128 s6 p0"),
    (130, 2056, 512, BF16, FULL, "fp8 64x128 s1 p0"),
    (53, 1880, 14688, BF16, FULL, "fp8 64x128 s13 p0"),
    (3590, 1032, 64, F16, FULL, "fp16 256x128 s1 p0"),
    (834, 10096, 96, F32, FULL, "fp16 256x128 s1 p1"),
    (4096, 4104, 512, F32, 0, "fp16 256x128 s1 p1"),
    (1622, 1160, 2080, F32, FULL, "fp16 256x128 s3 p0"),
    (806, 16936, 96, F32, FULL, "fp16 128x128 s1 p1"),
    (608, 1032, 2912, F16, FULL, "fp16 128x128 s5 p0"),
    (77, 5120, 17408, F32, FULL, "fp16 128x128 s6 p0"),
    (77, 5120, 17408, F16, FULL, "fp16 128x128 s6 p0"),
    (53, 1880, 14688, F32, FULL, "fp16 64x128 s15 p0"),
    (130, 2056, 512, F16, 0, "fp16 64x128 s1 p0"),
    (9, 264, 1056, BF16, FULL, "direct"),
]

#: (batch, m, n, k, result type, workspace bytes, plan)
BATCH = [
    (2, 3541, 3400, 416, BF16, FULL, "fp8 256x256 s1 p1"),
    (2, 1713, 2360, 512, BF16, 0, "fp8 256x256 s1 p0"),
    (2, 1365, 808, 9440, BF16, FULL, "fp8 256x256 s5 p0"),
    (2, 1829, 1032, 416, BF16, FULL, "fp8 128x256 s1 p0"),
    (4, 672, 688, 448, BF16, FULL, "fp8 128x128 s1 p0"),
    (2, 651, 272, 2496, BF16, FULL, "fp8 128x128 s5 p0"),
    (8, 2103, 8, 32, F32, 0, "fp16 128x128 s1 p0"),
    (8, 121, 9864, 96, F32, FULL, "fp16 128x128 s1 p1"),
    (2, 641, 440, 3072, F16, FULL, "fp16 128x128 s5 p0"),
]

#: (rows of each group, rows past the last one, n, k, result type, plan)
CONTIGUOUS = [
    ([1000, 0, 130, 700, 2, 900], 3, 520, 640, BF16, "fp8 256x256 s1 p0"),
    ([2000, 3, 0, 1500, 1210], 0, 3872, 416, BF16, "fp8 256x256 s1 p1"),
    ([600, 8, 0, 671], 1, 13872, 544, BF16, "fp8 128x256 s1 p1"),
    ([90] * 30 + [0, 127], 0, 3016, 96, F32, "fp16 128x128 s1 p1"),
    ([700, 0, 815], 5, 5800, 160, F32, "fp16 256x128 s1 p1"),
]

#: (valid rows of each slot, rows of a slot, n, k, result type, plan)
MASKED = [
    ([300, 0, 137, 1], 300, 264, 544, BF16, "fp8 256x256 s1 p0"),
    ([396, 255, 0], 396, 16408, 416, BF16, "fp8 256x256 s1 p1"),
    ([130, 200, 7], 200, 1032, 672, BF16, "fp8 256x256 s1 p2"),
    ([344, 1, 300], 344, 136, 96, F32, "fp16 256x128 s1 p0"),
    ([388, 0, 120], 388, 7232, 160, F32, "fp16 256x128 s1 p1"),
    ([137, 64, 0], 137, 264, 544, F16, "fp16 256x128 s1 p2"),
    ([81, 0, 70], 81, 264, 544, F16, "fp16 128x128 s1 p2"),
]

#: (K blocks of each group, m, n, result type, plan)
GROUP_K = [
    ([1, 3, 0, 2, 1, 5, 0, 1], 112, 9752, F32, "fp16 128x128 s1 p1"),
    ([2, 0, 5], 520, 1032, BF16, "fp16 256x128 s1 p0"),
]

"""Shapes of the ragged products' GPU tests with the kernel that each of them is
there for, at 152 SMs; tests/test_ragged_shapes.py holds the library's choices
to that on the CPU, so that no test falls back to another kernel unseen."""

# gemm_lora in CTA pairs: (M, N, K, R, L, run of rows of one adapter)
LORA_PAIRS = [
    (700, 7000, 264, 16, 6, 90),    # a last row tile of 188 rows
    (1500, 3400, 136, 32, 5, 300),
    (1033, 4100, 72, 8, 200, 1),    # many adapters per list
    (1500, 3339, 65, 64, 3, 1),     # odd features and depth: repacked, C by element
    (300, 10240, 200, 128, 9, 7),
    (513, 6667, 136, 24, 11, 19),
]

# gemm_lora, more rows than T's scratch holds: (M, N, K, R, L, run), panels in bf16 and fp16
LORA_PANELS = [
    ((4500, 1504, 72, 128, 256, 1), 2, 3),   # pairs, 4096 (2048) rows a panel
    ((16700, 72, 64, 128, 256, 1), 3, 5),    # single CTAs, 8192 (4096) rows
]

# gemm_grouped: (sizes, N, K, kernel)
ROWS_PAIRS = [
    ([700, 30, 0, 1100, 256, 513], 2048, 328), ([900, 300, 0, 0, 1500], 2088, 776),
    ([600, 1, 900, 33], 2503, 1032),
]
# fp32 results with a fused epilogue in pairs: the second and third with any beta
ROWS_PAIRS_F32 = [([7000, 300, 0, 6000], 4400, 776), ([7000, 300, 0, 6000], 4400, 4104),
                  ([4100, 1, 8500], 4567, 4100)]
ROWS_PAIRS_COUNTED = [([5000, 2000, 0, 300, 2900, 9], 2048, 4104)]
ROWS_SINGLE = [([50, 0, 49, 3] * 12, 520, 1000), ([40, 64, 1] * 10, 776, 136)]  # whole depth
ROWS_SPLIT = [([9], 1024, 16384, 8), ([2, 20], 264, 9000, 8), ([60], 520, 2048, 4)]

# gemm_grouped_k: (sizes, M, N). Pairs for 16-bit results that are written, for
# 16-bit results that are read (beta), and for fp32 ones, plain or with an
# epilogue; fp32 results that are read never get pairs.
DEPTH_PAIRS = [([1500, 0, 705, 704, 40], 1032, 1288), ([1, 3000, 63], 1040, 1800)]
DEPTH_PAIRS_READ = [([i * 7 % 61 for i in range(200)], 776, 776)]
DEPTH_PAIRS_F32 = [([1500, 0, 705, 704, 640], 2568, 2824)]
DEPTH_SINGLE = [([1500, 0, 705, 704, 40], 264, 328), ([2111], 136, 264)]

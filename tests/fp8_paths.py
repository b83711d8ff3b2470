"""Sizes at which the 8-bit products take each of their kernels, shared by the
host test of the rules and the GPU test of the kernels."""

# (M, out, in), path for float32 and float16 results, path for bfloat16 ones;
# each with a partial and with a whole last block of the depth
DENSE = [
    ((3, 300, 272), ("few",), ("few",)),
    ((16, 33, 512), ("few",), ("few",)),
    ((12, 300, 8208), ("rows",), ("rows",)),           # 16 rows in a pass
    ((15, 48, 4096), ("rows",), ("rows",)),
    ((20, 300, 2064), ("rows",), ("rows",)),           # 32
    ((32, 130, 2048), ("rows",), ("rows",)),
    ((40, 130, 272), ("tiles", 64, 64, 1), ("tiles", 64, 64, 1)),
    ((130, 520, 256), ("tiles", 64, 64, 1), ("tiles", 64, 64, 1)),
    ((70, 200, 4128), ("tiles", 64, 64, 8), ("tiles", 64, 64, 8)),
    ((64, 64, 8192), ("tiles", 64, 64, 16), ("tiles", 64, 64, 16)),
    ((1300, 2000, 272), ("tiles", 128, 128, 1), ("tiles", 128, 128, 1)),
    ((1290, 1990, 384), ("tiles", 128, 128, 1), ("tiles", 128, 128, 1)),
    ((4000, 2600, 272), ("tiles", 128, 128, 1), ("tiles", 256, 256, 1)),
    ((3990, 2570, 256), ("tiles", 128, 128, 1), ("tiles", 256, 256, 1)),
]

# pairs of each expert around the tile's edges, out, path for float32 and float16 results, path for bfloat16 ones
GROUPED = [
    ([16, 17, 0, 1, 15, 33, 32, 64], 530, ("tiles", 16, 128, 1), ("tiles", 16, 128, 1)),
    ([31, 32, 33, 0, 1, 63, 64, 65], 2060, ("tiles", 32, 128, 1), ("tiles", 32, 128, 1)),
    ([63, 65, 48, 49, 31, 47, 50, 40], 2580, ("tiles", 64, 128, 1), ("tiles", 64, 128, 1)),
    ([127, 128, 129, 0, 1, 255, 256, 257], 1030, ("tiles", 128, 128, 1), ("tiles", 128, 128, 1)),
    ([127, 128, 129, 0, 1, 255, 256, 257], 4100, ("tiles", 128, 256, 1), ("tiles", 128, 256, 1)),
    ([255, 256, 257, 0, 1, 511, 512, 513], 5130, ("tiles", 128, 256, 1), ("tiles", 256, 256, 1)),
]

# experts, tokens, pairs of each, out, in: around the most that one workgroup counts, in one slice of pairs and in several
MANY_EXPERTS = [(E, T, k, 130, 144) for E in (1023, 1024, 1025) for T, k in ((3000, 2), (6000, 3))]

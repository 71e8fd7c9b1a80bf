"""The FP8 product's kernels as (tokens per tile, slices of K); (0, 1) is the two-SM one."""

KERNELS = [(t, s) for t in (16, 32, 64, 96, 128) for s in (1, 2, 3, 4, 5, 6, 8, 12, 16)
           if s <= 8 or t <= 64] + [(0, 1)]

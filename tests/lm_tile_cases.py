"""Sizes of the feed-forward block (M, D, F, bf16) that together run every tile of every product, with k whole and with
k split; tests/test_lm_plan_cpu.py holds the list to that, tests/test_gpu_lm_tiles.py runs it."""

SIZES = [(72, 35, 35, 1), (69, 37, 36, 0), (1165, 49, 1899, 1), (2281, 35, 1452, 0), (708, 2697, 34, 1), (68, 2820, 276, 0),
         (1907, 83, 3096, 1), (518, 2873, 45, 0), (778, 3644, 414, 1), (4403, 1468, 67, 0), (2954, 34, 2729, 1),
         (6009, 1317, 35, 1), (4789, 213, 1811, 0), (4106, 202, 3601, 1)]

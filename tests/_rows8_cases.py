"""Sizes at which each kernel of the products in 8 bits runs (on 256 compute
units): test_rows8_plan.py holds that they do and that none is missing,
test_gpu_rows8_kernels.py compares each with exact sums.

A case: (kernel, parts of the contraction, few rows' parts and chunks, as the rule
gives them; "packed": rows laid on 16 bytes first), rows of the groups, N, K of the
experts, place of the first code (1: rows not on 16 bytes)."""
from _experts_cases import spread

I8 = [("256x256 1", spread(1, 5000), 2056, 144, 0), ("256x256 1", spread(4, 8192), 1033, 144, 0),
      ("256x256 1 packed", spread(8, 8192), 1032, 129, 0), ("128x256 1", spread(9, 600), 5000, 128, 0),
      ("128x128 1", spread(9, 8192), 520, 128, 0), ("128x128 1 packed", spread(3, 8192), 520, 1041, 0),
      ("128x128 4", spread(4, 300), 1032, 32768, 0), ("128x128 8", spread(1, 2048), 136, 32768, 0),
      ("128x128 8 packed", spread(3, 2048), 136, 32771, 0), ("64x128 1", spread(1, 2048), 1033, 272, 0),
      ("64x128 1", spread(3, 24), 9, 128, 0), ("64x128 1 packed", spread(3, 8), 8, 279, 0),
      ("64x128 2", spread(3, 16), 4104, 7168, 0), ("64x128 4", spread(4, 300), 520, 7168, 0),
      ("64x128 4 packed", spread(9, 600), 264, 7169, 1), ("64x128 8", spread(3, 20), 8, 7168, 0),
      ("64x128 8 packed", spread(6, 24), 9, 7173, 0), ("64x128 16", spread(1, 20), 8, 32768, 0),
      ("64x128 16 packed", spread(1, 20), 8, 16387, 0), ("any 1", spread(3, 16), 8, 144, 1), ("any 1", spread(1, 4096), 264, 129, 1),
      ("any 2", spread(3, 300), 8, 1040, 1), ("any 4", spread(1, 2048), 520, 7168, 1), ("any 4", spread(3, 100), 8, 2064, 1),
      ("any 8", spread(3, 24), 9, 4112, 1), ("any 16", spread(1, 20), 8, 16384, 1), ("few 1 1 1", spread(1, 8), 2841, 149, 0),
      ("few 1 1 1", spread(4, 4), 1032, 128, 1), ("few 1 1 1", [1, 0, 2, 1, 1, 0, 1, 2], 5000, 272, 1),
      ("few 1 1 4", spread(1, 8192), 9, 128, 0), ("few 1 2 1", spread(9, 16), 200, 145, 1), ("few 1 2 4", spread(1, 600), 72, 7168, 0),
      ("few 1 4 1", spread(3, 4), 8, 129, 0), ("few 1 4 4", spread(1, 20), 8, 7168, 0)]

"""Sizes at which each pair of a tile kernel and a number of parts that the rule of
the products in 8 bits takes runs (on 256 compute units), beyond those of
_rows8_cases.py and in its form: test_rows8_pairs.py holds that they do and that, over
a grid of sizes, no pair is missing; test_gpu_rows8_ranges.py compares each with exact
sums."""
from _experts_cases import spread

I8 = [("128x128 2", spread(8, 536), 1127, 15584, 0), ("128x128 2 packed", spread(1, 1487), 1194, 23587, 0),
      ("128x128 4 packed", spread(1, 4673), 139, 15431, 0), ("128x128 16", spread(1, 712), 271, 54912, 0),
      ("128x128 16 packed", spread(1, 584), 317, 69989, 0), ("64x128 2 packed", spread(1, 3246), 294, 13109, 0),
      ("128x256 1 packed", spread(1, 938), 7836, 4038, 0), ("128x256 2", spread(1, 1292), 2711, 95744, 0),
      ("128x256 2 packed", spread(1, 2956), 1224, 119090, 1), ("128x256 4", spread(1, 1468), 1240, 38832, 0),
      ("128x256 4 packed", spread(1, 1424), 1222, 40773, 0), ("128x256 8", spread(1, 1241), 662, 84576, 0),
      ("128x256 16", spread(3, 229), 600, 72976, 0), ("256x256 2", spread(4, 501), 8190, 39776, 0),
      ("256x256 4", spread(1, 213), 16115, 30064, 0), ("256x256 8", spread(1, 153), 7796, 31376, 0),
      ("256x256 16", spread(1, 143), 4075, 62480, 0)]

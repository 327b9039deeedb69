"""Sizes at which every product of the feed-forward layers takes every tile
and way of summing that some plan gives it (test_ffn_plan.py holds them to
that), ragged in each dimension.  (rows, inner or model width, columns or
hidden width), as in the calls; the last of each list fills the chip more than once."""

LINEAR = {
    "bfloat16": [(130, 303, 135), (449, 449, 499), (392, 8251, 388), (8237, 905, 407), (133, 6822, 791), (794, 6983, 130),
                 (132, 8446, 914), (1027, 301, 5605), (915, 565, 8214), (8301, 4091, 4203)],
    "float32": [(133, 325, 131), (131, 1218, 2453), (1667, 589, 581), (7750, 454, 491), (6350, 1102, 130), (130, 6381, 1116),
                (130, 7094, 1860), (1873, 7073, 130), (793, 309, 8786), (8529, 300, 1551), (4301, 2091, 4203)],
}
GATED = {
    "bfloat16": [(141, 304, 133), (473, 453, 456), (132, 398, 8580), (396, 8227, 142), (786, 6870, 259), (534, 303, 6572),
                 (262, 780, 6924), (898, 8334, 931), (779, 301, 7364), (912, 1132, 8229), (8201, 2093, 4203)],
    "float32": [(130, 304, 142), (1237, 302, 829), (3535, 354, 900), (391, 7449, 464), (1002, 7204, 193), (130, 1921, 3704),
                (2153, 6221, 130), (969, 300, 7172), (130, 1481, 8840), (8858, 303, 1473), (4201, 1093, 2203)],
}

# up to four rows: the kernel without tiles (forward, where nothing is kept in 8 bits)
FEW = [(1, 4101, 517), (2, 1031, 77), (3, 301, 1001), (4, 517, 4099)]

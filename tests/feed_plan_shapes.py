"""Sizes of the feed-forward, (dtype, rows, N, F, N_out), that with those of
test_gpu_feed_forward.SIZES take every tile, whole and at an edge, undivided
and divided, of every product in either type: test_feed_forward_plan.py checks
that they do, test_gpu_feed_forward_plan.py runs them."""

SHAPES = [
    ("bf16", 18546, 135, 130, 135), ("f32", 2767, 1410, 132, 1410), ("bf16", 5085, 12689, 1, 5172),
    ("f32", 1486, 1, 28361, 1), ("bf16", 1, 3715, 1603, 3715), ("f32", 132, 1906, 2441, 1906),
    ("bf16", 129, 2947, 2728, 2947), ("f32", 387, 16661, 1, 16661), ("f32", 1, 1013, 2203, 3781),
    ("bf16", 5466, 1, 1050, 1), ("f32", 2700, 898, 1502, 24), ("f32", 1071, 3, 1053, 4114),
    ("bf16", 135, 6135, 1464, 37), ("f32", 386, 903, 4225, 10), ("f32", 133, 149, 1, 2), ("bf16", 4295, 428, 5012, 1),
    ("bf16", 132, 20, 3547, 7552), ("bf16", 700, 4039, 2725, 2), ("bf16", 2468, 1678, 129, 5833),
    ("bf16", 7413, 45, 7533, 309), ("bf16", 7858, 1, 1588, 8322), ("f32", 3137, 20, 4836, 13036),
]

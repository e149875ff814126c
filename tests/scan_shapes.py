"""Shapes (rows of B H, tokens, channels) at which the elementwise scan's choice of a kernel reaches every kernel that it has,
with more steps than twice the tiles that a block keeps in shared memory, so that every tile's place is filled three times at
least.  test_scan_plan.py holds that; test_gpu_scan_plan.py runs them."""

# by type and by how the tiles are loaded: TMA, two values at a time (even rows off 16 bytes), one at a time (odd rows)
SHAPES = {
    ("bf16", "tma"): [(128, 770, 40), (256, 1538, 8), (56, 770, 40), (56, 1538, 24), (160, 770, 40), (56, 3145, 8), (300, 393, 24),
                      (160, 1175, 24), (1000, 393, 24), (1, 25262, 8)],
    ("bf16", "pairs"): [(256, 1538, 2), (300, 770, 2), (256, 393, 34), (256, 770, 18), (160, 3145, 2), (80, 1286, 34), (160, 1538, 18)],
    ("bf16", "single"): [(256, 1538, 1), (300, 770, 1), (256, 393, 33), (256, 770, 17), (160, 3145, 1), (80, 1286, 33), (160, 1538, 17)],
    ("f32", "tma"): [(256, 770, 8), (56, 393, 40), (80, 1286, 24), (80, 2632, 8), (256, 393, 24), (256, 262, 40), (16, 1175, 100),
                     (1, 12550, 4)],
    ("f32", "pairs"): [(256, 770, 2), (128, 393, 34), (128, 1952, 2), (40, 1286, 34)],
    ("f32", "single"): [(256, 770, 1), (128, 393, 33), (128, 1952, 1), (40, 1286, 33)],
}

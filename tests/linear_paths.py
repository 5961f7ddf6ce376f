"""Shapes of the whole linear by the kernels that they take: 'few' rows, middling tiles
('64x64', ...) or 256 x 256 'tiles'.  The GPU tests run them; a CPU test holds the rule
of csrc/linear_plan.hpp to them."""
import ctypes as C

import dynamic_mixed_precision_amd as dm

ROUTES = ["bf16", "int8", "nvfp4"]


def path(route, M, N, K, amax=False, head_dim=0):
    fn = dm.lib().dmpq_test_linear_path
    fn.argtypes, fn.restype = [C.c_int] * 3 + [C.c_int64] * 3 + [C.POINTER(C.c_int)], C.c_int
    tile = (C.c_int * 2)()
    kind = fn(ROUTES.index(route), int(amax), head_dim, M, N, K, tile)
    return ("few", f"{tile[0]}x{tile[1]}", "tiles")[kind]


# (M, N, K), the tile in BF16 and INT8; NVFP4 takes 64x64.  K leaves remainders of 16 to
# 112 (K % 128, and K % 64 in BF16), N pieces of 16 bytes or not
MID = [((300, 1000, 1936), "64x64"), ((333, 1001, 2000), "64x64"), ((64, 4400, 4112), "64x64"), ((700, 1920, 1952), "64x128"),
       ((900, 1923, 1968), "64x128"), ((900, 1920, 208), "64x128"), ((1100, 1920, 1040), "128x128"), ((1693, 1921, 2032), "128x128"),
       ((900, 2312, 1168), "128x128")]

# N a multiple of 16, for the fused amax
AMAX = [((300, 1008, 1936), "64x64"), ((900, 1920, 1968), "64x128"), ((1693, 1920, 400), "128x128")]

# n_q, n_k, D, extra columns, norm, layout, pairs, M (K 512), the tile in BF16 and INT8, in NVFP4
HEADS = [((30, 30, 64, 1920, 2, 0, 32, 1024), "64x128", "tiles"), ((20, 20, 32, 640, 1, 0, 5, 900), "64x128", "64x64"),
         ((20, 10, 64, 3, 2, 0, 32, 900), "64x128", "64x64"), ((15, 3, 32, 1344, 1, 1, 16, 1693), "128x128", "64x64"),
         ((10, 10, 64, 640, 2, 1, 24, 1693), "128x128", "64x64"), ((10, 10, 64, 641, 0, 1, 32, 1693), "128x128", "64x64"),
         ((10, 3, 128, 256, 1, 1, 64, 900), "64x128", "32x128"), ((6, 6, 128, 1, 2, 0, 30, 1693), "64x128", "32x128")]

# the two sides of each limit of a route
EDGES = {
    "bf16": [((32, 2184, 1920), "few"), ((32, 2185, 1920), "64x64"), ((23552, 256, 1920), "64x128"), ((23553, 256, 1920), "tiles"),
             ((10240, 256, 4096), "128x128"), ((10241, 256, 4112), "tiles")],
    "int8": [((32, 4369, 1920), "few"), ((32, 4370, 1920), "64x64"), ((30720, 256, 1920), "128x128"), ((30721, 256, 1920), "tiles"),
             ((14336, 256, 4096), "128x128"), ((14337, 256, 4112), "tiles")],
    "nvfp4": [((32, 2184, 1920), "few"), ((32, 2185, 1920), "64x64"), ((15360, 256, 1920), "64x64"), ((15361, 256, 1920), "tiles"),
              ((6144, 256, 4096), "64x64"), ((6145, 256, 4112), "tiles")],
}

# a shape of each of the larger paths, for what every epilogue has code of its own for
MIDDLING, WHOLE = (900, 1920, 208), (2900, 2904, 208)
# long enough in K that the tiles of the last round are split where there is a workspace
SPLIT = (2500, 1416, 4224)
# (rows in all, some of them, N, K): the first take one path, the second another
ACROSS = [((64, 16, 2185, 1920), "64x64", "few"), ((30721, 900, 256, 1920), "tiles", "64x64")]

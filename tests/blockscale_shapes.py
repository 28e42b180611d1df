"""Shapes (m, n, k) that reach every kernel of fp8_gemm_blockscale on 256
compute units: the kernel's value (fp8_gemm_blockscale_kernel) -> shapes.
N is odd or not a multiple of 8, the last tile of rows ragged, and for the
waves that split K there are more K blocks than waves and the last is ragged."""
from gemv_nvfp4_int8_amd import (QP_BLOCKSCALE_KSPLIT, QP_BLOCKSCALE_TILES_128, QP_BLOCKSCALE_TILES_256,
                                 QP_BLOCKSCALE_TILES_256_QUARTERS)

# numbers of K blocks: every remainder by the ring's five slots; the last block
# whole or ragged; 24 blocks, a multiple of most of what the kernels step by
TILES = {
    QP_BLOCKSCALE_TILES_128: [
        (1017, 1007, 128), (1001, 1007, 16), (1000, 1006, 256), (1003, 1002, 160), (1009, 1009, 384),
        (1004, 1019, 272), (1018, 1010, 512), (1005, 1013, 400), (1010, 1005, 640), (1007, 1002, 528),
        (1007, 1027, 768), (1005, 1030, 656), (1003, 1011, 896), (1003, 1004, 784), (1266, 739, 1024),
        (1006, 1006, 944), (1100, 1020, 1152), (1367, 797, 1040), (1224, 1003, 1280), (1093, 1126, 1168),
        (1157, 1041, 3056)],
    QP_BLOCKSCALE_TILES_256: [
        (11009, 7050, 128), (11009, 7050, 112), (3713, 11927, 256), (3713, 11927, 240), (4867, 5787, 384),
        (4871, 5789, 272), (5780, 4887, 512), (5023, 5651, 400), (3852, 3074, 640), (4374, 2692, 528),
        (2689, 4391, 768), (2708, 4387, 656), (4370, 2700, 896), (4355, 2701, 784), (2436, 4873, 1024),
        (4354, 2717, 912), (4353, 2717, 1152), (4381, 2699, 1040), (2705, 4369, 1280), (3099, 3852, 1168),
        (2708, 4387, 3056), (2816, 4480, 1024)],
    QP_BLOCKSCALE_TILES_256_QUARTERS: [
        (5665, 5851, 768), (5647, 5843, 656), (5941, 5509, 896), (5783, 5641, 784), (5911, 5505, 1024),
        (5637, 5782, 912), (5763, 5668, 1152), (5774, 5662, 1040), (5511, 5895, 1280), (5663, 5819, 1168),
        (4090, 4099, 2064)],
}

# (rows of A in 16s, rows of W in 16s): shape, and the shape that reads a
# weight past the caches
_KSPLIT = {
    (1, 1): [(1, 1, 1168), (1, 2004, 33488)], (2, 1): [(308, 197, 1184), (18, 3730, 72176)],
    (3, 1): [(277, 459, 1168), (34, 3030, 88640)], (4, 1): [(623, 394, 1184), (52, 4068, 66320)],
    (1, 2): [(292, 217, 1168), (1, 4454, 15072)], (2, 2): [(493, 369, 1168), (17, 7980, 33680)],
    (3, 2): [(644, 385, 1184), (34, 4754, 56640)], (4, 2): [(585, 629, 1168), (49, 7431, 36576)],
    (1, 3): [(291, 622, 1168), (1, 21636, 3104)], (2, 3): [(581, 458, 1200), (17, 11601, 23152)],
    (3, 3): [(581, 801, 1200), (35, 11348, 23744)], (4, 3): [(825, 743, 1168), (49, 9956, 26992)],
    (1, 5): [(66, 2771, 1168), (4, 17408, 5120)], (2, 5): [(874, 634, 1168), (17, 15277, 17600)],
    (3, 5): [(783, 924, 1168), (34, 17730, 15184)], (4, 5): [(1348, 674, 1200), (49, 18781, 14352)],
}
KSPLIT = {QP_BLOCKSCALE_KSPLIT + mt + 8 * nt + 64 * once: [shapes[once]]
          for (mt, nt), shapes in _KSPLIT.items() for once in (0, 1)}
KSPLIT[QP_BLOCKSCALE_KSPLIT + 1 + 8 * 1] += [(5, 260, 3056), (40, 163, 3040)]
KSPLIT[QP_BLOCKSCALE_KSPLIT + 1 + 8 * 5 + 64] += [(16, 25898, 2592)]

ALL = [(kernel, shape) for table in (TILES, KSPLIT) for kernel, shapes in table.items() for shape in shapes]

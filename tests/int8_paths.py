"""Sizes that reach every kernel and tile of the 8-bit products and input
gradients, and the path that each of them takes.  The dispatch rule is an
estimate: the CPU test asks it for every size here, so that another fit of it
cannot leave a path untested unseen."""
import ctypes
import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "group_wise_minmax_amd", "csrc")

# path, m, k, channels of each weight.  "short": k_i8_skinny, channels x tokens;
# the rest k_i8_gemm: 256 x 256 tiles, pieces, pieces with K split over
# workgroups ("odd": ranges of an odd number of 64 codes).  (None is short enough
# for k_i8_decode, which takes every product of 4 tokens or fewer with few codes.)
PRODUCTS = [
    ("short 16x16", 5, 2048, (513,)), ("short 16x16", 7, 5952, (4705,)), ("short 16x16", 20, 1088, (70, 33)),
    ("short 32x16", 9, 1024, (5001,)), ("short 32x16", 9, 4544, (8841,)), ("short 32x16", 16, 512, (9001, 130)),
    ("short 64x16", 36, 64, (4369,)), ("short 64x16", 39, 5952, (5079,)), ("short 64x16", 43, 4608, (2976, 1878, 247)),
    ("short 32x32", 100, 1024, (1001,)), ("short 32x32", 95, 4288, (1907,)), ("short 32x32", 1361, 64, (13, 11, 4)),
    ("short 64x32", 24, 1088, (9001,)), ("short 64x32", 172, 4544, (2369,)), ("short 64x32", 30, 2048, (9001, 70)),
    ("short 64x64", 600, 1088, (1001,)), ("short 64x64", 141, 5440, (4685,)), ("short 64x64", 520, 1024, (701, 300)),
    ("pieces 128x128", 333, 2048, (4001, 1025)), ("pieces 128x128", 333, 1024, (4001,)),
    ("pieces 128x128 odd", 257, 4160, (4101,)), ("pieces 128x128 odd", 67, 64, (5467,)),
    ("pieces 128x128 odd", 520, 1088, (5001, 1030)),
    ("split 128x128", 333, 8192, (1025,)), ("split 128x128", 130, 8192, (2001,)),
    ("split 128x128", 40, 16384, (2001, 1030)), ("split 128x128 odd", 70, 16448, (1500,)),
    ("pieces 128x256", 532, 128, (6535,)), ("pieces 128x256", 2048, 1088, (4001,)),
    ("pieces 128x256", 2000, 448, (3001,)), ("pieces 128x256", 5419, 64, (481, 10, 12)),
    ("tiles", 4609, 320, (2647,)), ("tiles", 4227, 384, (1861, 792, 23)), ("tiles", 2100, 4096, (14336,)),
    ("tiles and 128x256", 2614, 448, (8031,)), ("tiles and 128x256", 3300, 1024, (7001,)),
    ("tiles and 128x256", 3117, 384, (21, 3675, 2799)),
    ("tiles and 128x128", 4097, 192, (4101,)), ("tiles and 128x128", 4096, 1024, (8193,)),
    ("tiles and 128x128", 4400, 1024, (2048, 2101)),
]

# path, m, k, rows of each weight.  "short": k_i8_dx by its tokens, "ranges" where
# its reduction is split over workgroups; the rest k_bwd_dx's tiles, columns x
# tokens ("cut": whole rounds of 256 x 256 and the remaining columns in 128 x 128).
GRADIENTS = [
    ("short 16", 3, 64, (8,)), ("short 16 ranges", 1, 64, (1104,)), ("short 16 ranges", 1, 64, (32, 24, 1096)),
    ("short 32", 17, 8256, (8,)), ("short 32 ranges", 20, 1024, (4096, 1000)), ("short 32 ranges", 19, 1216, (1904,)),
    ("short 64", 300, 4096, (4096,)), ("short 64 ranges", 33, 2368, (3128,)), ("short 64 ranges", 40, 4096, (4096,)),
    ("tiles 128x128", 129, 16384, (1000,)), ("tiles 128x128", 200, 8192, (200, 72)), ("tiles 128x128", 1000, 4096, (2000,)),
    ("tiles 256x256", 4000, 4096, (328,)), ("tiles 256x256", 2000, 4160, (264, 136)),
    ("tiles 256x256", 1202, 10816, (8, 40, 24)),
    ("tiles 256x256 cut", 2304, 14336, (328,)), ("tiles 256x256 cut", 2304, 14336, (200, 72)),
    ("tiles 256x256 cut", 4509, 6336, (200,)),
    ("tiles 256x128", 2048, 4096, (1000, 72, 200)),
] + [("tiles 256x128", 1100, 4096, (n,)) for n in (72, 136, 200, 264, 328, 392, 456)]  # 2 to 8 steps of 64 rows

# The same for one weight with an adapter (its rows come by 64).
ADAPTED_GRADIENTS = [
    ("short 16 ranges", 1, 64, (1152,)), ("short 32 ranges", 19, 1216, (1920,)), ("short 64 ranges", 40, 4096, (4096,)),
    ("short 64", 300, 4096, (4096,)), ("tiles 128x128", 129, 16384, (1024,)), ("tiles 256x128", 1100, 4096, (448,)),
    ("tiles 256x256", 4000, 4096, (320,)), ("tiles 256x256 cut", 2304, 14336, (320,)),
]

PRODUCT_PATHS = {f"short {a}x{b}" for a, b in ((16, 16), (32, 16), (64, 16), (32, 32), (64, 32), (64, 64))} | {
    "pieces 128x128", "pieces 128x128 odd", "split 128x128", "split 128x128 odd", "pieces 128x256", "tiles",
    "tiles and 128x256", "tiles and 128x128"}
GRADIENT_PATHS = {f"short {t}{r}" for t in (16, 32, 64) for r in ("", " ranges")} | {
    "tiles 128x128", "tiles 256x128", "tiles 256x256", "tiles 256x256 cut"}


def named(case):
    path, m, k, ns = case
    return f"{path}, {m}x{k}x{'+'.join(map(str, ns))}"


def build_rule(where):
    """The dispatch rule as a library for the host, built into the folder `where`."""
    out = os.path.join(str(where), "i8_choice.so")
    cxx = shutil.which("g++") or shutil.which("clang++") or "/opt/rocm/llvm/bin/clang++"
    subprocess.run([cxx, "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, os.path.join(HERE, "i8_choice.cpp"), "-o", out],
                   check=True)
    return ctypes.CDLL(out)


def decodes(rule, m, k):
    return bool(rule.i8_decodes(ctypes.c_int64(m), ctypes.c_int64(k)))


def _ask(f, m, k, ns, split, size):
    out = (ctypes.c_int64 * size)()
    f((ctypes.c_int64 * len(ns))(*ns), len(ns), ctypes.c_int64(k), ctypes.c_int64(m), int(split), out)
    return list(out)


def product_path(rule, m, k, ns, split=True):
    tn, tm, whole, cut, ks, per, rest = _ask(rule.i8_product_path, m, k, ns, split, 7)
    if tn:
        return f"short {16 * tn}x{16 * tm}"
    piece = "128x256" if cut == 2 else "128x128"
    if whole:
        return f"tiles and {piece}" if rest else "tiles"
    return ("split " if ks > 1 else "pieces ") + piece + (" odd" if cut == 4 and per % 2 else "")


def gradient_path(rule, m, k, ns, split=True):
    tm, ks, _, bk, bm = _ask(rule.i8_gradient_path, m, k, ns, split, 5)
    if tm:
        return f"short {16 * tm}" + (" ranges" if ks > 1 else "")
    # several rounds of 256 x 256 tiles: the columns that fill whole ones
    rows = -(-m // 256)
    tiles = -(-k // 256) * rows
    columns = tiles // 256 * 256 // rows * 256
    cut = bk == bm == 256 and tiles > 256 and tiles % 256 != 0 and 0 < columns < k
    return f"tiles {bk}x{bm}" + (" cut" if cut else "")

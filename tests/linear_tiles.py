"""Sizes of the matrix product that take every tile of every type, and what csrc/ssd_linear_plan.h says of them."""
import os
import shutil
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mamba_ssd_prefill_amd", "csrc")
TYPES = ("f32", "f16", "bf16", "int8", "e4m3")
SHAPES = [(128, 128), (256, 256), (128, 192), (256, 160), (256, 128), (64, 128), (32, 64), (16, 64), (128, 128)]

# (rows, width, outs, type, tile, loads of 4 bytes, splits of the contraction): each more than a tile in both directions and no
# multiple of it, over several turns of the pipeline and a part of a step
PRODUCTS = [
    (3080, 268, 2050, "f32", 0, False, 1), (10328, 2856, 196, "f32", 0, False, 3), (3080, 268, 4099, "f32", 1, False, 1),
    (6905, 7080, 710, "f32", 1, False, 3), (8200, 268, 450, "f32", 2, False, 1), (3080, 268, 2565, "f32", 3, False, 1),
    (5130, 3180, 450, "f32", 3, False, 4), (6150, 268, 130, "f32", 5, False, 1), (1030, 1676, 450, "f32", 5, False, 3),
    (6150, 269, 130, "f32", 5, True, 1), (1030, 1677, 450, "f32", 5, True, 3), (2050, 652, 65, "f32", 6, False, 1),
    (390, 1036, 65, "f32", 6, False, 6), (2050, 653, 65, "f32", 6, True, 1), (390, 1037, 65, "f32", 6, True, 6),
    (17, 652, 65, "f32", 7, False, 1), (17, 844, 65, "f32", 7, False, 6), (17, 653, 65, "f32", 7, True, 1),
    (17, 845, 65, "f32", 7, True, 6), (200, 536, 16390, "f16", 0, False, 1), (6150, 4888, 257, "f16", 0, False, 3),
    (3080, 536, 4099, "f16", 1, False, 1), (777, 9560, 5125, "f16", 1, False, 3), (200, 1304, 16390, "f16", 2, False, 1),
    (515, 51160, 517, "f16", 2, False, 16), (390, 536, 16390, "f16", 3, False, 1), (4100, 12760, 257, "f16", 3, False, 6),
    (390, 3352, 12301, "f16", 4, False, 1), (6150, 12760, 257, "f16", 4, False, 3), (6150, 536, 130, "f16", 5, False, 1),
    (259, 12760, 257, "f16", 5, False, 16), (6150, 538, 130, "f16", 5, True, 1), (259, 12762, 257, "f16", 5, True, 16),
    (2050, 1304, 65, "f16", 6, False, 1), (390, 2072, 65, "f16", 6, False, 6), (2050, 1306, 65, "f16", 6, True, 1),
    (390, 2074, 65, "f16", 6, True, 6), (17, 1304, 65, "f16", 7, False, 1), (17, 2072, 65, "f16", 7, False, 6),
    (17, 1306, 65, "f16", 7, True, 1), (17, 2074, 65, "f16", 7, True, 6), (8200, 1176, 130, "f16", 8, False, 1),
    (1030, 12760, 130, "f16", 8, False, 12), (200, 536, 16390, "bf16", 0, False, 1), (6150, 4888, 257, "bf16", 0, False, 3),
    (3080, 536, 4099, "bf16", 1, False, 1), (777, 9560, 5125, "bf16", 1, False, 3), (200, 1304, 16390, "bf16", 2, False, 1),
    (515, 51160, 517, "bf16", 2, False, 16), (390, 536, 16390, "bf16", 3, False, 1),
    (4100, 12760, 257, "bf16", 3, False, 6), (390, 3352, 12301, "bf16", 4, False, 1),
    (6150, 12760, 257, "bf16", 4, False, 3), (6150, 536, 130, "bf16", 5, False, 1), (259, 12760, 257, "bf16", 5, False, 16),
    (6150, 538, 130, "bf16", 5, True, 1), (259, 12762, 257, "bf16", 5, True, 16), (2050, 1304, 65, "bf16", 6, False, 1),
    (390, 2072, 65, "bf16", 6, False, 6), (2050, 1306, 65, "bf16", 6, True, 1), (390, 2074, 65, "bf16", 6, True, 6),
    (17, 1304, 65, "bf16", 7, False, 1), (17, 2072, 65, "bf16", 7, False, 6), (17, 1306, 65, "bf16", 7, True, 1),
    (17, 2074, 65, "bf16", 7, True, 6), (8200, 1176, 130, "bf16", 8, False, 1), (1030, 12760, 130, "bf16", 8, False, 12),
    (200, 1072, 16390, "int8", 0, False, 1), (6150, 9776, 257, "int8", 0, False, 3),
    (3080, 1072, 4099, "int8", 1, False, 1), (777, 19120, 5125, "int8", 1, False, 3),
    (200, 2608, 16390, "int8", 2, False, 1), (515, 102320, 517, "int8", 2, False, 16),
    (390, 1072, 16390, "int8", 3, False, 1), (4100, 25520, 257, "int8", 3, False, 6),
    (390, 6704, 12301, "int8", 4, False, 1), (6150, 25520, 257, "int8", 4, False, 3),
    (2050, 1072, 450, "int8", 5, False, 1), (259, 25520, 257, "int8", 5, False, 16), (2050, 1076, 450, "int8", 5, True, 1),
    (259, 25524, 257, "int8", 5, True, 16), (2050, 2608, 65, "int8", 6, False, 1), (390, 4144, 65, "int8", 6, False, 6),
    (2050, 2612, 65, "int8", 6, True, 1), (390, 4148, 65, "int8", 6, True, 6), (17, 2608, 65, "int8", 7, False, 1),
    (17, 4144, 65, "int8", 7, False, 6), (17, 2612, 65, "int8", 7, True, 1), (17, 4148, 65, "int8", 7, True, 6),
    (8200, 2352, 130, "int8", 8, False, 1), (1030, 25520, 130, "int8", 8, False, 12),
    (200, 1072, 16390, "e4m3", 0, False, 1), (6150, 9776, 257, "e4m3", 0, False, 3),
    (3080, 1072, 4099, "e4m3", 1, False, 1), (777, 19120, 5125, "e4m3", 1, False, 3),
    (200, 2608, 16390, "e4m3", 2, False, 1), (515, 102320, 517, "e4m3", 2, False, 16),
    (390, 1072, 16390, "e4m3", 3, False, 1), (4100, 25520, 257, "e4m3", 3, False, 6),
    (390, 6704, 12301, "e4m3", 4, False, 1), (6150, 25520, 257, "e4m3", 4, False, 3),
    (2050, 1072, 450, "e4m3", 5, False, 1), (259, 25520, 257, "e4m3", 5, False, 16), (2050, 1076, 450, "e4m3", 5, True, 1),
    (259, 25524, 257, "e4m3", 5, True, 16), (2050, 2608, 65, "e4m3", 6, False, 1), (390, 4144, 65, "e4m3", 6, False, 6),
    (2050, 2612, 65, "e4m3", 6, True, 1), (390, 4148, 65, "e4m3", 6, True, 6), (17, 2608, 65, "e4m3", 7, False, 1),
    (17, 4144, 65, "e4m3", 7, False, 6), (17, 2612, 65, "e4m3", 7, True, 1), (17, 4148, 65, "e4m3", 7, True, 6),
    (8200, 2352, 130, "e4m3", 8, False, 1), (1030, 25520, 130, "e4m3", 8, False, 12),
]
# (rows, width, outs, type, tile of both products' launch)
GRADIENTS = [
    (294, 9872, 291, "f32", 0), (626, 10704, 613, "f32", 1), (130, 11944, 168, "f32", 2), (394, 10068, 385, "f32", 3),
    (429, 10628, 808, "f32", 4), (259, 2050, 257, "f32", 5), (259, 517, 257, "f32", 6), (259, 33, 257, "f32", 7),
    (515, 4099, 517, "f16", 0), (515, 10570, 517, "f16", 1), (1300, 2050, 771, "f16", 2), (600, 6153, 650, "f16", 3),
    (3080, 771, 4099, "f16", 4), (515, 1030, 517, "f16", 5), (515, 65, 1541, "f16", 6), (515, 33, 517, "f16", 7),
    (515, 1541, 1030, "f16", 8), (515, 4099, 517, "bf16", 0), (515, 10570, 517, "bf16", 1), (1300, 2050, 771, "bf16", 2),
    (600, 6153, 650, "bf16", 3), (3080, 771, 4099, "bf16", 4), (515, 1030, 517, "bf16", 5), (515, 65, 1541, "bf16", 6),
    (515, 33, 517, "bf16", 7), (515, 1541, 1030, "bf16", 8),
]

PROGRAM = r"""
#include <stdio.h>
#include "ssd_linear_plan.h"
int main() {
    char what;
    long M, K, N, stride;
    int type;
    while (scanf(" %c %ld %ld %ld %ld %d", &what, &M, &K, &N, &stride, &type) == 6) {
        const size_t es = type == ssd::LT_F32 ? 4 : type <= ssd::LT_BF16 ? 2 : 1;
        const ssd::LinearPlan p = what == 'p' ? ssd::linear_form(M, K, N, stride, type, es).plan
                                              : ssd::linear_back_form(M, K, N, type, es).both_plan;
        printf("%d %d %d\n", p.tile, (int)p.narrow, p.splits);
    }
}
"""


def compiler():
    return shutil.which("g++")


def plans(folder, sizes):
    """(tile, loads of 4 bytes, splits) of each ("p" product or "g" gradients, rows, width, outs, type) by the header."""
    src, exe = os.path.join(folder, "plan.cpp"), os.path.join(folder, "plan")
    if not os.path.exists(exe):
        with open(src, "w") as f:
            f.write(PROGRAM)
        subprocess.run([compiler(), "-O2", "-std=c++17", "-I", CSRC, src, "-o", exe], check=True)
    text = "".join("%s %d %d %d 0 %d\n" % (what, M, K, N, TYPES.index(t)) for what, M, K, N, t in sizes)
    out = subprocess.run([exe], input=text.encode(), stdout=subprocess.PIPE, check=True).stdout.split()
    return [(int(a), bool(int(b)), int(c)) for a, b, c in zip(out[::3], out[1::3], out[2::3])]

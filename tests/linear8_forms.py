"""Sizes of the 8-bit products by the form of the tile kernels that runs them.

A form: the product, tile, wave groups that share K, operands read through
registers because they are unaligned, operands laid out again first, and how
the tiles are divided ("direct": one workgroup each, "split": several along K
each, "mixed": some and some).  Every size has ragged ends on all three axes
and at least eight stages of K per wave group, more than a ring holds, so that
each kernel's main loop, its last stages and its way out are all run.
"""
import ctypes
from typing import NamedTuple

from matrix_aware_optimizer_muon_amd._lib import load

PAD = 16  # elements between rows, so that what lies past a row's end is known


class Form(NamedTuple):
    product: int      # 0 matmul, 1 grad_input, 2 grad_weight
    tile: int
    groups: int
    unaligned: bool
    packed: bool
    division: str


FORMS = {
    Form(0, 64, 4, False, False, "direct"): (71, 74, 2352),
    Form(0, 64, 4, False, False, "split"): (69, 2092, 7280),
    Form(0, 64, 4, True, False, "direct"): (67, 68, 2362),
    Form(0, 64, 4, True, False, "split"): (66, 2056, 7069),
    Form(0, 128, 1, False, False, "direct"): (262, 11170, 528),
    Form(0, 128, 1, False, False, "mixed"): (5788, 2928, 1840),
    Form(0, 128, 1, True, False, "direct"): (11200, 270, 540),
    Form(0, 128, 1, True, False, "mixed"): (658, 11685, 3755),
    Form(0, 128, 2, False, False, "direct"): (130, 5648, 1184),
    Form(0, 128, 2, False, False, "split"): (208, 4308, 3888),
    Form(0, 128, 2, True, False, "direct"): (136, 5600, 1163),
    Form(0, 128, 2, True, False, "split"): (5656, 133, 3203),
    Form(0, 256, 1, False, False, "direct"): (9386, 787, 544),
    Form(0, 256, 1, False, False, "mixed"): (1459, 11652, 1760),
    Form(0, 256, 1, False, False, "split"): (8352, 392, 8112),
    Form(0, 256, 1, False, True, "direct"): (11456, 659, 520),
    Form(0, 256, 1, False, True, "mixed"): (2617, 6347, 1731),
    Form(0, 256, 1, False, True, "split"): (1568, 2488, 6200),
    Form(1, 64, 4, False, False, "direct"): (72, 1200, 65),
    Form(1, 64, 4, False, False, "split"): (2691, 2640, 66),
    Form(1, 64, 4, True, False, "direct"): (80, 1197, 68),
    Form(1, 64, 4, True, False, "split"): (68, 2565, 2728),
    Form(1, 128, 1, False, False, "direct"): (11347, 264, 272),
    Form(1, 128, 1, False, False, "mixed"): (10665, 888, 1552),
    Form(1, 128, 1, True, False, "direct"): (11496, 262, 272),
    Form(1, 128, 1, True, False, "mixed"): (10241, 911, 788),
    Form(1, 128, 2, False, False, "direct"): (5844, 592, 129),
    Form(1, 128, 2, False, False, "split"): (196, 1840, 4416),
    Form(1, 128, 2, True, False, "direct"): (5783, 578, 133),
    Form(1, 128, 2, True, False, "split"): (4239, 1738, 197),
    Form(1, 256, 1, False, False, "direct"): (11232, 264, 644),
    Form(1, 256, 1, False, False, "mixed"): (11600, 904, 1426),
    Form(1, 256, 1, False, False, "split"): (403, 7792, 4272),
    Form(1, 256, 1, False, True, "direct"): (656, 265, 10944),
    Form(1, 256, 1, False, True, "mixed"): (1960, 1185, 8692),
    Form(1, 256, 1, False, True, "split"): (400, 4380, 8577),
    Form(2, 64, 4, False, False, "direct"): (1231, 72, 72),
    Form(2, 64, 4, False, False, "split"): (3472, 2064, 68),
    Form(2, 64, 4, True, False, "direct"): (1196, 70, 65),
    Form(2, 64, 4, True, False, "split"): (2576, 69, 2843),
    Form(2, 128, 1, False, False, "direct"): (262, 11440, 272),
    Form(2, 128, 1, False, False, "mixed"): (912, 1600, 10467),
    Form(2, 128, 1, True, False, "direct"): (264, 261, 11270),
    Form(2, 128, 1, True, False, "mixed"): (893, 7951, 1056),
    Form(2, 128, 2, False, False, "direct"): (592, 144, 5593),
    Form(2, 128, 2, False, False, "split"): (1861, 200, 4218),
    Form(2, 128, 2, True, False, "direct"): (601, 133, 5952),
    Form(2, 128, 2, True, False, "split"): (1865, 193, 4277),
    Form(2, 256, 1, False, False, "direct"): (272, 656, 10896),
    Form(2, 256, 1, False, False, "mixed"): (921, 11584, 1433),
    Form(2, 256, 1, False, False, "split"): (3887, 8680, 396),
    Form(2, 256, 1, False, True, "direct"): (264, 669, 11062),
    Form(2, 256, 1, False, True, "mixed"): (1473, 1435, 11680),
    Form(2, 256, 1, False, True, "split"): (4254, 405, 8944),
}


def choice(kind, t, n, k, pad=PAD):
    """(form or None for the few-rows kernel, stages of the whole sum, splits)
    of operands at aligned addresses with `pad` elements between their rows."""
    f = load().muon_l8_choice
    P, I, L = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    f.argtypes, f.restype = [I, P, L, P, L, L, L, L, P], None
    v = (L * 10)()
    f(kind, 0, (k if kind == 0 else n) + pad, 0, k + pad, t, n, k, v)
    few, tile, groups, unaligned, pack_a, pack_b, direct, split, splits, stages = v
    if few:
        return None, stages, 1
    division = "direct" if split == 0 else "mixed" if direct else "split"
    return Form(kind, tile, groups, bool(unaligned), bool(pack_a or pack_b), division), stages, splits

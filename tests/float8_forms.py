"""One size for each form that a product of the 8-bit floating-point layer can
take (csrc/float8.h, muon_f8_choice): its kernel, tile, wave groups, a gradient's
dy laid out again, and whether tiles are whole, split along K, or both."""
from float8_common import MATMUL, choice

P = 1 << 20

# (product, bf16, experts or 0, t, n, k); widths and sums that end inside tiles,
# stages and chunks
SIZES = [
    (0, 1, 0, 13, 333, 1111), (0, 0, 0, 11, 300, 701), (0, 1, 0, 29, 333, 1111), (0, 0, 0, 30, 300, 701),
    (0, 1, 9, 9, 333, 1111), (0, 0, 9, 9, 300, 701),
    (0, 1, 0, 40, 150, 610), (0, 0, 0, 40, 150, 693), (0, 1, 0, 37, 100, 2693), (0, 0, 0, 35, 94, 2666),
    (0, 1, 0, 65, 8565, 682), (0, 0, 0, 886, 1156, 619), (0, 1, 0, 34, 66, 3332), (0, 0, 0, 795, 1280, 2820),
    (0, 1, 0, 3776, 1030, 678), (0, 0, 0, 6595, 591, 646), (0, 1, 0, 2681, 3200, 3380), (0, 0, 0, 3425, 2365, 785),
    (0, 1, 0, 5952, 1418, 645), (0, 1, 0, 4754, 6882, 698), (0, 1, 7, 1000, 300, 605), (0, 0, 7, 1000, 300, 613),
    (0, 1, 18, 5390, 1724, 313),
    (1, 0, 0, 70, 288, 100), (1, 1, 0, 70, 276, 100), (1, 0, 0, 50, 1520, 99), (1, 1, 0, 50, 1454, 99),
    (1, 1, 0, 915, 344, 1259), (1, 0, 0, 129, 274, 5668), (1, 0, 0, 67, 1864, 8208), (1, 1, 0, 8209, 1961, 68),
    (1, 0, 0, 1147, 280, 3651), (1, 1, 0, 8531, 287, 396), (1, 0, 0, 2432, 2112, 3352), (1, 0, 0, 3345, 1618, 2431),
    (1, 0, 0, 7065, 280, 1216), (1, 0, 0, 2919, 271, 2905), (1, 0, 0, 4258, 752, 4032), (1, 1, 0, 2560, 415, 6617),
    (1, 1, 0, 2816, 8448, 711), (1, 1, 0, 8738, 8023, 133),
    (1, 0, 5, 300, 328, 130), (1, 1, 5, 300, 335, 131), (1, 1, 49, 6912, 288, 960), (1, 0, 9, 2300, 292, 3333),
    (2, 0, 0, 310, 80, 100), (2, 1, 0, 275, 81, 100), (2, 1, 0, 1805, 72, 66), (2, 1, 0, 1984, 66, 8303),
    (2, 0, 0, 321, 144, 5917), (2, 0, 0, 285, 325, 2700), (2, 1, 0, 1864, 8200, 66), (2, 1, 0, 4677, 193, 1458),
    (2, 1, 0, 273, 2000, 2137), (2, 1, 0, 273, 3253, 1285), (2, 1, 0, 2880, 1088, 7433), (2, 1, 0, 1387, 7241, 1078),
    (2, 0, 0, 320, 1624, 5120), (2, 0, 0, 320, 3217, 2491), (2, 0, 0, 604, 5632, 3028), (2, 0, 0, 384, 6619, 2508),
    (2, 1, 0, 4160, 8960, 403), (2, 1, 0, 3840, 443, 8448),
    (2, 1, 3, 326, 88, 77), (2, 0, 3, 313, 81, 77), (2, 0, 11, 33, 4376, 130), (2, 1, 11, 33, 4011, 129),
    (2, 0, 8, 1500, 1064, 2100), (2, 1, 8, 1500, 1091, 2100), (2, 1, 4, 700, 1928, 4001),
]


def every_form():
    """Kinds as csrc/float8.h numbers them: the forward product of bf16 and fp32
    results, the input and the weight gradient."""
    forms = {("few", 16, grouped, kind) for grouped in (False, True) for kind in (0, 1)}
    forms |= {("few", 32, False, kind) for kind in (0, 1)}
    for kind in range(4):
        for pack in (0, 1) if kind > 1 else (0,):
            forms |= {(kind, 64, 4, pack, "whole"), (kind, 64, 4, pack, "split"), (kind, 128, 2, pack, "whole"),
                      (kind, 128, 2, pack, "split"), (kind, 128, 1, pack, "whole"), (kind, 128, 1, pack, "mixed"),
                      (kind, 128, 1, pack, "grouped")}
            if kind != 1:  # (fp32 results take no 256-wide tiles)
                forms |= {(kind, 256, 1, pack, "whole"), (kind, 256, 1, pack, "mixed"), (kind, 256, 1, pack, "grouped")}
            if kind > 1:
                forms.add((kind, 256, 1, pack, "split"))
    return forms


def form(product, bf16, experts, t, n, k, a=P):
    lda = (k + 15) // 16 * 16 if product == MATMUL else n
    c = choice(product, a, lda, experts > 0, max(experts, 1), t, n, k, bf16)
    if c["few"]:
        return ("few", c["few"], experts > 0, c["kind"])
    tiles = "grouped" if experts else "split" if c["split"] and c["splits"] > 1 and not c["direct"] else \
        "mixed" if c["splits"] > 1 else "whole"
    return (c["kind"], c["tile"], c["groups"], c["pack"], tiles)

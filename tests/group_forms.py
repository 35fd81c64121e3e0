"""Products grouped by expert for each way the library does them: rows of each group, cin, cout, and the form
(kernel for few rows, rows and columns of a tile, whole 16-byte accesses) of each product that it is there for."""

FEW16, FEW16_LOOSE, FEW32, FEW32_LOOSE = (True, 16, 128, True), (True, 16, 128, False), (True, 32, 128, True), (True, 32, 128, False)
LOOSE, SMALL, MIDDLE, LARGE = (False, 128, 128, False), (False, 128, 128, True), (False, 192, 256, True), (False, 256, 256, True)
ROWWISE = ("fwd", "glu", "dgrad", "glu_dgrad")  # a result for each grouped row


def rowwise(form, **others):
    return dict(dict.fromkeys(ROWWISE, form), **others)


FORMS = [
    ("few", [3, 0, 7], 64, 128, rowwise(FEW16)),
    ("few_loose", [5, 9, 1], 77, 133, rowwise(FEW16_LOOSE)),
    ("few_long", [48, 60, 33], 256, 192, rowwise(FEW32)),
    ("few_long_loose", [40, 30, 35], 77, 133, rowwise(FEW32_LOOSE)),
    ("few_long_narrow", [40, 0, 80, 35], 5, 3, rowwise(FEW32_LOOSE)),
    ("loose", [300, 200], 77, 133, rowwise(LOOSE, wgrad=LOOSE)),
    ("loose_narrow", [300, 0, 200], 3, 6, rowwise(LOOSE, wgrad=LOOSE)),
    ("small", [300, 200], 64, 128, rowwise(SMALL, wgrad=SMALL)),
    ("middle", [600, 0, 1500], 264, 520, rowwise(MIDDLE, wgrad=SMALL)),
    ("large", [700, 0, 1200] * 24, 256, 264, rowwise(LARGE)),
    ("large_short", [700, 0, 1200] * 24, 256, 64, dict(dgrad=LARGE, glu_dgrad=SMALL)),
    ("large_wgrad", [40000, 7, 23000], 256, 256, dict(wgrad=LARGE)),
]

"""Sizes (M, K, N) of the FP8 projection with the kernels that its forward, d_x and d_w run.

("few", waves), ("batch", row blocks, column blocks), ("tile", its number, K split, last round in halves); fourth
for d_x and d_w in one launch: the first product and whether the second's last round is in halves."""


def tile(shape, split=False, half=False):
    return ("tile", shape, split, half)


CHOICES = [
    ((1, 16, 16), (("few", 8), ("few", 8), tile(4), None)),
    ((1, 16, 8208), (("few", 8), ("few", 16), tile(3), None)),
    ((1, 16528, 1168), (("few", 16), ("few", 8), tile(0, half=True), None)),
    ((2, 11376, 4128), (("batch", 1, 2), ("few", 16), tile(0), None)),
    ((15, 1424, 16), (("batch", 1, 1), ("few", 8), tile(4), None)),
    ((16, 2048, 7168), (("batch", 1, 2), ("batch", 1, 1), tile(0), None)),
    ((16, 7168, 4112), (("batch", 1, 2), ("batch", 1, 2), tile(0), None)),
    ((17, 4496, 2880), (tile(4, split=True), ("batch", 2, 2), tile(0), None)),
    ((30, 1040, 272), (("batch", 2, 1), ("batch", 2, 1), tile(4), None)),
    ((30, 4112, 48), (tile(5, split=True), ("batch", 2, 2), tile(4), None)),
    ((34, 16, 16544), (tile(3), tile(5, split=True), tile(2), None)),
    ((65, 11520, 7808), (tile(3, split=True), tile(1, split=True), tile(0, half=True), None)),
    ((67, 16, 16464), (tile(2), tile(5, split=True), tile(2), None)),
    ((129, 11072, 13744), (tile(1, split=True), tile(0, split=True), tile(0, half=True), None)),
    ((199, 10272, 8576), (tile(1, split=True), tile(1, split=True), tile(0, half=True), None)),
    ((300, 16, 16), (tile(5), tile(5), tile(4), None)),
    ((643, 160, 16608), (tile(0), tile(3, split=True), tile(1), None)),
    ((666, 400, 14048), (tile(0), tile(3, split=True), tile(1), None)),
    ((1409, 16, 16), (tile(5), tile(5), tile(4, split=True), None)),
    ((1443, 16, 13632), (tile(0, half=True), tile(3, split=True), tile(3), None)),
    ((1698, 16, 1168), (tile(2), tile(5), tile(3, split=True), None)),
    ((1896, 2032, 3120), (tile(1), tile(3), tile(1), None)),
    ((3370, 144, 144), (tile(4), tile(4), tile(4, split=True), None)),
    ((3657, 144, 608), (tile(2), tile(4), tile(4, split=True), None)),
    ((4373, 16, 8448), (tile(0, half=True), tile(3, split=True), tile(2, split=True), None)),
    ((6569, 6688, 16), (tile(2, split=True), tile(0), tile(4, split=True), None)),
    ((7865, 144, 5536), (tile(0), tile(3), tile(1, split=True), None)),
    ((329, 14144, 432), (tile(3, split=True), tile(0, half=True), tile(0, half=True), ("dx", True))),
    ((353, 11792, 352), (tile(3, split=True), tile(0, half=True), tile(0, half=True), ("dx", False))),
    ((419, 11216, 336), (tile(3, split=True), tile(0, half=True), tile(0, half=True), ("dw", False))),
    ((472, 14288, 336), (tile(3, split=True), tile(0, half=True), tile(0, half=True), ("dw", True))),
    ((2306, 5056, 2560), (tile(1), tile(0), tile(0), ("dx", False))),
    ((3383, 3152, 2800), (tile(0), tile(0), tile(0), ("dw", True))),
]

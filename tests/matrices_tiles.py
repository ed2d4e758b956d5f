"""Shapes that take each tile size, for the tests that run the kernels on them and the
one that asks the entry points which they take."""

# (m, n, k) of one product, the side of its tiles: ragged sides, several k tiles; long k (from 1024 on
# fewer tiles are enough) and short
PRODUCTS = [((2900, 2904, 320), 128), ((2050, 2600, 1088), 128), ((2100, 6200, 1024), 256), ((4100, 8008, 192), 256)]
# (side, k) of one gram
GRAMS = [((4000, 320), 128), ((3900, 1100), 128), ((5000, 1088), 256), ((8100, 192), 256)]
# (rows, cols, count) of a list for the momentum step, the sides of the tiles of S and its
# polynomial, and of X
STEPS = [((2450, 2600, 1), 128, 128), ((2700, 2500, 1), 128, 128), ((1100, 10000, 1), 64, 256), ((10000, 1100, 1), 64, 256),
         ((251, 683, 100), 64, 128), ((683, 251, 100), 64, 128), ((251, 683, 224), 128, 256), ((683, 251, 224), 128, 256),
         ((5000, 5100, 1), 256, 256)]

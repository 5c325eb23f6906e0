"""Sizes that take each form of the attention kernels, with the form that they are meant for."""

# lq of each sequence, lk - lq, Hq, Hkv, dh, window; 128-row units, pieces of the key axis, rows of a joining
# workgroup, row tiles in two orders
PACKED = [
    (([43], [8000], 24, 8, 128, 0), dict(qt=1, splits=16, join=4)),   # 129 rows of each key head: 4 and 1 left
    (([43], [8000], 24, 8, 64, 0), dict(qt=1, splits=16, join=4)),
    (([20, 23], [8000, 7000], 24, 8, 128, 0), dict(qt=1, splits=10, join=4)),
    (([43], [8000], 24, 8, 128, 4000), dict(qt=1, splits=13, join=4)),
    (([64, 36], [6000, 5000], 6, 2, 64, 0), dict(qt=1, splits=21, join=1)),
    (([5], [9000], 6, 2, 128, 0), dict(qt=1, splits=35, join=1)),
    (([300], [2000], 10, 5, 64, 0), dict(qt=1, splits=7, join=16)),
    (([90], [4000], 16, 8, 64, 1500), dict(qt=1, splits=5, join=16)),
    (([64, 1, 0, 33], [1900, 2500, 1000, 0], 4, 2, 128, 0), dict(qt=1, splits=5, join=8)),
    (([4200], [0], 30, 15, 128, 0), dict(qt=2, splits=1)),
    (([3000], [3000], 60, 30, 128, 2300), dict(qt=2, splits=1)),
    (([1000], [3000], 32, 32, 128, 2500), dict(qt=2, splits=2, join=8)),
    (([250], [4200], 64, 8, 128, 0), dict(qt=2, splits=4, join=8)),
    (([2200, 0, 1, 1500], [3000, 900, 2000, 3500], 48, 12, 128, 0), dict(qt=2, splits=1, longest=True)),
    (([700, 0, 1, 1500], [300, 900, 2000, 3500], 32, 16, 128, 900), dict(qt=1, splits=1, longest=True)),
    (([1030], [0], 32, 8, 128, 0), dict(qt=1, splits=1, reversed=True)),
    (([1000, 1040], [0, 50], 16, 4, 128, 0), dict(qt=1, splits=1, reversed=True)),
    (([3000], [0], 16, 8, 64, 0), dict(qt=1, splits=1, reversed=True)),
    (([1500, 1490], [0, 70], 16, 8, 64, 600), dict(qt=1, splits=1, reversed=True)),
    (([3100], [0], 32, 8, 64, 0), dict(qt=1, splits=1, reversed=False)),
]

# lengths, pages of the table, page size, Hq, Hkv, dh, window; waves of a workgroup, pieces, rows of a joining one
DECODE = [
    (([9590, 0, 1, 4000, 333], 150, 64, 208, 8, 128, 0), dict(waves=4, splits=9, join=4)),
    (([5990, 0, 1, 4000, 333], 375, 16, 208, 8, 64, 0), dict(waves=4, splits=11, join=4)),
    (([2995], 188, 16, 8, 2, 128, 1000), dict(waves=4, splits=7, join=8)),   # from token 1995: inside tile and page
    (([2995], 188, 16, 8, 2, 64, 1000), dict(waves=4, splits=7, join=16)),
    (([7000, 900], 500, 16, 4, 2, 64, 5001), dict(waves=4, splits=39, join=1)),
    (([1000, 0, 1, 999, 32, 33] + [7 * i for i in range(58)], 63, 16, 16, 8, 128, 0),
     dict(waves=2, splits=1)),
    (([1000, 0, 1, 999, 32, 33] + [7 * i for i in range(58)], 63, 16, 16, 8, 128, 801),
     dict(waves=2, splits=1)),
    (([2100, 0, 1, 2099, 1700, 33] + [9 * i for i in range(24)], 132, 16, 16, 8, 128, 0),
     dict(waves=2, splits=3, join=8)),
    (([2100, 0, 1, 2099, 1700, 33] + [9 * i for i in range(24)], 132, 16, 16, 8, 128, 1703),
     dict(waves=2, splits=3, join=8)),
    (([2100, 0, 1, 2099, 1700, 33], 132, 16, 160, 4, 128, 0), dict(waves=4, splits=6, join=8)),
    (([700, 0, 1, 699, 500, 33] + [9 * i for i in range(24)], 132, 16, 160, 4, 128, 0),
     dict(waves=2, splits=3, join=8)),                                       # 40 heads to a key head
]

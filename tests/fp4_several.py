"""Sizes of 4-bit products and of input gradients whose workgroups take several
tiles, one after the other (test helper): every tile that the plan gives such a
product, for both result types, with and without tiles in parts behind it.

(M, N, K, fp32 results, tile, tiles computed whole, tiles in parts, parts); of a
gradient, M x N is the result and K is summed over."""

FORWARD = [
    (10284, 2321, 768, False, 0, 410, 0, 1), (401, 52470, 700, False, 0, 410, 0, 1),
    (13617, 2050, 768, True, 0, 486, 0, 1), (405, 57469, 1255, True, 0, 450, 0, 1),
    (16384, 5760, 2880, False, 0, 1472, 0, 1), (49382, 1021, 2304, False, 0, 768, 4, 3),
    (968, 33620, 4608, True, 0, 512, 16, 6),
    (663, 22632, 768, False, 1, 356, 0, 1), (1180, 16434, 761, True, 1, 455, 0, 1),
    (10316, 4738, 2304, False, 1, 1024, 2, 3), (1775, 19631, 3584, True, 1, 768, 2, 4),
    (293, 45041, 3840, False, 2, 704, 0, 1), (13148, 795, 1024, True, 2, 483, 0, 1),
    (34271, 347, 7424, True, 2, 512, 25, 9),
    (608, 21874, 768, False, 3, 855, 0, 1), (454, 22812, 700, True, 3, 716, 0, 1),
    (52404, 637, 8960, False, 3, 2048, 2, 11),
    (58132, 80, 11520, False, 4, 455, 0, 1), (72, 59693, 9984, True, 4, 467, 0, 1),
    (292, 34897, 10752, False, 4, 768, 51, 5),
]
GRADIENT = [
    (12321, 1798, 192, False, 0, 392, 0, 1), (57344, 273, 150, True, 0, 448, 0, 1),
    (16384, 2880, 5760, False, 0, 768, 0, 1), (8867, 5531, 704, False, 0, 768, 2, 3),
    (1231, 39328, 550, True, 0, 768, 2, 3),
    (2344, 6849, 192, False, 1, 351, 0, 1), (2344, 6849, 191, True, 1, 351, 0, 1),
    (531, 44360, 1408, False, 1, 512, 10, 7), (531, 44360, 1350, True, 1, 512, 10, 7),
    (43959, 272, 1856, False, 2, 687, 0, 1), (13097, 1168, 896, True, 2, 690, 0, 1),
    (32882, 298, 4416, False, 2, 512, 4, 23), (32882, 298, 4400, True, 2, 512, 4, 23),
    (11059, 1284, 192, False, 3, 957, 0, 1), (11059, 1284, 190, True, 3, 957, 0, 1),
    (1634, 10041, 4928, False, 3, 1024, 3, 25), (627, 27833, 5760, True, 3, 1024, 66, 3),
    (8192, 2880, 2880, False, 3, 1472, 0, 1),
    (25620, 345, 10624, False, 4, 512, 91, 2), (25620, 345, 10600, True, 4, 512, 91, 2),
]
# From the codes, 64 rows of dY a workgroup: n in parts, rows of dY at eighths
DIRECT = [(256, 2880, 5760, False, 2), (256, 2880, 5760, True, 2), (512, 2880, 5760, False, 1), (768, 1024, 8192, True, 2)]

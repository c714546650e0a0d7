"""Sizes that take the dense products through every kernel they have: for each
product, tile and whether the contraction is one K range or several, the first
with the shortest contraction found, the second with a long one, ragged in most
dimensions. tests/test_dense_tiles_host.py asserts that they are what the
library chooses.

  forward, glu_i8, linear: rows x hidden -> inter (out), contraction hidden
  dx: contraction inter (gate and up); dw: contraction rows
"""

# (product, tile, several ranges): (rows, hidden, inter), ...
SIZES = {
    ("forward", 0, False): ((389, 46, 8478), (1417, 711, 2695)),
    ("forward", 0, True): ((1747, 2466, 1166), (1484, 2444, 1375)),
    ("forward", 1, False): ((69, 44, 8249), (1094, 711, 897)),
    ("forward", 1, True): ((582, 2434, 818), (643, 2481, 740)),
    ("forward", 2, False): ((43, 41, 41), (40, 734, 40)),
    ("forward", 2, True): ((40, 991, 40), (40, 1012, 40)),
    ("forward", 3, False): ((1014, 1190, 1028), (867, 1154, 1192)),
    ("forward", 3, True): ((646, 3463, 762), (731, 3475, 676)),
    ("glu_i8", 0, False): ((389, 46, 8478), (1922, 1418, 2089)),
    ("glu_i8", 0, True): ((1165, 4908, 1748), (1541, 5135, 1318)),
    ("glu_i8", 1, False): ((69, 44, 8249), (1071, 1420, 966)),
    ("glu_i8", 1, True): ((393, 4542, 1157), (519, 4607, 901)),
    ("glu_i8", 2, False): ((43, 41, 41), (40, 1413, 43)),
    ("glu_i8", 2, True): ((41, 1940, 42), (41, 2001, 42)),
    ("glu_i8", 3, False): ((1101, 2312, 948), (1007, 2329, 1033)),
    ("glu_i8", 3, True): ((672, 6979, 748), (738, 6965, 700)),
    ("linear", 0, False): ((16654, 52, 387), (3282, 1421, 2465)),
    ("linear", 0, True): ((2050, 4900, 1993), (2478, 5193, 1669)),
    ("linear", 1, False): ((16482, 47, 65), (1702, 1410, 1172)),
    ("linear", 1, True): ((708, 4751, 1371), (1237, 4789, 776)),
    ("linear", 2, False): ((43, 41, 41), (40, 1413, 43)),
    ("linear", 2, True): ((41, 1940, 42), (41, 2001, 42)),
    ("linear", 3, False): ((1592, 2335, 1306), (1685, 2318, 1224)),
    ("linear", 3, True): ((809, 6939, 1271), (1202, 7031, 850)),
    ("dx", 0, False): ((16669, 385, 43), (2319, 3336, 756)),
    ("dx", 0, True): ((1492, 2705, 1289), (1674, 2390, 1281)),
    ("dx", 1, False): ((16590, 65, 41), (2566, 1554, 720)),
    ("dx", 1, True): ((583, 772, 2211), (772, 1253, 1159)),
    ("dx", 2, False): ((43, 41, 41), (670, 322, 700)),
    ("dx", 2, True): ((40, 40, 476), (40, 41, 711)),
    ("dx", 3, False): ((1686, 1182, 588), (1492, 1349, 713)),
    ("dx", 3, True): ((1049, 968, 1744), (847, 1156, 1781)),
    ("dw", 0, False): ((41, 402, 8342), (702, 1026, 3585)),
    ("dw", 0, True): ((2596, 1736, 1154), (2494, 1674, 1201)),
    ("dw", 1, False): ((40, 8629, 65), (715, 865, 1171)),
    ("dw", 1, True): ((2378, 773, 639), (2517, 740, 644)),
    ("dw", 2, False): ((43, 41, 41), (723, 40, 40)),
    ("dw", 2, True): ((971, 42, 41), (966, 41, 43)),
    ("dw", 3, False): ((1174, 1259, 769), (1158, 798, 1246)),
    ("dw", 3, True): ((3484, 530, 908), (3472, 666, 730)),
}


def cases(*products):
    return [(p, t, s, *size) for (p, t, s), sizes in SIZES.items() if p in products for size in sizes]

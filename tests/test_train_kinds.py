"""Which tiles and splits the shared expert's training calls take (CPU only): every kind of launch that the sizes of real
layers and odd ones lead to has a layer in LAYERS, which test_gpu_train_kinds.py compares with float64.

A kind is the call, its tiles, whether the product (of a backward call: the input gradient) is whole, split into one
batch of dense_finish's loads or into more, whether the weight gradient is split, and the weights' layout."""

import math
import random

import pytest
import torch

from mixture_experts_ffn_05_amd import binding as B

BF = torch.bfloat16
LAYOUTS = (B.MOE_W_KN, B.MOE_W_NK)

# (call, T, H, I_s): small layers of every kind
LAYERS = [
    (0, 1, 8, 8), (0, 1, 392, 8), (0, 1, 1240, 1624), (0, 1, 1416, 8), (0, 1, 1480, 8), (0, 1, 2568, 8),
    (0, 1, 7696, 72), (0, 5, 3776, 5696), (0, 70, 2712, 4176), (0, 71, 5736, 328), (0, 132, 456, 432),
    (0, 193, 3448, 2112), (0, 201, 8, 8072), (0, 264, 3096, 264), (0, 335, 1960, 472), (0, 390, 3264, 400),
    (0, 390, 7104, 4224), (0, 393, 464, 1168), (0, 450, 4240, 712), (0, 599, 6016, 392), (0, 961, 264, 4104),
    (0, 1220, 904, 1288), (0, 2675, 2848, 8), (0, 5464, 1296, 8), (1, 1, 8, 8), (1, 1, 8, 392), (1, 1, 8, 1288),
    (1, 1, 8, 1544), (1, 1, 8, 2824), (1, 1, 8, 5136), (1, 68, 1408, 3136), (1, 587, 528, 8088), (1, 653, 72, 5760),
    (1, 2328, 392, 456), (1, 2626, 8, 2832), (1, 4008, 8, 1856), (1, 6617, 1160, 272), (1, 8072, 392, 8),
    (1, 8295, 400, 6080), (1, 8794, 264, 904), (2, 1, 8, 8), (2, 1, 392, 8), (2, 1, 776, 3888), (2, 1, 912, 5904),
    (2, 1, 912, 6168), (2, 1, 1288, 8), (2, 1, 1544, 8), (2, 1, 2824, 8), (2, 1, 3896, 776), (2, 1, 4008, 1288),
    (2, 1, 5128, 8), (2, 2, 776, 3592), (2, 2, 2832, 1032), (2, 2, 3872, 1360), (2, 68, 136, 7376),
    (2, 134, 200, 6424), (2, 194, 208, 8048), (2, 266, 136, 7464), (2, 532, 544, 6888), (2, 585, 592, 6728),
    (2, 769, 8, 8), (2, 770, 2832, 8), (2, 772, 3808, 8), (2, 777, 8, 3856), (2, 784, 8, 3144), (2, 791, 2440, 8),
    (2, 964, 3856, 8), (2, 1104, 3472, 72), (2, 1112, 392, 776), (2, 1429, 7568, 688), (2, 1603, 4744, 32),
    (2, 1685, 4632, 56), (2, 1809, 2824, 8), (2, 1810, 1736, 8), (2, 1886, 264, 592), (2, 1924, 1992, 8),
    (2, 2694, 2696, 8), (2, 7024, 1192, 648), (2, 7170, 8, 8), (2, 8673, 4800, 136), (2, 8844, 6624, 136),
    (3, 1, 8, 8), (3, 1, 8, 200), (3, 1, 8, 648), (3, 1, 8, 776), (3, 1, 8, 1416), (3, 1, 8, 2568), (3, 1, 776, 1952),
    (3, 1, 1288, 1984), (3, 1, 1352, 1944), (3, 1, 3080, 904), (3, 1, 3592, 392), (3, 1, 3872, 392),
    (3, 1, 5904, 456), (3, 2, 1040, 1424), (3, 66, 7088, 72), (3, 130, 6192, 104), (3, 201, 8080, 104),
    (3, 263, 7432, 72), (3, 515, 6904, 288), (3, 587, 6184, 336), (3, 769, 8, 8), (3, 772, 8, 1232),
    (3, 774, 3144, 8), (3, 781, 8, 1432), (3, 784, 8, 1912), (3, 785, 3864, 8), (3, 970, 8, 1928),
    (3, 1092, 72, 1792), (3, 1109, 784, 200), (3, 1247, 400, 6648), (3, 1437, 400, 5264), (3, 1507, 40, 2376),
    (3, 1720, 56, 2320), (3, 1813, 8, 880), (3, 1831, 608, 136), (3, 1846, 8, 1416), (3, 2007, 8, 976),
    (3, 2699, 8, 1352), (3, 6581, 656, 600), (3, 7170, 8, 8), (3, 7588, 136, 4360), (3, 8542, 136, 2384),
]


def kind(call, T, H, I_s, layout):
    tiles, d, w = B.moe_shared_train_tiles(BF, call, T, H, I_s, layout)
    batch = 4 if call == 0 else 8   # splits that dense_finish loads together
    return call, tiles, "whole" if d == 1 else "one batch" if d <= batch else "batches", w > 1, layout


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))   # noqa: E731
    step = rng.choice([8, 64])
    return log(1, 9000), step * log(1, 8192 // step), step * log(1, 8192 // step)


def test_every_kind_has_a_layer():
    if torch.cuda.is_available() and torch.cuda.get_device_properties(0).multi_processor_count != 256:
        pytest.skip("LAYERS were drawn for 256 compute units")
    have = {kind(*c, layout) for c in LAYERS for layout in LAYOUTS}
    rng = random.Random(15)
    for _ in range(30000):
        size = draw(rng)
        for call in range(4):
            for layout in LAYOUTS:
                k = kind(call, *size, layout)
                assert k in have, f"no layer of kind {k}: add {(call, *size)}"
    # both sides of a backward call split, in both calls and layouts, is among them
    for call in (2, 3):
        for layout in LAYOUTS:
            assert any(k[0] == call and k[2] != "whole" and k[3] and k[4] == layout for k in have)

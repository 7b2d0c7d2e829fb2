"""Selective scans for each form of the kernel, long enough that every stage of its pipeline comes round again (two
tiles are on their way while one is computed): five tiles and a rest in every sequence that is to count, or in
its segments, and sizes of channels and states that do and do not fill a tile.  test_scan_plan.py asserts on
the host which form each runs, test_gpu_scan_forms.py the values."""

# (lanes, state values in a lane, cut into segments, lengths (one number: B sequences of it), D, N, G, x type)
FORMS = [
    (4, 2, False, (16, 165), 1024, 8, 1, "bf16"),
    (4, 2, False, (16, 170), 1000, 5, 1, "f32"),
    (4, 2, False, [171, 0, 200, 3, 180] + [2, 1, 5] * 22, 990, 8, 1, "bf16"),
    (4, 4, False, (16, 165), 1024, 16, 1, "bf16"),
    (4, 4, False, (16, 170), 1000, 11, 2, "f32"),
    (4, 4, False, [171, 0, 200, 3, 180] + [2, 1, 5] * 22, 990, 16, 1, "bf16"),
    (16, 1, False, (1, 340), 2768, 16, 1, "bf16"),
    (16, 1, False, (2, 325), 1390, 10, 2, "f32"),
    (16, 1, False, [330, 0, 5, 341], 701, 16, 1, "bf16"),
    (16, 2, False, (1, 340), 2768, 32, 1, "bf16"),
    (16, 2, False, (2, 325), 1390, 20, 1, "f32"),
    (16, 2, False, [330, 0, 5, 341], 701, 32, 1, "bf16"),
    (16, 4, False, (3, 250), 40, 64, 1, "bf16"),
    (16, 4, False, (2, 245), 70, 50, 2, "f32"),
    (16, 4, False, [245, 3, 0, 251], 56, 64, 1, "bf16"),
    (16, 8, False, (3, 90), 40, 128, 1, "bf16"),
    (16, 8, False, (2, 101), 70, 90, 1, "f32"),
    (16, 8, False, [97, 3, 0, 115], 56, 128, 1, "bf16"),
    (16, 1, True, (1, 1700), 1600, 16, 1, "bf16"),
    (16, 1, True, (1, 1700), 1590, 12, 1, "f32"),
    (16, 1, True, [1500, 1700, 0, 900], 460, 16, 1, "bf16"),
    (16, 2, True, (1, 1700), 1600, 32, 1, "bf16"),
    (16, 2, True, (1, 1500), 1590, 18, 1, "f32"),
    (16, 2, True, [1500, 1700, 0, 900], 460, 32, 1, "bf16"),
    (16, 4, True, (1, 1200), 1600, 64, 1, "bf16"),
    (16, 4, True, (1, 1150), 1590, 41, 1, "f32"),
    (16, 4, True, [1250, 1100, 0, 900], 460, 64, 1, "bf16"),
    (16, 8, True, (1, 1000), 640, 128, 1, "bf16"),
    (16, 8, True, (1, 950), 630, 77, 1, "f32"),
    (16, 8, True, [700, 650, 0, 400], 460, 128, 1, "bf16"),
]


def lengths(case):
    """(lengths, packed) of a case."""
    lens = case[3]
    return ([lens[1]] * lens[0], False) if isinstance(lens, tuple) else (lens, True)

"""Which kernel runs a selective scan (csrc/scan_plan.h), on the host."""
import os
import random
import shutil
import subprocess

import pytest

from scan_forms import FORMS, lengths

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CXX = shutil.which("g++") or shutil.which("c++")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    if CXX is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path_factory.mktemp("plan") / "scan_plan")
    subprocess.run([CXX, "-O1", "-Wall", "-Wextra", "-Werror", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    "-I", os.path.join(ROOT, "gated_delta_rule_70_amd", "csrc"),
                    os.path.join(ROOT, "tests", "c_abi", "scan_plan.cpp"), "-o", exe], check=True)

    def run(scans):
        """(lanes, states, tokens of a tile, segments, tokens of a segment) for each (B, T, D, N, G, packed)."""
        text = "\n".join(" ".join(str(int(n)) for n in s) for s in scans)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
        assert len(out) == len(scans)
        return [tuple(int(n) for n in line.split()) for line in out]
    return run


def test_sizes_run_the_form_they_are_there_for(plans):
    cases = [lengths(c) for c in FORMS]
    got = plans([(len(lens), sum(lens) if packed else lens[0], c[4], c[5], c[6], packed) for c, (lens, packed) in zip(FORMS, cases)])
    for c, (lens, packed), (lanes, states, tokens, segs, seg_len) in zip(FORMS, cases, got):
        assert (lanes, states, segs > 1) == c[:3], c
        run = [n for n in ((min(seg_len, n) for n in lens) if segs > 1 else lens) if n > 5]
        assert all(n >= 5 * tokens for n in run), (c, tokens, seg_len)
        # a rest in some tile
        assert any(n % (seg_len if segs > 1 else tokens) % tokens for n in lens), c
    # every form, dense and packed, with channels and states that fill their places and that do not
    for lanes, states in ((4, 2), (4, 4), (16, 1), (16, 2), (16, 4), (16, 8)):
        for cut in (False, True) if lanes == 16 else (False,):
            mine = [c for c in FORMS if c[:3] == (lanes, states, cut)]
            assert {lengths(c)[1] for c in mine} == {False, True}
            assert {c[5] == lanes * states for c in mine} == {False, True}
            assert any(c[4] % (256 // lanes) for c in mine) and {c[7] for c in mine} == {"bf16", "f32"}


# Dense scans (B, T, D, N) that were faster cut, and whole.
CUT = [(1, 520, 64, 4), (1, 1100, 512, 16), (1, 4097, 2000, 16), (2, 4000, 512, 24), (4, 1000, 256, 32), (1, 4097, 2000, 64),
       (4, 1000, 256, 64), (1, 1100, 512, 96), (1, 4097, 1024, 128), (4, 1000, 256, 128), (1, 300, 64, 128)]
WHOLE = [(8, 600, 256, 4), (8, 600, 256, 16), (8, 600, 256, 32), (8, 600, 256, 64), (8, 600, 256, 96), (8, 600, 256, 128),
         (8, 1043, 416, 30), (1, 3026, 2592, 30), (1, 1340, 2768, 30), (3, 3496, 944, 64), (3, 2779, 688, 64), (8, 1071, 448, 8),
         (4, 585, 512, 64), (4, 543, 368, 128), (1, 510, 2896, 16), (4, 300, 256, 16)]


def test_dense_scans_are_cut_where_that_pays(plans):
    for sizes, cut in ((CUT, True), (WHOLE, False)):
        for case, plan in zip(sizes, plans([(*s, 1, 0) for s in sizes])):
            assert (plan[3] > 1) == cut, case


def test_packed_batches_are_cut_where_that_pays(plans):
    """Few rows are not worth a second launch, whatever the lengths; batches in which one sequence may be far longer
    than the others are cut."""
    few = [(2, 260, 64, 16), (2, 500, 64, 16), (3, 390, 64, 16), (3, 480, 64, 16), (3, 390, 64, 64)]
    many = [(10, 3000, 64, 16), (20, 6000, 128, 16), (40, 12000, 64, 16), (20, 6000, 64, 128), (8, 1040, 64, 16), (2, 500, 64, 128)]
    for sizes, cut in ((few, False), (many, True)):
        for case, plan in zip(sizes, plans([(*s, 1, 1) for s in sizes])):
            assert (plan[3] > 1) == cut, case


def test_segments_make_up_the_sequences(plans):
    """A dense sequence has as many segments as its tokens need; a packed batch's slots suffice for any lengths."""
    rng = random.Random(2)
    some = lambda lo, hi: int(round(2 ** rng.uniform(lo, hi)))  # noqa: E731
    scans = []
    for _ in range(20000):
        G = rng.choice([1, 1, 2, 3])
        scans.append((some(0, 8), some(0, 20), G * some(0, 11), some(0, 7), G, rng.random() < 0.5))
    for (B, T, D, N, G, packed), (_, _, _, segs, seg_len) in zip(scans, plans(scans)):
        if segs == 1:
            continue
        assert seg_len % 64 == 0
        if packed:
            assert segs * B >= T // seg_len + B
        else:
            assert (segs - 1) * seg_len < T <= segs * seg_len

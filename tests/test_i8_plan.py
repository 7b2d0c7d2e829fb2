"""Which kernels a product runs on (csrc/i8_plan.h), on the host: the sizes of i8_forms.py run the
form that they are there for, and the launches of any product make up its rows."""
import os
import random
import shutil
import subprocess

import pytest

from i8_forms import FORMS, TWO

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CXX = shutil.which("g++") or shutil.which("c++")
TILES = {"16x16": (16, 16), "32x32": (32, 32), "32x64": (32, 64), "128x64": (128, 64), "128x128 deep": (128, 128),
         "128x128": (128, 128), "192x256": (192, 256), "256x256": (256, 256)}


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    if CXX is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path_factory.mktemp("plan") / "i8_plan")
    subprocess.run([CXX, "-O1", "-Wall", "-Wextra", "-Werror", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    "-I", os.path.join(ROOT, "gated_delta_rule_70_amd", "csrc"),
                    os.path.join(ROOT, "tests", "c_abi", "i8_plan.cpp"), "-o", exe], check=True)

    def run(products):
        text = "\n".join(" ".join(map(str, p)) for p in products)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
        assert len(out) == len(products)
        return [[(int(f), int(n), form, way == "moved") for f, n, form, way in (p.split(",") for p in line.split(";") if p)]
                for line in out]
    return run


def test_sizes_run_the_form_they_are_there_for(launches):
    got = launches([(M, N, K, off, K + pad, off, K + pad) for _, _, M, N, K, pad, off in FORMS])
    for case, runs in zip(FORMS, got):
        form, moved, M = case[:3]
        assert runs == [(0, M, form, moved)], case
    # each form, in place and moved, with the ends of a reduction that there are
    for form in TILES:
        for moved in (False, True):
            ends = {(K % 128 == 0 and "whole") or (K % 16 == 0 and 16) or (K % 4 == 0 and 4) or 1
                    for f, m, _, _, K, _, _ in FORMS if (f, m) == (form, moved)}
            assert ends == (set() if moved and form == "128x128 deep" else {"whole", 16, 1} if moved else {"whole", 16, 4, 1})


def test_sizes_of_two_launches(launches):
    got = launches([(M, N, K, 0, K, 0, K) for M, N, K, _, _ in TWO])
    for (M, N, K, one, two), runs in zip(TWO, got):
        assert [r[2] for r in runs] == [one, two] and [r[3] for r in runs] == [K % 4 != 0] * 2


def test_launches_make_up_the_rows(launches):
    rng = random.Random(1)
    some = lambda lo, hi: int(round(2 ** rng.uniform(lo, hi)))  # noqa: E731
    products = []
    for _ in range(20000):
        M, N, K = some(0, 30), some(0, 26), some(0, 17) - 1 or 1
        if (M + 255) // 256 * ((N + 255) // 256) >= 1 << 23:
            continue
        far = rng.random() < 0.2
        stride = [K + rng.randrange(8) if rng.random() < 0.7 else 0 if rng.random() < 0.1 else K + some(0, 31 if far else 10)
                  for _ in range(2)]
        products.append((M, N, K, rng.randrange(20), stride[0], rng.randrange(20), stride[1]))
    for (M, N, K, a_off, a_stride, w_off, w_stride), runs in zip(products, launches(products)):
        at = 0
        for first, rows, form, moved in runs:
            assert first == at and rows > 0
            at += rows
            bm, bn = TILES[form]
            tiles = -(-rows // bm) * -(-N // bn)
            assert tiles < 1 << 23 and (form not in ("32x32", "128x128 deep") or tiles <= 256)
            words = (a_off + first * a_stride) % 4 == 0 and w_off % 4 == 0 and \
                (rows == 1 or a_stride % 4 == 0) and (N == 1 or w_stride % 4 == 0)
            assert moved == (not words) and not (moved and form == "128x128 deep")
            if form not in ("16x16", "32x32", "32x64"):  # tiles hold their rows' places in 31 bits
                for n, stride, tile in ((rows, a_stride, bm), (N, w_stride, bn)):
                    assert (min(n, tile) - 1) * stride + K + 8 < 1 << 31
        assert at == M

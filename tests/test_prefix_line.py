"""How svg_prefix_attention's work is divided among the CTAs, on the host: the same
code as on the device (csrc/prefix_line.h), built with the host compiler. Every block of
every item has one CTA, an item's pieces lie where the join looks for them, no CTA needs two
slots of a kind or has more than its share."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
FEW, MIXED, GATHERED, JOINT = range(4)


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    if not os.path.exists(os.path.join(cuda, "cuda_runtime.h")):
        cuda = "/usr/local/cuda/include"
    lib = str(tmp_path_factory.mktemp("line") / "line.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", cuda,
                    "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "video_dit_spatial_b200", "csrc"),
                    os.path.join(HERE, "native", "prefix_line_check.cpp"), "-o", lib], check=True)
    f = ctypes.CDLL(lib).check_call

    def call(B, H_kv, GL, d, prefix, lens, sms=148, ok_prefix=1):
        out = (ctypes.c_int * 5)()
        bad = f(B, H_kv, GL, d, prefix, sms, (ctypes.c_int * B)(*lens), ok_prefix, out)
        assert bad == 0, f"line {bad}: {(B, H_kv, GL, d, prefix, lens, sms)}"
        return list(out)

    return call


def log(rng, lo, hi):
    return round(lo * (hi / lo) ** rng.random())


@pytest.mark.parametrize("seed", range(8))
def test_random_calls(check, seed):
    rng = random.Random(seed)
    forms = set()
    for _ in range(250):
        B, H_kv, GL = log(rng, 1, 1024), log(rng, 1, 64), log(rng, 1, 3000)
        while B * H_kv * GL > 2_000_000:
            B, GL = max(B // 2, 1), max(GL // 2, 1)
        prefix = rng.choice([0, log(rng, 1, 100), log(rng, 1, 60000)])
        top = rng.choice([1, 40, 500, 6000])
        lens = [rng.choice([-1, prefix, max(prefix - 3, 0), 0]) if rng.random() < 0.2
                else prefix + rng.randint(0, top) for _ in range(B)]
        out = check(B, H_kv, GL, rng.choice([64, 128]), prefix, lens, sms=rng.choice([148, 148, 132, 7, 2]))
        forms.add(out[0])
    assert forms == {FEW, MIXED, GATHERED, JOINT}


# B, H_kv, query rows of a sequence and key head, d, prefix, rows of their own, form, rounds.
# With items of one one-tile block each (cost 3), x of them to a CTA: rounds = (3 x - 4) / 4, as many
# items of the largest possible cost as fit beside a block that each CTA keeps.
ROUNDS = {
    "none": (3, 6, 20, 64, 700, [9, 0, 100], GATHERED, 0),
    "one": (6, 74, 20, 64, 0, [100] * 6, JOINT, 1),                 # x = 3
    "ten": (60, 38, 20, 64, 0, [100] * 60, JOINT, 10),              # x = 15.4
    "eleven": (60, 40, 20, 64, 0, [100] * 60, JOINT, 11),           # x = 16.2
    "fifteen": (44, 74, 20, 64, 0, [100] * 44, JOINT, 15),          # x = 22
    "sixteen": (46, 74, 20, 64, 0, [100] * 46, JOINT, 16),          # x = 23
    "clamped": (60, 80, 20, 64, 0, [100] * 60, JOINT, 16),          # x = 32.4: 23 without the limit
    "clamped_uneven": (61, 80, 20, 64, 0, [(i * 37) % 129 for i in range(61)], JOINT, 16),
    # 900 rows: groups of 256 and one of 132, 13 blocks of cost 4 each: 480 items of 52
    "prefix_and_own": (3, 40, 900, 64, 600, [900, 900, 900], JOINT, 3),
    "two_kinds": (12, 24, 20, 128, 700, [600 + 97 * i for i in range(12)], GATHERED, None),
    "beside_few_rows": (150, 60, 4, 64, 1000, [b % 60 for b in range(150)], MIXED, None),
    "whole_rounds": (148, 4, 17, 128, 0, [128] * 148, JOINT, None),
}


@pytest.mark.parametrize("name", sorted(ROUNDS))
def test_rounds(check, name):
    B, H_kv, GL, d, prefix, own, form, rounds = ROUNDS[name]
    out = check(B, H_kv, GL, d, prefix, [prefix + n for n in own])
    assert out[0] == form
    if rounds is not None:
        assert out[3] == rounds


def test_nothing_to_do(check):
    for form, (B, GL) in {FEW: (2, 4), MIXED: (9, 4), GATHERED: (7, 31), JOINT: (3, 300)}.items():
        prefix = 0 if form == JOINT else 100
        assert check(B, 2, GL, 64, prefix, [-1] * B)[0] == form
        assert check(B, 2, GL, 64, prefix, [300] * B, ok_prefix=0)[1:] == [0] * 4
        if form == JOINT:
            assert check(B, 2, GL, 64, 0, [0] * B)[1:] == [0] * 4


@pytest.mark.parametrize("d", [64, 128])
def test_the_largest_sums(check, d):
    """2^20 rows a sequence, the most entries: costs and their products with CTA numbers past 2^31."""
    longest = 1 << 20
    check(1024, 2, 1, d, longest, [longest] * 1024)
    check(1024, 1, 300, d, longest // 2, [longest] * 1024)
    check(1, 1, 1 << 20, d, 1000, [1000 + longest // 2])


@pytest.mark.parametrize("sms", [1, 2, 3, 148, 200])
def test_any_number_of_sms(check, sms):
    """A share of a device may have a single one; two kernels of a batch still get a CTA each."""
    for B, H_kv, GL, prefix in ((9, 4, 4, 100), (2, 4, 4, 900), (7, 3, 31, 411), (3, 2, 300, 1000)):
        for own in (0, 40, 700):
            check(B, H_kv, GL, 128, prefix, [prefix + own * (b % 3) for b in range(B)], sms=sms)

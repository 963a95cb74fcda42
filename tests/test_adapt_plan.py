"""Which kernels take a product with adapters (csrc/adapt_plan.h) under AddressSanitizer and UndefinedBehaviorSanitizer,
CPU only.  The GPU tests reach a kernel by its sizes; tests/adapt/check_adapt.cpp says which one those are.
"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "post_weight_quantization_gptq_amd", "csrc", "adapt_plan.h")
CHECKER = os.path.join(ROOT, "tests", "adapt", "check_adapt.cpp")
GXX = shutil.which("g++")
FLAGS = ["-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
         "-fno-omit-frame-pointer", "-Wall", "-Wextra", "-Werror"]

pytestmark = pytest.mark.skipif(GXX is None, reason="g++ not found")


def run(tmp_path, header):
    with open(str(tmp_path / "adapt_plan.h"), "w") as f:
        f.write(header)
    exe = str(tmp_path / "check_adapt")
    b = subprocess.run([GXX] + FLAGS + ["-I", str(tmp_path), CHECKER, "-o", exe], capture_output=True, text=True)
    assert b.returncode == 0, b.stdout + b.stderr
    return subprocess.run([exe], capture_output=True, text=True, timeout=300)


def source():
    with open(HEADER) as f:
        return f.read()


def test_sizes_take_the_kernels_that_the_tests_mean(tmp_path):
    r = run(tmp_path, source())
    assert r.returncode == 0, r.stdout + r.stderr
    assert "adapter checks passed" in r.stdout


# (name, text in adapt_plan.h, replacement, phrase that the checker must print)
MISTAKES = [
    ("a-tile-that-costs-more", "{128, 256, 62, 0}", "{128, 256, 90, 0}", "2048 x 4090 x 96"),
    ("sums-of-one-workgroup", "* p.parts * (p.shape == 1", "* (p.shape == 1", "bytes of sums"),
    ("threads-of-a-launch-in-33-bits", "product < 1LL << 32;", "product < 1LL << 33;", "said to"),
    ("more-workgroups-than-rows", "std::min(M, 32))", "32)", "slots"),
]


@pytest.mark.parametrize("name,old,new,phrase", MISTAKES, ids=[m[0] for m in MISTAKES])
def test_checker_rejects_a_planted_mistake(tmp_path, name, old, new, phrase):
    src = source()
    assert src.count(old) == 1, "the planted text must appear once: %r" % old
    r = run(tmp_path, src.replace(old, new))
    assert r.returncode != 0, "the checker accepted the mistake %s" % name
    assert phrase in r.stderr, r.stderr[-2000:]

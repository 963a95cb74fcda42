"""The attention's launch shapes (csrc/attend_plan.h) under AddressSanitizer and UndefinedBehaviorSanitizer, CPU only.

tests/attend/check_attend.cpp replays what the kernels' threads read and write for every shape.  The planted-mistake
cases recompile it against the header with one slip each and require it to reject that.
"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "post_weight_quantization_gptq_amd", "csrc", "attend_plan.h")
CHECKER = os.path.join(ROOT, "tests", "attend", "check_attend.cpp")
GXX = shutil.which("g++")
FLAGS = ["-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
         "-fno-omit-frame-pointer", "-Wall", "-Wextra", "-Werror"]

pytestmark = pytest.mark.skipif(GXX is None, reason="g++ not found")


def run(tmp_path, header):
    with open(str(tmp_path / "attend_plan.h"), "w") as f:
        f.write(header)
    exe = str(tmp_path / "check_attend")
    b = subprocess.run([GXX] + FLAGS + ["-I", str(tmp_path), CHECKER, "-o", exe], capture_output=True, text=True)
    assert b.returncode == 0, b.stdout + b.stderr
    return subprocess.run([exe], capture_output=True, text=True, timeout=300)


def source():
    with open(HEADER) as f:
        return f.read()


def test_shapes_pass_the_checker(tmp_path):
    r = run(tmp_path, source())
    assert r.returncode == 0, r.stdout + r.stderr
    assert "attention checks passed" in r.stdout


# (name, text in attend_plan.h, replacement, phrase that the checker must print)
MISTAKES = [
    ("join-threads-past-the-rows", "return JoinPlan{G, rows, rows * q4 * G};", "return JoinPlan{G, rows, 256};", "reads sum"),
    ("join-partners-a-row-apart", "tid / (dim / 4) % G, 4 * (tid % (dim / 4))", "tid % G, 4 * (tid / G % (dim / 4))", "partner"),
    ("threads-of-a-launch-in-33-bits", "attention_threads(p, dim) < 1LL << 32 &&", "attention_threads(p, dim) < 1LL << 33 &&", "seqs"),
    ("rows-of-a-join-not-counted", "join < 1LL << 32", "join >= 0", "seqs"),
]


@pytest.mark.parametrize("name,old,new,phrase", MISTAKES, ids=[m[0] for m in MISTAKES])
def test_checker_rejects_a_planted_mistake(tmp_path, name, old, new, phrase):
    src = source()
    assert src.count(old) == 1, "the planted text must appear once: %r" % old
    r = run(tmp_path, src.replace(old, new))
    assert r.returncode != 0, "the checker accepted the mistake %s" % name
    assert phrase in r.stderr, r.stderr[-2000:]

"""Index arithmetic of the serving step (csrc/qst_index.h) at the ends of its
types, compiled for the host (CPU only)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "dequant_matmul_amd", "csrc", "qst_index.h")


def run(tmp_path, body):
    """Lines of numbers that a host program with `body` as main prints."""
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    src, exe = tmp_path / "index.cpp", str(tmp_path / "index")
    src.write_text('#include "%s"\n#include <cstdio>\nusing namespace qmm;\nint main()\n{\n%s\nreturn 0;\n}\n' % (HEADER, body))
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover",
                    str(src), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    return [[int(v) for v in line.split()] for line in out.splitlines()]


def test_pages_up_to_the_largest_lengths(tmp_path):
    most = 2 ** 31 - 1
    cases = [(n, s) for s in (6, 7, 16, 24, 29, 30)
             for n in (0, 1, (1 << s) - 1, 1 << s, most // 2, most // 2 + 2, most - (1 << s) + 1, most - 1, most)
             + (((1 << s) + 1,) if s < 30 else ((1 << 30) + 1,))]
    body = "\n".join('printf("%%d\\n", pages_of(%d, %d));' % c for c in cases)
    assert run(tmp_path, body) == [[-(-n // (1 << s))] for n, s in cases]


def test_sums_stay_at_their_cap(tmp_path):
    """Once at the cap, which can be 2^31 (tokens 2^31 - 1 and one), they do not wrap."""
    caps = [0, 1, 5, 2 ** 31 - 1, 2 ** 31, 2 ** 32 - 1]
    cases = [(a, b, c) for c in caps for a in {0, 1, c // 2, c // 2 + 1, c - 1, c} for b in {0, 1, c // 2, c - 1, c}
             if 0 <= a <= c and 0 <= b <= c]
    body = "\n".join('printf("%%u\\n", sat_add(%du, %du, %du));' % c for c in cases)
    assert run(tmp_path, body) == [[min(a + b, c)] for a, b, c in cases]


def test_sums_of_pairs_of_the_longest_requests(tmp_path):
    """As the lanes add them, at the most tokens: no later sum is a smaller one."""
    body = """uint32_t v[8] = {0x7fffffffu, 0x7fffffffu, 0x7fffffffu, 0x7fffffffu, 1, 0, 0, 0}, cap = 0x80000000u;
for (int d = 1; d < 8; d *= 2)
    for (int i = 7; i >= d; --i)
        v[i] = sat_add(v[i], v[i - d], cap);
for (int i = 0; i < 8; ++i)
    printf("%u\\n", v[i]);"""
    assert [v for v, in run(tmp_path, body)] == [2 ** 31 - 1] + [2 ** 31] * 7

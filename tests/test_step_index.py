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

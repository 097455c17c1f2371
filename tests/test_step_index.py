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
    body = "\n".join('printf("%%u\\n", sat_add<%s>(%du, %du, %du));' % (str(c[2] >= 2 ** 31).lower(), *c) for c in cases)
    assert run(tmp_path, body) == [[min(a + b, c)] for a, b, c in cases]


def test_sums_of_pairs_of_the_longest_requests(tmp_path):
    """As the lanes add them, at the most tokens: no later sum is a smaller one."""
    body = """uint32_t v[8] = {0x7fffffffu, 0x7fffffffu, 0x7fffffffu, 0x7fffffffu, 1, 0, 0, 0}, cap = 0x80000000u;
for (int d = 1; d < 8; d *= 2)
    for (int i = 7; i >= d; --i)
        v[i] = sat_add<true>(v[i], v[i - d], cap);
for (int i = 0; i < 8; ++i)
    printf("%u\\n", v[i]);"""
    assert [v for v, in run(tmp_path, body)] == [2 ** 31 - 1] + [2 ** 31] * 7


# (bytes of a block, its elements, elements of a lane's unit) of the types whose rows
# begin anywhere
Q4_0, Q8_0, Q5_0, Q6_K = (18, 32, 32), (34, 32, 32), (22, 32, 32), (210, 256, 64)


@pytest.mark.parametrize("bb,be,ue", [Q4_0, Q8_0, Q5_0, Q6_K])
def test_items_stay_inside_the_matrix_and_their_part_of_lds(bb, be, ue, tmp_path):
    """Every item of rows of up to 20 segments, in rounds of as many waves as the kernel
    takes: whole chunks and last bytes lie inside the matrix, hold all of the item, and
    land in the wave's own part."""
    body = """
const int64_t BB = %d, BE = %d, UE = %d, SEGB = 64 * UE / BE * BB;
const int64_t MOST = SEGB + 16;
long seen = 0, bad = 0, tails = 0, behind = 0;
for (int64_t blocks = 1; blocks <= 20 * 64 * UE / BE; blocks += blocks < 70 ? 1 : 13)
    for (int64_t n = 1; n <= 5; ++n) {
        const int64_t rb = blocks * BB, units = blocks * BE / UE, segs = (units + 63) / 64;
        const int64_t waves = segs < 8 ? segs : 8, rounds = (segs + waves - 1) / waves;
        const int64_t rpi = units > 32 ? 1 : units > 16 ? 2 : 4, end = n * rb;
        for (int64_t row0 = 0; row0 < n; row0 += rpi)
            for (int64_t seg = 0; seg < rounds * waves; ++seg) {
                const int64_t from = row0 * rb + seg * SEGB;
                const int shift = (int)(from & 15);
                int64_t bytes = rpi > 1 ? (rpi * rb < end - from ? rpi * rb : end - from)
                                        : (SEGB < rb - seg * SEGB ? SEGB : rb - seg * SEGB);
                bytes = bytes > 0 ? bytes : 0;
                const int64_t left = end - from + shift, whole = whole_chunks(bytes, shift, left);
                const int tail = last_bytes(64 * seg < units, left, (int)MOST);
                const int64_t to = left & ~(int64_t)15;
                ++seen, tails += tail != 0, behind += left < 0;
                bad += whole < 0 || whole %% 16 != 0 || whole > MOST + 15;
                bad += bytes > 0 && (from - shift < 0 || from - shift + whole > end);
                bad += bytes > 0 && whole < bytes + shift && whole + tail < bytes + shift;
                bad += bytes == 0 && whole != 0;
                bad += tail != 0 && (to < 0 || to + tail > MOST || end - tail < 0);
            }
    }
printf("%%ld %%ld %%ld %%ld\\n", seen, bad, tails, behind);""" % (bb, be, ue)
    (seen, bad, tails, behind), = run(tmp_path, body)
    assert bad == 0 and seen > 1000 and tails > 10 and behind > 10

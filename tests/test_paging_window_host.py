"""Keys that a part of an attention tile goes through (csrc/w4_paging.h), compiled as plain C++ and checked
against brute force: all that any row sees, each once, and no aligned 16 keys that no row sees, so that
no page outside every row's window is looked up.
"""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "w4_paging.h"
using namespace w4;
static uint64_t state = 88172645463325252ull;
static int64_t rnd(int64_t lo, int64_t hi) {
    state ^= state << 13; state ^= state >> 7; state ^= state << 17;
    return lo + (int64_t)(state % (uint64_t)(hi - lo + 1));
}
#define CHECK(c) do { if (!(c)) { std::printf("line %d: %s\n", __LINE__, #c); return 1; } } while (0)
int main() {
    for (int trial = 0; trial < 20000; ++trial) {
        const int64_t G = rnd(1, 8), window = rnd(0, 3) ? rnd(1, 300) : 0, parts = rnd(1, 9);
        const int64_t least = 64 * rnd(1, 4), R = rnd(0, 1) ? 16 : 32;
        const Seq s = clamp_seq(rnd(-3, 5), rnd(0, 60), rnd(-5, 900), 50, 800);
        for (int64_t row0 = 0; row0 < s.n * G; row0 += R) {
            const int64_t rows = imin(R, s.n * G - row0);
            const Span most = key_span(s, row0, rows, G, window, parts, least), k = seen_span(most);
            CHECK(k.parts >= 1 && k.parts <= most.parts && k.chunk == most.chunk && k.end == most.end);
            std::vector<int> seen(s.ctx + 1, 0), taken(s.ctx + 1, 0);
            for (int64_t r = row0; r < row0 + rows; ++r) {
                const int64_t pos = s.ctx - s.n + r / G;
                for (int64_t j = window ? imax(0, pos - window + 1) : 0; j <= pos; ++j) seen[j] = 1;
            }
            for (int p = 0; p < k.parts; ++p) {
                const int32_t k0 = k.begin + p * k.chunk, k1 = lesser(k.end - k0, k.chunk) + k0;
                CHECK(k0 % 16 == 0 && k0 >= 0 && k1 <= s.ctx && (k.end > k.begin ? k0 < k1 : k0 == k1));
                // keys past the last whole tile are masked by what the rows see: only the last part has any
                CHECK((k1 - k0) % kKeyTile == 0 || k1 == k.end);
                for (int32_t j = k0; j < k1; j += 16) {
                    int any = 0;
                    for (int32_t i = j; i < lesser(j + 16, k1); ++i) { any |= seen[i]; ++taken[i]; }
                    CHECK(any);
                }
            }
            for (int64_t j = 0; j < s.ctx; ++j) CHECK(taken[j] <= 1 && taken[j] >= seen[j]);
        }
    }
    // the longest contexts: nothing passes 32 bits
    const Seq far = clamp_seq(0, 8, 1 << 30, 8, 1 << 30);
    const Span k = seen_span(key_span(far, 0, 8, 1, 0, 1, 256));
    CHECK(k.begin == 0 && k.parts == 1 && k.end == 1 << 30 && k.chunk == 1 << 30);
    for (int32_t window : {100, 1 << 29, (1 << 30) - 64, (1 << 30) - 5}) {
        const Span w = seen_span(key_span(far, 0, 8, 1, window, 1, 256));
        CHECK(w.begin == imax(0, (1 << 30) - 7 - window) / 16 * 16 && w.end == 1 << 30 && w.parts == 1);
    }
    std::printf("ok\n");
    return 0;
}
"""


def test_parts_of_windows(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "window.cpp", tmp_path / "window"
    src.write_text(PROGRAM)
    inc = os.path.join(ROOT, "dequant_gemv_w4_amd", "csrc")
    subprocess.run([gxx, "-std=c++17", "-O1", "-D_GLIBCXX_ASSERTIONS", "-I", inc, str(src), "-o", str(exe)],
                   check=True, capture_output=True, timeout=120)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout

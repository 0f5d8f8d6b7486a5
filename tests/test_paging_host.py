"""The paged index arithmetic that the kernels share with the host (csrc/w4_paging.h), compiled
as plain C++ and checked against brute force: every row of every sequence in exactly one tile,
every key that a row sees in exactly one part, no page outside the cache, and pages of requests.
"""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
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
    for (int trial = 0; trial < 400; ++trial) {
        const int64_t B = rnd(1, 9), G = rnd(1, 9), R = trial % 2 ? 32 : 256;
        std::vector<int64_t> cu(1, 0);
        for (int64_t b = 0; b < B; ++b) cu.push_back(cu.back() + (rnd(0, 3) ? rnd(0, 150) : 0));
        const int64_t T = cu[B] + rnd(0, 5);
        std::vector<std::vector<int>> seen(B);
        for (int64_t b = 0; b < B; ++b) seen[b].assign((cu[b + 1] - cu[b]) * G, 0);
        for (int64_t tile = 0; tile < tile_bound(T, B, G, R); ++tile) {
            int64_t b = 0;
            while (b + 1 < B && first_tile(cu[b + 1], b + 1, G, R) <= tile) ++b;
            const int64_t row0 = (tile - first_tile(cu[b], b, G, R)) * R;
            CHECK(row0 >= 0);
            for (int64_t r = row0; r < imin(row0 + R, (cu[b + 1] - cu[b]) * G); ++r) seen[b].at(r)++;
        }
        for (auto& s : seen) for (int c : s) CHECK(c == 1);
    }
    for (int trial = 0; trial < 20000; ++trial) {
        const int64_t G = rnd(1, 8), window = rnd(0, 1) ? rnd(1, 300) : 0, parts = rnd(1, 9);
        const int64_t least = 64 * rnd(1, 4), R = 32;
        const Seq s = clamp_seq(rnd(-3, 5), rnd(0, 60), rnd(-5, 900), 50, 800);
        CHECK(s.start >= 0 && s.n >= 0 && s.start + s.n <= 50 && s.ctx >= 0 && s.ctx <= 800);
        for (int64_t row0 = 0; row0 < s.n * G; row0 += R) {
            const int64_t rows = imin(R, s.n * G - row0);
            const Span k = key_span(s, row0, rows, G, window, parts, least);
            CHECK(k.parts >= 1 && k.parts <= parts && k.begin % kKeyTile == 0 && k.chunk % kKeyTile == 0);
            CHECK(k.begin >= 0 && k.end <= s.ctx + 0 * k.chunk && k.begin + k.parts * k.chunk >= k.end);
            CHECK(k.parts == 1 || k.begin + (k.parts - 1) * k.chunk < k.end);
            std::vector<int> part_of(s.ctx + 1, -1);
            for (int p = 0; p < k.parts; ++p)
                for (int64_t j = k.begin + p * k.chunk; j < imin(k.end, k.begin + (p + 1) * k.chunk); ++j) {
                    CHECK(j < s.ctx && part_of[j] < 0);
                    part_of[j] = p;
                }
            int64_t last = -1;
            for (int64_t r = row0; r < row0 + rows; ++r) {
                const int64_t pos = s.ctx - s.n + r / G;
                for (int64_t j = 0; j <= pos; ++j)
                    if (!window || j > pos - window) { CHECK(part_of[j] >= 0); last = imax(last, j); }
            }
            CHECK(k.end == (last < 0 ? k.begin : last + 1));
        }
    }
    CHECK(checked_page(-1, 5) == -1 && checked_page(5, 5) == -1 && checked_page(4, 5) == 4 && checked_page(0, 5) == 0);
    CHECK(checked_page(INT32_MAX, 5) == -1 && checked_page(INT32_MIN, 5) == -1);
    for (int trial = 0; trial < 20000; ++trial) {
        const int64_t page = 1 << rnd(4, 8), len = rnd(-2, 1000), fresh = rnd(-2, 500), most = rnd(1, 60);
        const Need d = page_need(len, fresh, page, most);
        if (len < 0 || fresh < 0) { CHECK(!d.fits && d.take == 0); continue; }
        int64_t have = 0, want = 0;
        while (have * page < len) ++have;
        while (want * page < len + fresh) ++want;
        CHECK(d.fits == (want <= most) && d.have == have && d.take == (d.fits ? want - have : 0));
    }
    CHECK(!page_need(INT32_MAX, INT32_MAX, 16, 1 << 30).fits);
    std::printf("ok\n");
    return 0;
}
"""


def test_paging_arithmetic(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "paging.cpp", tmp_path / "paging"
    src.write_text(PROGRAM)
    inc = os.path.join(ROOT, "dequant_gemv_w4_amd", "csrc")
    subprocess.run([gxx, "-std=c++17", "-O1", "-D_GLIBCXX_ASSERTIONS", "-I", inc, str(src), "-o", str(exe)],
                   check=True, capture_output=True, timeout=120)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout

"""How the attention numbers its tiles (csrc/w4_paging.h), compiled as plain C++ and run as the kernels run
it, against brute force: with the tiles and parts that the host plans, every query row of every sequence
lies in exactly one tile that runs, whatever the lengths, and no tile has more parts than are launched.
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
    int kinds[2][2][3] = {};                                  // both, by token, tile
    for (int trial = 0; trial < 6000; ++trial) {
        const int64_t B = rnd(0, 3) ? rnd(1, 12) : rnd(60, 200), G = rnd(0, 3) ? rnd(1, 9) : rnd(10, 70), kv = 1 << rnd(0, 5);
        const bool fp8 = rnd(0, 1), one = rnd(0, 2) == 0;     // a token each, or up to 150
        std::vector<int64_t> cu(1, 0);
        for (int64_t b = 0; b < B; ++b) cu.push_back(cu.back() + (one ? 1 : rnd(0, 2) ? rnd(0, 4) : rnd(0, 6) ? 0 : rnd(0, 150)));
        int64_t T = imax(1, cu[B] + (rnd(0, 1) ? rnd(0, 5) : 0));
        if (rnd(0, 4) == 0 && cu[B] <= B) T = B;              // as many rows as sequences, not one each
        const int64_t capacity = 16 << rnd(0, 10), window = rnd(0, 1) ? rnd(1, 3000) : 0;
        AttendPlan p;
        plan_attend(T, B, G * kv, kv, capacity, fp8, &p);
        CHECK(p.narrow_tiles % kv == 0 && p.wide_tiles % kv == 0 && p.narrow_fill <= p.narrow_parts && p.wide_fill <= imax(p.wide_parts, 1));
        kinds[p.both][T == B][p.narrow_tile == 16 ? 0 : p.few_tiles]++;
        std::vector<std::vector<int>> seen(B);
        for (int64_t b = 0; b < B; ++b) seen[b].assign((cu[b + 1] - cu[b]) * G, 0);
        for (int wide = 0; wide < 2; ++wide) {
            const int64_t R = wide ? kWideRows : p.narrow_tile, count = (wide ? p.wide_tiles : p.narrow_tiles) / kv;
            for (int64_t tile = 0; tile < count; ++tile) {
                int64_t b, row0;
                if (!wide && p.both) {
                    b = few_sequence(tile, B);
                    row0 = few_row0(tile, B, R);
                } else {
                    auto first = [&](int64_t x) { return !wide && T == B ? token_tile(cu[x], G, R) : first_tile(cu[x], x, G, R); };
                    b = 0;
                    while (b + 1 < B && first(b + 1) <= tile) ++b;
                    row0 = (tile - first(b)) * R;
                }
                CHECK(b >= 0 && b < B);
                const int64_t rows = (cu[b + 1] - cu[b]) * G;
                if (!tile_runs(wide, p.both, row0, rows, p.few_tiles)) continue;
                for (int64_t r = row0; r < imin(row0 + R, rows); ++r) seen[b].at(r)++;
                const int64_t ctx = rnd(0, capacity), reach = window ? imin(ctx, window) : ctx;
                const Seq s = clamp_seq(cu[b], cu[b + 1], ctx, T, capacity);
                const int64_t most = !wide ? (p.both && rows > R ? p.narrow_fill : p.narrow_parts) : reach < kWideEven ? p.wide_fill : p.wide_parts;
                const Span k = seen_span(key_span(s, row0, imin(R, rows - row0), G, window, most, wide ? kWideLeast : kNarrowLeast));
                CHECK(k.parts >= 1 && k.parts <= (wide ? p.wide_parts : p.narrow_parts) && k.parts <= kMaxParts);
            }
        }
        for (auto& s : seen) for (int c : s) CHECK(c == 1);
    }
    // every way of numbering was met: alone by token and not, with 16 rows and 32; beside wide tiles with 1 and 2
    CHECK(kinds[0][1][0] && kinds[0][1][1] + kinds[0][1][2] && kinds[0][0][0] && kinds[1][0][1] && kinds[1][0][2]);
    std::printf("ok\n");
    return 0;
}
"""


def test_every_row_in_one_tile(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "tiles.cpp", tmp_path / "tiles"
    src.write_text(PROGRAM)
    inc = os.path.join(ROOT, "dequant_gemv_w4_amd", "csrc")
    subprocess.run([gxx, "-std=c++17", "-O1", "-D_GLIBCXX_ASSERTIONS", "-I", inc, str(src), "-o", str(exe)],
                   check=True, capture_output=True, timeout=120)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout

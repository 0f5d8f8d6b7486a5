// Index arithmetic of the paged cache and of the attention's work split, in plain C++ so that
// the kernels and a host program share it.
//
// A sequence b has the query rows cu[b] .. cu[b+1] of the packed batch and lens[b] keys, its new
// tokens' among them.  Its key j lies in row j % page of page table[b][j / page].  Query t of a
// sequence with n new tokens stands at position lens - n + t and sees the keys up to itself,
// with a window the last `window` of them.
//
// Attention works on tiles of R rows, one kv head each: row r of a sequence is head r % G of its
// token r / G (G query heads share a kv head), so that one pass over the keys serves all of them.
#pragma once

#include <stdint.h>

#ifdef __HIPCC__
#define W4_HD __host__ __device__ __forceinline__
#else
#define W4_HD inline
#endif

namespace w4 {

W4_HD int64_t imin(int64_t a, int64_t b) { return a < b ? a : b; }
W4_HD int64_t imax(int64_t a, int64_t b) { return a > b ? a : b; }
W4_HD int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// What a workgroup of the attention computes before its first load is in 32 bits: tokens times query
// heads stay below 2^26 and keys at 2^30 or less, and a division in 64 bits is a hundred instructions.
W4_HD int32_t lesser(int32_t a, int32_t b) { return a < b ? a : b; }
W4_HD int32_t greater(int32_t a, int32_t b) { return a > b ? a : b; }
W4_HD int32_t quotient(int32_t a, int32_t b) { return (int32_t)((uint32_t)a / (uint32_t)b); }   // a >= 0, b > 0

// First tile of sequence b when the tiles of all sequences are numbered without knowing their
// lengths: floor(cu[b] G / R) + b.  It grows by at least ceil(n G / R) and at least 1 from one
// sequence to the next (floor(a + c) - floor(a) + 1 >= ceil(c)); numbers past a sequence's
// tiles stay idle.  All tiles lie below floor(T G / R) + B.
W4_HD int32_t first_tile(int32_t cu_b, int32_t b, int32_t G, int32_t R) { return quotient(cu_b * G, R) + b; }
W4_HD int64_t tile_bound(int64_t T, int64_t B, int64_t G, int64_t R) { return T * G / R + B; }

// The other two ways to number tiles.  By token, where there are as many tokens as sequences: each token has
// the tiles that its G rows fill, so a sequence's first follows from its first token.
W4_HD int32_t token_tile(int32_t cu_b, int32_t G, int32_t R) { return cu_b * quotient(G + R - 1, R); }
// Of sequences with few rows beside wide tiles: all first tiles, then all second ones, which mostly have no
// rows: taking turns, they would leave every other place that the workgroups go to in turn without work
// (31 single tokens over 4000 beside a chunk: 143 us instead of 113).
W4_HD int32_t few_sequence(int32_t tile, int32_t B) { return tile < B ? tile : tile - B; }
W4_HD int32_t few_row0(int32_t tile, int32_t B, int32_t R) { return tile < B ? 0 : R; }

// Attention: query rows of a tile in the two kernels, keys a part takes at least, parts at most.
constexpr int kFewRows = 32, kWideRows = 256;   // narrow: 16 or kFewRows
constexpr int kNarrowLeast = 256, kWideLeast = 128, kWideEven = 4096, kMaxParts = 64;

// Whether a tile has rows: where both kinds are launched, a sequence of at most few_tiles (1 or 2) * kFewRows
// rows has narrow tiles, as many, and the others have wide ones.
W4_HD bool tile_runs(bool wide, bool both, int32_t row0, int32_t rows, int32_t few_tiles) {
    const bool few = rows <= few_tiles * kFewRows;
    return row0 >= 0 && row0 < rows && (wide ? !few : few || !both);
}

// A sequence as the kernels read it, whatever the arrays hold: its rows lie in [0, T) and its
// keys in the table.
struct Seq {
    int32_t start;   // first query row
    int32_t n;       // query rows
    int32_t ctx;     // keys
};
W4_HD Seq clamp_seq(int32_t cu0, int32_t cu1, int32_t len, int32_t T, int32_t capacity) {
    Seq s;
    s.start = lesser(greater(cu0, 0), T);
    s.n = greater(lesser(cu1, T) - s.start, 0);
    s.ctx = lesser(greater(len, 0), capacity);
    return s;
}

// Keys lo .. hi that the row at position pos sees of ctx: those up to itself, with a prefix the first `prefix`
// ones too; none ahead of `first` (the first of its document) or of its window.  None where hi < lo.
struct KeyRange {
    int32_t lo, hi;
};
W4_HD KeyRange key_range(int32_t pos, int32_t ctx, int32_t window, int32_t first, int32_t prefix) {
    KeyRange k;
    k.hi = greater(pos, lesser(greater(prefix, 0), ctx) - 1);
    k.lo = greater(0, lesser(first, ctx));                   // ctx: behind every key
    if (window > 0) k.lo = greater(k.lo, pos - window + 1);
    return k;
}

// Keys of a tile of rows [row0, row0 + rows) of a sequence (rows >= 1), and their split:
// [first, end) is what any row sees, begin is first rounded down to a multiple of kKeyTile; part p of
// `parts` takes [begin + p * chunk, begin + (p + 1) * chunk).  The parts are cut by the actual
// lengths, at least `least` keys each and none below twice that, whatever number the launch allows.
constexpr int kKeyTile = 64;
struct Span {
    int32_t first, begin, end, chunk, parts;
};
W4_HD Span cut_span(int32_t first, int32_t end, int32_t max_parts, int32_t least) {
    Span k;
    k.first = first;
    k.end = end;
    k.begin = k.first / kKeyTile * kKeyTile;
    k.chunk = 2 * least;
    k.parts = 1;
    if (k.end <= k.begin) {
        k.first = k.end = k.begin;
        return k;
    }
    const int32_t len = k.end - k.begin;
    if (len > 2 * least && max_parts > 1) {
        k.chunk = greater(least, (quotient(len + max_parts - 1, max_parts) + kKeyTile - 1) / kKeyTile * kKeyTile);
        k.parts = quotient(len + k.chunk - 1, k.chunk);
    } else {
        k.chunk = greater(2 * least, (len + kKeyTile - 1) / kKeyTile * kKeyTile);
    }
    return k;
}
W4_HD Span key_span(const Seq& s, int32_t row0, int32_t rows, int32_t G, int32_t window,
                    int32_t max_parts, int32_t least) {
    const int32_t pos0 = s.ctx - s.n;                        // position of the first new token
    const int32_t end = lesser(s.ctx, pos0 + quotient(row0 + rows - 1, G) + 1);
    return cut_span(window > 0 ? greater(0, pos0 + quotient(row0, G) - window + 1) : 0, end, max_parts, least);
}

// The span without the keys ahead of the 16 that hold the first one seen.  Pages hold a multiple of 16
// keys, so no page is looked up that lies wholly ahead of every row's window: a user may have given it
// back, and its entry may name another request's page or none (looked up, such entries set the status and
// had all rows computed again: 32 single tokens with a window of 1024 took 6 ms instead of 25 us).  All
// parts move, so that each but the last is still whole tiles long.
W4_HD Span seen_span(Span k) {
    const int32_t begin = k.first / 16 * 16;
    if (begin > k.begin) {
        k.begin = begin;
        k.parts = quotient(k.end - begin + k.chunk - 1, k.chunk);
    }
    return k;
}

// What the host knows of a call decides the launches; the parts that a tile really has follow
// from the lengths on the device.
struct AttendPlan {
    int64_t narrow_tiles, wide_tiles;   // workgroups of one part
    int narrow_tile;                    // rows of a narrow tile: 16 or kFewRows
    int few_tiles;                      // narrow tiles of a sequence that has no wide ones, beside wide ones
    int narrow_parts, narrow_fill, wide_parts, wide_fill;
    bool both;
};

// Parts that a launch allows per tile, to make up to `target` workgroups.  256 is one a compute unit (LDS
// holds no second).  Single tokens, workgroups up to 256: 24 requests of up to 2000 tokens (192 tiles)
// take 35 us unsplit, 42 in two parts each; 5 of up to 8000 over 32 kv heads 113 and 128; 32 of up to 8192
// 155 with 256 workgroups, 165 with 512, 168 with 1024.  Wide tiles: up to 256 as well, since a part
// costs a pass over its rows' results (1100 tokens over 500: 60 us unsplit, 86 in two parts; over 2000 136
// and 160), but where the keys are many (kWideEven) about 512, so that the last round of workgroups is a
// small one (over 8000: 448 and 400, over 30,000 1602 and 1284).  At least kNarrowLeast keys a part, and
// none below twice that: one request over 1000 keys takes 11.2 us with parts of 256, 12.1 with 512, over
// 500 8.5 unsplit and 10.2 split.  Wide: 16 tokens over 2000 16.0 with 128, 17.2 with 256, 22.8 with 512.
inline int parts_for(int64_t tiles, int64_t target, int64_t longest, int64_t least) {
    const int64_t want = longest > 2 * least ? target / tiles : 1;
    return (int)imax(1, imin(want, imin(ceil_div(longest, least), kMaxParts)));
}

inline void plan_attend(int64_t T, int64_t B, int64_t heads, int64_t kv_heads, int64_t capacity, bool fp8, AttendPlan* p) {
    const int64_t G = heads / kv_heads;
    // As many tokens as sequences are taken for one each, and then as for too few rows in all the wide
    // kernel is left out.  The lengths are on the device: a prompt among idle sequences has narrow tiles for
    // every 16 rows there (a prompt of 500 in 512 places 55 us, 36 with one row more; 200 tokens and 56
    // single ones over 2000 in 256 places 145 and 106; 4000 over 4000 in 4096 places 2490 and 910).  Single
    // tokens are what such a batch mostly holds, and both kernels would cost them more: 32 over up to 8192
    // 156 us, 178 with one row more; 256 over 2000 336 and 346.
    p->both = T != B && T * G > kFewRows;
    // Sequences of 33 to 64 rows as two narrow tiles: a wide one would have no rows for most of its waves.
    // 16 requests of up to 8 tokens (8 heads a kv head) over up to 4000 take 69 us so, 91 with wide tiles, 8 over
    // an E4M3 cache 38 and 55, 32 78 and 113.  Of a bfloat16 cache the keys come from memory twice where the
    // second tiles have to wait for a compute unit: 32 requests 113 and 95.
    p->few_tiles = fp8 || 2 * B * kv_heads <= 256 ? 2 : 1;
    // 32 rows a narrow tile where 16 would read a sequence's keys twice: single tokens of 32 requests over up
    // to 8192, 32 heads a kv head, take 51.6 us instead of 71.6, four tokens of 32 over 4000 (8 heads) 81.6
    // instead of 97.0.  Not where the keys could not even give every compute unit a workgroup of 16 rows: one
    // request over 8000, 2 kv heads, takes 14.8 us with 16 and 16.1 with 32.
    const int64_t fine = T * ceil_div(G, 16) * kv_heads * ceil_div(capacity, kNarrowLeast);
    p->narrow_tile = p->both || (G > 16 && fine > 256) ? kFewRows : 16;
    const int64_t R = p->narrow_tile;
    p->narrow_tiles = (p->both ? B * p->few_tiles : T == B ? T * ceil_div(G, R) : tile_bound(T, B, G, R)) * kv_heads;
    // beside wide tiles most sequences have one narrow tile, which may then take the parts of the idle ones
    p->narrow_fill = parts_for(p->narrow_tiles, 256, capacity, kNarrowLeast);
    p->narrow_parts = p->both ? parts_for(B * kv_heads, 256, capacity, kNarrowLeast) : p->narrow_fill;
    p->wide_tiles = p->both ? tile_bound(T, B, G, kWideRows) * kv_heads : 0;
    p->wide_fill = p->both ? parts_for(p->wide_tiles, 256, capacity, kWideLeast) : 1;
    p->wide_parts = p->both && capacity >= kWideEven
                        ? parts_for(p->wide_tiles, 511 + p->wide_tiles, capacity, kWideLeast) : p->wide_fill;
}

// Number of a page if the cache has it, else -1.
W4_HD int64_t checked_page(int64_t page, int64_t pages) { return page >= 0 && page < pages ? page : -1; }

// Pages that a request with `len` cached tokens takes for `fresh` new ones, if its lengths are valid
// and its table of max_pages entries is wide enough.
struct Need {
    int64_t have;    // pages of the cached tokens
    int64_t take;    // pages more
    bool fits;       // lengths valid, table wide enough
};
W4_HD Need page_need(int64_t len, int64_t fresh, int64_t page, int64_t max_pages) {   // page: a power of two
    Need d;
    const int shift = __builtin_ctzll((unsigned long long)page);
    d.have = d.take = 0;
    d.fits = len >= 0 && fresh >= 0;
    if (!d.fits) return d;
    d.have = (len + page - 1) >> shift;
    const int64_t want = (len + fresh + page - 1) >> shift;
    d.fits = want <= max_pages && len + fresh <= INT32_MAX;
    d.take = d.fits ? want - d.have : 0;
    return d;
}

}  // namespace w4

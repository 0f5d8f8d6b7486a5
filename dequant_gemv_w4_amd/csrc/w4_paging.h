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

// Keys of a tile of rows [row0, row0 + rows) of a sequence (rows >= 1), and their split:
// [first, end) is what any row sees, begin is first rounded down to a multiple of kKeyTile; part p of
// `parts` takes [begin + p * chunk, begin + (p + 1) * chunk).  The parts are cut by the actual
// lengths, at least `least` keys each and none below twice that, whatever number the launch allows.
constexpr int kKeyTile = 64;
struct Span {
    int32_t first, begin, end, chunk, parts;
};
W4_HD Span key_span(const Seq& s, int32_t row0, int32_t rows, int32_t G, int32_t window,
                    int32_t max_parts, int32_t least) {
    Span k;
    const int32_t pos0 = s.ctx - s.n;                        // position of the first new token
    k.end = lesser(s.ctx, pos0 + quotient(row0 + rows - 1, G) + 1);
    k.first = window > 0 ? greater(0, pos0 + quotient(row0, G) - window + 1) : 0;
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

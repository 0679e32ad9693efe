// kv_index.hpp -- the paged 8-bit key/value cache: its layout, and how rows of a batch find
// their sequence, position and page.  Integer arithmetic only, for host and device, so that
// the walk over pages and tiles can be checked without a GPU.
//
// kv [pages, kv_heads, 2, page * head_dim] bytes: of each page and head the keys, then the
// values.  Bytes hold code + 128, code in [-127, 127].  Both parts are tiles of 16 tokens
// (16 * head_dim bytes), a tile is chunks of 64 elements (1024 bytes; the last one 32 wide,
// 512 bytes, where head_dim % 64 == 32), and a chunk is one record of 16 (8) bytes for each
// lane of a wavefront, at lane * 16 (8):
//   keys    lane = token + 16 g: elements 16 g .. 16 g + 15 (8 g .. 8 g + 7) of the chunk
//   values  lane = e + 16 g: byte 4 j + i is element 16 j + e of token 4 g + i
// So a wavefront reads a chunk as 1024 consecutive bytes, and each lane then holds its part
// of the operands of v_mfma_f32_16x16x32_f16: of K as A[token][element], twice 8 elements,
// and of V^T as A[element][token], four tokens for each of four tiles of 16 elements, in
// the order in which the product K Q^T leaves its results (lane q + 16 g: tokens 4 g .. + 3).
// scale [pages, kv_heads, 2]: the keys' and the values' scale, value = code * scale.
#pragma once

#include <stdint.h>

#ifdef __HIPCC__
#include <hip/hip_runtime.h>
#define KV_INLINE __host__ __device__ __forceinline__
#else
#define KV_INLINE inline
#endif

namespace w4a8 {

template <class T>
KV_INLINE T kv_min(T a, T b) { return a < b ? a : b; }
template <class T>
KV_INLINE T kv_max(T a, T b) { return a < b ? b : a; }

// Offset of element d (a multiple of 8) of token r in a 16-token tile of keys: 8 bytes.
KV_INLINE int kv8_key_offset(int r, int d, int dim) {
    const int c = d >> 6, in = d & 63;
    if (dim - (c << 6) >= 64) return c * 1024 + (((in >> 4) << 4) + r) * 16 + (in & 15);
    return c * 1024 + (((in >> 3) << 4) + r) * 8;
}
// Offset of tokens 4 g .. 4 g + 3 of element d in a 16-token tile of values: 4 bytes.
KV_INLINE int kv8_value_offset(int g, int d, int dim) {
    const int c = d >> 6, in = d & 63;
    const int lane = (g << 4) + (d & 15);
    return c * 1024 + lane * (dim - (c << 6) >= 64 ? 16 : 8) + ((in >> 4) << 2);
}

// Rows of a batch: sequence s has rows start[s] .. start[s + 1] - 1 (one row, s, where
// start is null), its last tokens: row i of n is token len - n + i.
struct KvBatch {
    const int32_t *start, *lens, *table;
    int64_t ldb;                   // entries from one sequence's block table to the next
    int32_t seqs, blocks, pages;   // blocks: entries of a sequence's table
    int32_t rows;                  // of the whole batch
    int page_shift;
};
struct KvSeq {
    int32_t first_row, n, len;
};
// Whatever the arrays hold, the rows stay inside the batch.
KV_INLINE KvSeq kv_seq(const KvBatch &b, int s) {
    int lo = s, hi = s + 1;
    if (b.start) {
        lo = b.start[s];
        hi = b.start[s + 1];
    }
    lo = kv_max(0, kv_min(lo, b.rows));
    hi = kv_max(lo, kv_min(hi, b.rows));
    return KvSeq{lo, hi - lo, kv_max(0, b.lens[s])};
}
// The page of block `at` of sequence s, or -1 (outside the table, or no page of the cache).
KV_INLINE int kv_page(const KvBatch &b, int s, int64_t at) {
    if (at < 0 || at >= b.blocks) return -1;
    const int p = b.table[s * b.ldb + at];
    return p >= 0 && p < b.pages ? p : -1;
}

// How many of the 64 lanes hold: a ballot on the device (every lane of the wavefront calls
// it), a loop on the host.
template <class F>
KV_INLINE int kv_count64(F holds) {
#ifdef __HIP_DEVICE_COMPILE__
    return __popcll(__ballot(holds((int)__lane_id())));
#else
    int n = 0;
    for (int lane = 0; lane < 64; ++lane) n += holds(lane) ? 1 : 0;
    return n;
#endif
}

// Work items of ragged sequences without a table of them: sequence s takes the items from
// base(s) = (start[s] * num >> shift) + extra * s on, `extra` enough that base(s + 1) -
// base(s) covers what its rows need; a launch holds base(seqs) of them with start[seqs] =
// rows.  Returns the last sequence with base(s) <= item, 64 candidates at a time: one load
// deep for 64 sequences, where a bisection is six dependent ones.
KV_INLINE int64_t kv_base(const KvBatch &b, int s, int num, int shift, int extra) {
    const int64_t st = b.start ? kv_max(0, kv_min(b.start[s], b.rows)) : s;
    return ((st * num) >> shift) + (int64_t)extra * s;
}
KV_INLINE int kv_find_seq(const KvBatch &b, int64_t item, int num, int shift, int extra,
                          int64_t &base) {
    int lo = 0, n = b.seqs;
    while (n > 1) {
        const int step = (int)(((int64_t)n + 63) / 64);
        int below = kv_count64([&](int lane) {
            const int64_t at = (int64_t)lane * step;
            return at < n && kv_base(b, lo + (int)at, num, shift, extra) <= item;
        });
        below = kv_max(below, 1) - 1;
        lo += below * step;
        n = kv_min(step, n - below * step);
    }
#ifdef __HIP_DEVICE_COMPILE__
    lo = __builtin_amdgcn_readfirstlane(lo);
#endif
    base = kv_base(b, lo, num, shift, extra);
    return lo;
}

// A page that rows of a sequence reach: n rows touch at most n / page + 2 of them.
struct KvPageItem {
    int page;                      // -1: none
    int first, last;               // the rows' tokens, counted in the page (none: 0, 0)
    int64_t row;                   // the row of token `first`
};
KV_INLINE int64_t kv_page_items(int64_t rows, int64_t seqs, bool ragged, int page) {
    return ragged ? rows / page + 2 * seqs : seqs;
}
KV_INLINE KvPageItem kv_page_item(const KvBatch &b, int64_t item) {
    KvPageItem it{-1, 0, 0, 0};
    int64_t base = item;
    int s = (int)item;
    if (b.start) s = kv_find_seq(b, item, 1, b.page_shift, 2, base);
    const KvSeq q = kv_seq(b, s);
    const int from = q.len - q.n;                                 // position of its first row
    const int64_t block = (int64_t)(kv_max(from, 0) >> b.page_shift) + (item - base);
    const int64_t at = block * ((int64_t)1 << b.page_shift);
    const int64_t t0 = kv_max((int64_t)kv_max(from, 0), at);
    const int64_t t1 = kv_min((int64_t)q.len, at + ((int64_t)1 << b.page_shift));
    if (t1 <= t0) return it;
    it.first = (int)(t0 - at);
    it.last = (int)(t1 - at);
    it.row = q.first_row + (t0 - from);
    it.page = kv_page(b, s, block);
    return it;
}

// A tile of attention: up to 1 << shift packed rows (row i of the sequence, head g of the
// group: i * group + g) from row0 on, and the tokens they see, [lo, hi).
struct KvTile {
    KvSeq seq;
    int s, row0, rows, lo, hi;
};
// tiles: of each sequence, or 0 (items found by kv_find_seq; then base(seqs) of them).
KV_INLINE int64_t kv_tile_items(int64_t rows, int64_t seqs, int64_t group, int shift) {
    return (rows * group >> shift) + seqs;
}
KV_INLINE bool kv_tile(const KvBatch &b, int64_t item, int tiles, int group, int shift,
                       int max_rows, bool causal, int window, KvTile &t) {
    int64_t base;
    if (tiles) {
        t.s = (int)(item / tiles);
        base = (int64_t)t.s * tiles;
    } else {
        t.s = kv_find_seq(b, item, group, shift, 1, base);
    }
    t.seq = kv_seq(b, t.s);
    const int64_t row0 = (item - base) * ((int64_t)1 << shift);
    const int64_t all = (int64_t)kv_min(t.seq.n, max_rows) * group;
    if (row0 < 0 || row0 >= all) return false;
    t.row0 = (int)row0;
    t.rows = (int)kv_min((int64_t)1 << shift, all - row0);
    const int from = t.seq.len - t.seq.n;
    const int64_t first = from + t.row0 / group, last = from + (t.row0 + t.rows - 1) / group;
    // without a page nothing is seen; with one, its first bytes may always be read
    const int64_t cap = b.pages > 0 ? kv_min((int64_t)t.seq.len, (int64_t)b.blocks << b.page_shift) : 0;
    t.hi = (int)kv_max((int64_t)0, causal ? kv_min(cap, last + 1) : cap);
    t.lo = window ? (int)kv_max((int64_t)0, kv_min((int64_t)t.hi, first - window + 1)) : 0;
    return true;
}

// Whether rows of sequence q see any of the 64 tokens from `run` * 64 on, so that bytes may be
// read for them: without a page not even the cache's first is there.
KV_INLINE bool kv_run_seen(const KvBatch &b, const KvSeq &q, int run, int window) {
    const int64_t first = window ? (int64_t)q.len - q.n - window + 1 : 0, at = (int64_t)run * 64;
    return b.pages > 0 && q.n > 0 && at < q.len && at + 64 > first;
}

}  // namespace w4a8

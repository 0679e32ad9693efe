// The index arithmetic of the paged cache on the host, for test_kv_index_host.py.
#include "kv_index.hpp"

using namespace w4a8;

static KvBatch batch(const int32_t *start, const int32_t *lens, const int32_t *table, int64_t ldb,
                     int seqs, int blocks, int pages, int rows, int shift) {
    return KvBatch{start, lens, table, ldb, seqs, blocks, pages, rows, shift};
}

extern "C" {
// Of every page item: {page, first, last, row}.  Returns the number of items.
int64_t page_items(const int32_t *start, const int32_t *lens, const int32_t *table, int64_t ldb,
                   int seqs, int blocks, int pages, int rows, int shift, int64_t *out) {
    const KvBatch b = batch(start, lens, table, ldb, seqs, blocks, pages, rows, shift);
    const int64_t items = kv_page_items(rows, seqs, start != nullptr, 1 << shift);
    for (int64_t i = 0; out && i < items; ++i) {
        const KvPageItem it = kv_page_item(b, i);
        out[4 * i] = it.page;
        out[4 * i + 1] = it.first;
        out[4 * i + 2] = it.last;
        out[4 * i + 3] = it.row;
    }
    return items;
}
// Of every tile: {found, s, first_row, n, row0, rows, lo, hi}.
int64_t tile_items(const int32_t *start, const int32_t *lens, const int32_t *table, int64_t ldb,
                   int seqs, int blocks, int pages, int rows, int shift, int tiles, int group,
                   int tile_shift, int max_rows, int causal, int window, int64_t *out) {
    const KvBatch b = batch(start, lens, table, ldb, seqs, blocks, pages, rows, shift);
    const int64_t items = tiles ? (int64_t)seqs * tiles : kv_tile_items(rows, seqs, group, tile_shift);
    for (int64_t i = 0; out && i < items; ++i) {
        KvTile t{};
        const bool ok = kv_tile(b, i, tiles, group, tile_shift, max_rows, causal, window, t);
        const int64_t v[8] = {ok, t.s, t.seq.first_row, t.seq.n, t.row0, t.rows, t.lo, t.hi};
        for (int k = 0; k < 8; ++k) out[8 * i + k] = v[k];
    }
    return items;
}
int key_offset(int token, int d, int dim) {
    return token / 16 * 16 * dim + kv8_key_offset(token % 16, d, dim);
}
int value_offset(int token, int d, int dim) {
    return token / 16 * 16 * dim + kv8_value_offset(token % 16 / 4, d, dim) + token % 4;
}
}

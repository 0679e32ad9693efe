// Which runs of 64 tokens are converted to halves, on the host, for test_kv_run_host.py.
#include "kv_index.hpp"

using namespace w4a8;

extern "C" int run_seen(int seqs, const int32_t *start, const int32_t *lens, int pages, int rows,
                        int s, int run, int window) {
    const KvBatch b{start, lens, nullptr, 0, seqs, 0, pages, rows, 4};
    return kv_run_seen(b, kv_seq(b, s), run, window);
}

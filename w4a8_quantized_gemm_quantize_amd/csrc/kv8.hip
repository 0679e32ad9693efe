// kv8.hip -- writing keys and values into the paged 8-bit cache (kv_index.hpp) and reading them
// back (w4a8_kv8_write, w4a8_kv8_read in w4a8.h).
//
// One workgroup per page written to and head, so nothing is shared between workgroups: it
// takes the maximum of the new tokens' keys and of their values, decides the page's two
// scales, stores the codes, and takes older tokens' codes over to a scale that grew.
// Reading is the same walk backwards.
// Both are bound by memory from a few hundred rows on, by launch and load latency below.
#include "device_common.hpp"
#include "kv_index.hpp"
#include "launch.hpp"

namespace w4a8 {
namespace {

// Codes within +-127 as bytes code + 128.
__device__ __forceinline__ u32x2 biased8(const float f[8], float inv) {
    u32x2 c = codes8(f, inv);
    c.x ^= 0x80808080u;
    c.y ^= 0x80808080u;
    return c;
}
// Four bytes code + 128 times a ratio of scales, rounded half to even; only those of `mask`.
__device__ __forceinline__ uint32_t rescaled4(uint32_t w, float ratio, uint32_t mask) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float c = (float)(int)((w >> (8 * i)) & 0xffu) - 128.0f;
        r |= (uint32_t)(sat_rne_code(c * ratio, 127.0f) + 128) << (8 * i);
    }
    return (r & mask) | (w & ~mask);
}

// Maximum over the workgroup of two non-negative values.
template <int THREADS>
__device__ __forceinline__ void block_max2(float &a, float &b, uint32_t (*slot)[2]) {
    uint32_t x = wave_max_u32(__float_as_uint(a)), y = wave_max_u32(__float_as_uint(b));
    if constexpr (THREADS > 64) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
            slot[wave][0] = x;
            slot[wave][1] = y;
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < THREADS / 64; ++w) {
            x = max(x, slot[w][0]);
            y = max(y, slot[w][1]);
        }
    }
    a = __uint_as_float(x);
    b = __uint_as_float(y);
}

// The tokens of the 8 bytes at `off` of a page's keys or values: keys have one, values the
// four from there on.
__device__ __forceinline__ int unit_lane(int off, int dim, int &tile) {
    tile = off / (16 * dim);
    const int in = off - tile * 16 * dim, full = dim >> 6 << 10;
    return in < full ? (in & 1023) >> 4 : (in - full) >> 3;
}
__device__ __forceinline__ int key_unit_token(int off, int dim) {
    int tile;
    const int lane = unit_lane(off, dim, tile);
    return tile * 16 + (lane & 15);
}
__device__ __forceinline__ int value_unit_token(int off, int dim) {
    int tile;
    const int lane = unit_lane(off, dim, tile);
    return tile * 16 + (lane >> 4) * 4;
}

struct KvRows {
    KvBatch b;
    int64_t ldk, ldv;              // elements from one row to the next
    int heads, dim;
};

struct WriteArgs {
    KvRows r;
    const void *k, *v;
    uint8_t *kv;
    float *scale;
};

// Eight values of a row, as they are in memory.
template <bool BF16>
struct Raw8 {
    u32x4 w[BF16 ? 1 : 2];
    __device__ __forceinline__ void load(const void *p, int64_t at) {
        const u32x4 *q = (const u32x4 *)((const uint8_t *)p + at * (BF16 ? 2 : 4));
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i) w[i] = __builtin_nontemporal_load(q + i);
    }
    __device__ __forceinline__ void values(float f[8]) const {
        if constexpr (BF16) {
            bf16x8_to_f32(w[0], f);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i >> 2][i & 3]);
        }
    }
};

// ITEMS vectors of eight values a thread stay in registers between the maximum and the
// codes; a page of more is read twice.  The codes are put together in LDS as the page holds
// them and leave as runs of consecutive bytes.
template <int THREADS, int ITEMS, bool BF16>
__global__ __launch_bounds__(THREADS) void kv8_write_kernel(WriteArgs a) {
    extern __shared__ uint8_t codes[];                            // keys, values: page * dim bytes
    __shared__ uint32_t slot[THREADS / 64][2];
    const int head = blockIdx.x % a.r.heads;
    const KvPageItem it = kv_page_item(a.r.b, blockIdx.x / a.r.heads);
    const int dim = a.r.dim, vecs = dim >> 3, items = (it.last - it.first) * vecs;
    const int part = dim << a.r.b.page_shift;                     // bytes of the keys
    uint8_t *keys = a.kv + ((int64_t)it.page * a.r.heads + head) * 2 * part;
    float *scale = a.scale + ((int64_t)it.page * a.r.heads + head) * 2;

    Raw8<BF16> rk[ITEMS], rv[ITEMS];
    auto load = [&](int first) {
#pragma unroll
        for (int n = 0; n < ITEMS; ++n) {
            const int i = first + n * THREADS + threadIdx.x;
            if (i < items) {
                const int64_t row = it.row + i / vecs;
                const int at = head * dim + i % vecs * 8;
                rk[n].load(a.k, row * a.r.ldk + at);
                rv[n].load(a.v, row * a.r.ldv + at);
            }
        }
    };
    // the first loads go out before the page's number is there
    load(0);
    if (it.page < 0) return;
    float mk = 0.0f, mv = 0.0f, f[8];
    for (int first = 0; first < items; first += THREADS * ITEMS) {
        if (first > 0) load(first);
#pragma unroll
        for (int n = 0; n < ITEMS; ++n)
            if (first + n * THREADS + threadIdx.x < items) {
                rk[n].values(f);
                mk = fmaxf(mk, absmax_f32x8(f));
                rv[n].values(f);
                mv = fmaxf(mv, absmax_f32x8(f));
            }
    }
    float ok = 0.0f, ov = 0.0f;
    if (it.first > 0) {
        ok = scale[0];
        ov = scale[1];
    }
    block_max2<THREADS>(mk, mv, slot);
    float sk = mk / 127.0f, sv = mv / 127.0f, grow_k = 1.0f, grow_v = 1.0f;
    if (it.first > 0) {
        if (sk > ok) grow_k = ok / sk;
        else sk = ok;
        if (sv > ov) grow_v = ov / sv;
        else sv = ov;
    }
    __syncthreads();                                              // every thread has the scales
    if (threadIdx.x == 0) {
        scale[0] = sk;
        scale[1] = sv;
    }
    const float ik = sk > 0.0f ? 1.0f / sk : 0.0f, iv = sv > 0.0f ? 1.0f / sv : 0.0f;

    for (int first = 0; first < items; first += THREADS * ITEMS) {
        if (items > THREADS * ITEMS) load(first);
#pragma unroll
        for (int n = 0; n < ITEMS; ++n) {
            const int i = first + n * THREADS + threadIdx.x;
            if (i >= items) continue;
            const int t = it.first + i / vecs, d = i % vecs * 8, tile = (t >> 4) * 16 * dim;
            rk[n].values(f);
            *(u32x2 *)(codes + tile + kv8_key_offset(t & 15, d, dim)) = biased8(f, ik);
            rv[n].values(f);
            const u32x2 c = biased8(f, iv);
            uint8_t *l = codes + part + tile + kv8_value_offset((t & 15) >> 2, d, dim) + (t & 3);
            const int step = dim - (d & ~63) >= 64 ? 16 : 8;      // from element to element
#pragma unroll
            for (int e = 0; e < 8; ++e) l[e * step] = (uint8_t)((e < 4 ? c.x : c.y) >> (8 * (e & 3)));
        }
    }
    __syncthreads();
    // keys: 8 bytes belong to one token
    for (int off = ((grow_k != 1.0f ? 0 : it.first >> 4) * 16 * dim) + threadIdx.x * 8;
         off < ((it.last + 15) >> 4) * 16 * dim; off += THREADS * 8) {
        const int t = key_unit_token(off, dim);
        u32x2 *to = (u32x2 *)(keys + off);
        if (t >= it.first && t < it.last) {
            *to = *(const u32x2 *)(codes + off);
        } else if (grow_k != 1.0f && t < it.first) {
            u32x2 w = *to;
            w.x = rescaled4(w.x, grow_k, ~0u);
            w.y = rescaled4(w.y, grow_k, ~0u);
            *to = w;
        }
    }
    // values: to the same four tokens twice; of words that the rows only partly fill single bytes
    uint8_t *values = keys + part;
    for (int off = ((grow_v != 1.0f ? 0 : it.first >> 4) * 16 * dim) + threadIdx.x * 8;
         off < ((it.last + 15) >> 4) * 16 * dim; off += THREADS * 8) {
        const int t = value_unit_token(off, dim);
        const u32x2 c = *(const u32x2 *)(codes + part + off);
        if (t >= it.first && t + 4 <= it.last) {
            *(u32x2 *)(values + off) = c;
            continue;
        }
        if (grow_v != 1.0f && t < it.first) {
            const uint32_t older = t + 4 <= it.first ? ~0u : (1u << (8 * (it.first - t))) - 1u;
            u32x2 w = *(const u32x2 *)(values + off);
            w.x = rescaled4(w.x, grow_v, older);
            w.y = rescaled4(w.y, grow_v, older);
            *(u32x2 *)(values + off) = w;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int at = t + (e & 3);
            if (at >= it.first && at < it.last)
                values[off + e] = (uint8_t)((e < 4 ? c.x : c.y) >> (8 * (e & 3)));
        }
    }
}

// STREAM: past the caches.  A cache read back cold gains (65536 tokens of 8 heads of 128 to
// bf16: 73 us for 83), one just written loses (8191 tokens to binary32: 25 us for 18.5).
constexpr int64_t kStreamBytes = 64 << 20;
template <bool STREAM, class T>
__device__ __forceinline__ T load_once(const T *p) {
    return STREAM ? __builtin_nontemporal_load(p) : *p;
}

struct ReadArgs {
    KvRows r;
    const uint8_t *kv;
    const float *scale;
    void *k, *v;
    int bf16;
};

__device__ __forceinline__ void store8(void *p, int64_t at, bool bf16, const float f[8]) {
    if (bf16) {
        *(u32x4 *)((uint16_t *)p + at) =
            u32x4{bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]), bf16x2_rne(f[4], f[5]),
                  bf16x2_rne(f[6], f[7])};
    } else {
        *(f32x4 *)((float *)p + at) = f32x4{f[0], f[1], f[2], f[3]};
        *(f32x4 *)((float *)p + at + 4) = f32x4{f[4], f[5], f[6], f[7]};
    }
}

// Keys straight from the page, values through LDS.
constexpr int kReadThreads = 256;
template <bool STREAM>
__global__ __launch_bounds__(kReadThreads) void kv8_read_kernel(ReadArgs a) {
    extern __shared__ u32x4 page_v[];                             // page * dim bytes
    const int head = blockIdx.x % a.r.heads;
    const KvPageItem it = kv_page_item(a.r.b, blockIdx.x / a.r.heads);
    const int dim = a.r.dim, vecs = dim >> 3, tokens = it.last - it.first;
    if (tokens <= 0) return;
    const bool have = it.page >= 0;                               // no page: zeros
    const int part = dim << a.r.b.page_shift;
    const uint8_t *keys = a.kv + ((int64_t)it.page * a.r.heads + head) * 2 * part;
    const u32x4 *values = (const u32x4 *)(keys + part);
    float sk = 0.0f, sv = 0.0f;
    if (have) {
        const int t0 = it.first >> 4, t1 = (it.last + 15) >> 4;   // whole tiles
        for (int i = t0 * dim + threadIdx.x; i < t1 * dim; i += kReadThreads)
            page_v[i] = load_once<STREAM>(values + i);
        sk = a.scale[((int64_t)it.page * a.r.heads + head) * 2];
        sv = a.scale[((int64_t)it.page * a.r.heads + head) * 2 + 1];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < tokens * vecs; i += kReadThreads) {
        const int t = it.first + i / vecs, d = i % vecs * 8, tile = (t >> 4) * 16 * dim;
        const int64_t row = it.row + i / vecs;
        float f[8] = {0, 0, 0, 0, 0, 0, 0, 0}, g[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (have) {
            const u32x2 c = load_once<STREAM>(
                (const u32x2 *)(keys + tile + kv8_key_offset(t & 15, d, dim)));
            const uint8_t *l = (const uint8_t *)page_v + tile +
                               kv8_value_offset((t & 15) >> 2, d, dim) + (t & 3);
            const int step = dim - (d & ~63) >= 64 ? 16 : 8;      // from element to element
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                f[e] = ((float)(((e < 4 ? c.x : c.y) >> (8 * (e & 3))) & 0xffu) - 128.0f) * sk;
                g[e] = ((float)l[e * step] - 128.0f) * sv;
            }
        }
        store8(a.k, row * a.r.ldk + head * dim + d, a.bf16, f);
        store8(a.v, row * a.r.ldv + head * dim + d, a.bf16, g);
    }
}

}  // namespace

int64_t kv8_page_items(int64_t rows, int64_t seqs, bool ragged, int page) {
    return kv_page_items(rows, seqs, ragged, page);
}

static KvRows kv_rows(const KvCall &c, int64_t ldk, int64_t ldv) {
    KvRows r;
    r.b = KvBatch{c.start, c.lens, c.table, c.ldb, c.seqs, c.blocks, c.pages, (int32_t)c.rows,
                  __builtin_ctz(c.page)};
    r.ldk = ldk;
    r.ldv = ldv;
    r.heads = c.kv_heads;
    r.dim = c.dim;
    return r;
}

template <int THREADS, int ITEMS>
static void launch_write(const WriteArgs &a, bool bf16, uint32_t grid, size_t lds, hipStream_t s) {
    if (bf16) kv8_write_kernel<THREADS, ITEMS, true><<<grid, THREADS, lds, s>>>(a);
    else kv8_write_kernel<THREADS, ITEMS, false><<<grid, THREADS, lds, s>>>(a);
}

hipError_t launch_kv8_write(const KvCall &c, const void *k, int64_t ldk, const void *v, int64_t ldv,
                            bool bf16, uint8_t *kv, float *scale, hipStream_t stream) {
    const int64_t items = kv8_page_items(c.rows, c.seqs, c.start != nullptr, c.page);
    const WriteArgs a{kv_rows(c, ldk, ldv), k, v, kv, scale};
    const uint32_t grid = (uint32_t)(items * c.kv_heads);
    const size_t lds = (size_t)2 * c.page * c.dim;
    // vectors of a full page, or of the few rows that a sequence has on average
    const int64_t mean = c.seqs ? (c.rows + c.seqs - 1) / c.seqs : 0;
    const int64_t most = (mean < c.page ? mean : c.page) * c.dim / 8;
    if (most <= 64) launch_write<64, 1>(a, bf16, grid, lds, stream);
    else if (most <= 512) launch_write<256, 2>(a, bf16, grid, lds, stream);
    else if (most <= 1024) launch_write<256, 4>(a, bf16, grid, lds, stream);
    else launch_write<512, 4>(a, bf16, grid, lds, stream);
    return hipGetLastError();
}

hipError_t launch_kv8_read(const KvCall &c, const uint8_t *kv, const float *scale, void *k,
                           int64_t ldk, void *v, int64_t ldv, bool bf16, hipStream_t stream) {
    const int64_t items = kv8_page_items(c.rows, c.seqs, c.start != nullptr, c.page);
    ReadArgs a{kv_rows(c, ldk, ldv), kv, scale, k, v, bf16 ? 1 : 0};
    const dim3 grid((uint32_t)(items * c.kv_heads));
    const size_t lds = (size_t)c.page * c.dim;
    if (c.rows * c.kv_heads * c.dim * 2 > kStreamBytes)
        kv8_read_kernel<true><<<grid, kReadThreads, lds, stream>>>(a);
    else
        kv8_read_kernel<false><<<grid, kReadThreads, lds, stream>>>(a);
    return hipGetLastError();
}

}  // namespace w4a8

// kv8.hip -- writing keys and values into the paged 8-bit cache (kv_index.hpp) and reading them
// back (w4a8_kv8_write, w4a8_kv8_read in w4a8.h).
//
// One workgroup per page written to and head, so nothing is shared between workgroups: it
// takes the maximum of the new tokens' keys and of their values, decides the page's two
// scales, takes older tokens' codes over to a scale that grew, and stores the codes.
// Values go through LDS to their place in the layout.  Reading is the same walk backwards.
// Both are bound by memory from a few hundred rows on, by launch and load latency below.
#include "device_common.hpp"
#include "kv_index.hpp"
#include "launch.hpp"

namespace w4a8 {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void load8(const void *p, int64_t at, bool bf16, float f[8]) {
    if (bf16) {
        bf16x8_to_f32(*(const u32x4 *)((const uint16_t *)p + at), f);
    } else {
        const f32x4 a = *(const f32x4 *)((const float *)p + at);
        const f32x4 b = *(const f32x4 *)((const float *)p + at + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = a[i];
            f[4 + i] = b[i];
        }
    }
}

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
__device__ __forceinline__ void block_max2(float &a, float &b, uint32_t (*slot)[2]) {
    const int wave = threadIdx.x >> 6;
    const uint32_t x = wave_max_u32(__float_as_uint(a)), y = wave_max_u32(__float_as_uint(b));
    if ((threadIdx.x & 63) == 0) {
        slot[wave][0] = x;
        slot[wave][1] = y;
    }
    __syncthreads();
    uint32_t mx = 0, my = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) {
        mx = max(mx, slot[w][0]);
        my = max(my, slot[w][1]);
    }
    a = __uint_as_float(mx);
    b = __uint_as_float(my);
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
    int bf16;
};

__global__ __launch_bounds__(kThreads) void kv8_write_kernel(WriteArgs a) {
    extern __shared__ uint32_t codes_v[];                         // page * dim bytes
    __shared__ uint32_t slot[kThreads / 64][2];
    const int head = blockIdx.x % a.r.heads;
    const KvPageItem it = kv_page_item(a.r.b, blockIdx.x / a.r.heads);
    if (it.page < 0) return;
    const int dim = a.r.dim, vecs = dim >> 3, tokens = it.last - it.first;
    uint8_t *keys = a.kv + (((int64_t)it.page * a.r.heads + head) * 2 << a.r.b.page_shift) * dim;
    uint8_t *values = keys + ((int64_t)dim << a.r.b.page_shift);
    float *scale = a.scale + ((int64_t)it.page * a.r.heads + head) * 2;

    float mk = 0.0f, mv = 0.0f, f[8];
    for (int i = threadIdx.x; i < tokens * vecs; i += kThreads) {
        const int64_t row = it.row + i / vecs;
        const int at = head * dim + i % vecs * 8;
        load8(a.k, row * a.r.ldk + at, a.bf16, f);
        mk = fmaxf(mk, absmax_f32x8(f));
        load8(a.v, row * a.r.ldv + at, a.bf16, f);
        mv = fmaxf(mv, absmax_f32x8(f));
    }
    block_max2(mk, mv, slot);
    float sk = mk / 127.0f, sv = mv / 127.0f, rk = 1.0f, rv = 1.0f;
    if (it.first > 0) {
        const float ok = scale[0], ov = scale[1];
        if (sk > ok) rk = ok / sk;
        else sk = ok;
        if (sv > ov) rv = ov / sv;
        else sv = ov;
    }
    __syncthreads();                                              // scales are read
    if (threadIdx.x == 0) {
        scale[0] = sk;
        scale[1] = sv;
    }
    const float ik = sk > 0.0f ? 1.0f / sk : 0.0f, iv = sv > 0.0f ? 1.0f / sv : 0.0f;

    if (rk != 1.0f)
        for (int i = threadIdx.x; i < it.first * vecs; i += kThreads) {
            const int t = i / vecs, d = i % vecs * 8;
            u32x2 *p = (u32x2 *)(keys + (t >> 4) * 16 * dim + kv8_key_offset(t & 15, d, dim));
            u32x2 w = *p;
            w.x = rescaled4(w.x, rk, ~0u);
            w.y = rescaled4(w.y, rk, ~0u);
            *p = w;
        }
    for (int i = threadIdx.x; i < tokens * vecs; i += kThreads) {
        const int t = it.first + i / vecs, d = i % vecs * 8;
        const int64_t row = it.row + i / vecs;
        load8(a.k, row * a.r.ldk + head * dim + d, a.bf16, f);
        *(u32x2 *)(keys + (t >> 4) * 16 * dim + kv8_key_offset(t & 15, d, dim)) = biased8(f, ik);
        load8(a.v, row * a.r.ldv + head * dim + d, a.bf16, f);
        const u32x2 c = biased8(f, iv);
        uint8_t *l = (uint8_t *)codes_v + (t >> 4) * 16 * dim + (t & 3);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            l[kv8_value_offset((t & 15) >> 2, d + e, dim)] = (uint8_t)((e < 4 ? c.x : c.y) >> (8 * (e & 3)));
    }
    __syncthreads();
    // Words of four tokens; those that the rows only partly fill keep their other bytes.
    const int w0 = rv != 1.0f ? 0 : it.first >> 2, w1 = (it.last + 3) >> 2;
    for (int i = threadIdx.x; i < (w1 - w0) * dim; i += kThreads) {
        const int q = w0 + i / dim, d = i % dim;                   // tokens 4 q .. 4 q + 3
        const int off = (q >> 2) * 16 * dim + kv8_value_offset(q & 3, d, dim);
        uint32_t fresh = 0, older = 0;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (4 * q + t >= it.first && 4 * q + t < it.last) fresh |= 0xffu << (8 * t);
            if (4 * q + t < it.first) older |= 0xffu << (8 * t);
        }
        uint32_t w = 0;
        if (fresh != ~0u) {
            w = *(const uint32_t *)(values + off);
            if (rv != 1.0f) w = rescaled4(w, rv, older);
        }
        w = (w & ~fresh) | (codes_v[off >> 2] & fresh);
        *(uint32_t *)(values + off) = w;
    }
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

__global__ __launch_bounds__(kThreads) void kv8_read_kernel(ReadArgs a) {
    extern __shared__ u32x4 page_v[];                             // page * dim bytes
    const int head = blockIdx.x % a.r.heads;
    const KvPageItem it = kv_page_item(a.r.b, blockIdx.x / a.r.heads);
    const int dim = a.r.dim, vecs = dim >> 3, tokens = it.last - it.first;
    if (tokens <= 0) return;
    const bool have = it.page >= 0;                               // no page: zeros
    const uint8_t *keys = a.kv + (((int64_t)it.page * a.r.heads + head) * 2 << a.r.b.page_shift) * dim;
    const u32x4 *values = (const u32x4 *)(keys + ((int64_t)dim << a.r.b.page_shift));
    float sk = 0.0f, sv = 0.0f;
    if (have) {
        sk = a.scale[((int64_t)it.page * a.r.heads + head) * 2];
        sv = a.scale[((int64_t)it.page * a.r.heads + head) * 2 + 1];
        const int t0 = it.first >> 4, t1 = (it.last + 15) >> 4;   // whole tiles
        for (int i = t0 * dim + threadIdx.x; i < t1 * dim; i += kThreads) page_v[i] = values[i];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < tokens * vecs; i += kThreads) {
        const int t = it.first + i / vecs, d = i % vecs * 8;
        const int64_t row = it.row + i / vecs;
        float f[8] = {0, 0, 0, 0, 0, 0, 0, 0}, g[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (have) {
            const u32x2 c = *(const u32x2 *)(keys + (t >> 4) * 16 * dim + kv8_key_offset(t & 15, d, dim));
            const uint8_t *l = (const uint8_t *)page_v + (t >> 4) * 16 * dim + (t & 3);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                f[e] = ((float)(((e < 4 ? c.x : c.y) >> (8 * (e & 3))) & 0xffu) - 128.0f) * sk;
                g[e] = ((float)l[kv8_value_offset((t & 15) >> 2, d + e, dim)] - 128.0f) * sv;
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

hipError_t launch_kv8_write(const KvCall &c, const void *k, int64_t ldk, const void *v, int64_t ldv,
                            bool bf16, uint8_t *kv, float *scale, hipStream_t stream) {
    const int64_t items = kv8_page_items(c.rows, c.seqs, c.start != nullptr, c.page);
    WriteArgs a{kv_rows(c, ldk, ldv), k, v, kv, scale, bf16 ? 1 : 0};
    kv8_write_kernel<<<dim3((uint32_t)(items * c.kv_heads)), kThreads, (size_t)c.page * c.dim,
                       stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_kv8_read(const KvCall &c, const uint8_t *kv, const float *scale, void *k,
                           int64_t ldk, void *v, int64_t ldv, bool bf16, hipStream_t stream) {
    const int64_t items = kv8_page_items(c.rows, c.seqs, c.start != nullptr, c.page);
    ReadArgs a{kv_rows(c, ldk, ldv), kv, scale, k, v, bf16 ? 1 : 0};
    kv8_read_kernel<<<dim3((uint32_t)(items * c.kv_heads)), kThreads, (size_t)c.page * c.dim,
                      stream>>>(a);
    return hipGetLastError();
}

}  // namespace w4a8

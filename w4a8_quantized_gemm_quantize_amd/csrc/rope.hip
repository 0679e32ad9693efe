// rope.hip -- RMS norms of queries and keys per head with the position rotation in the same
// pass (w4a8_qk_norm_rope in w4a8.h).
//
// A group of lanes (a power of two, 8 elements each) holds one head: y = x * (1 / sqrt(mean
// x^2 + eps)) * w, the sum of squares over the group by lane swaps, then the pairs (a, b) of
// the first `rot` elements become (a c - b s, b c + a s).  Where pairs are half of rot apart,
// a lane of the rotated part holds four elements of each half instead of eight in a row, so
// that both of a pair are its own.  All in binary32 (the mean of up to 256 squares too), one
// rounding at the end.  Bound by memory for prompts, by launch and load latency in decode.
#include "device_common.hpp"
#include "launch.hpp"

namespace w4a8 {
namespace {

constexpr int kThreads = 256;

struct RopeArgs {
    const void *q, *k;
    void *qo, *ko;
    const float *qw, *kw, *table;
    const int32_t *pos;
    int64_t ldq, ldk, ldqo, ldko, tokens, max_pos;
    float eps, inv_dim;
    int q_heads, heads, dim, rot, interleaved, per_token;   // per_token: workgroups of a token
};

template <bool BF16>
__device__ __forceinline__ void load4(const void *p, int64_t at, float f[4]) {
    if constexpr (BF16) {
        const u32x2 w = *(const u32x2 *)((const uint16_t *)p + at);
        f[0] = __uint_as_float(w.x << 16);
        f[1] = __uint_as_float(w.x & 0xffff0000u);
        f[2] = __uint_as_float(w.y << 16);
        f[3] = __uint_as_float(w.y & 0xffff0000u);
    } else {
        const f32x4 w = *(const f32x4 *)((const float *)p + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = w[i];
    }
}
template <bool BF16>
__device__ __forceinline__ void store4(void *p, int64_t at, const float f[4]) {
    if constexpr (BF16)
        *(u32x2 *)((uint16_t *)p + at) = u32x2{bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3])};
    else
        *(f32x4 *)((float *)p + at) = f32x4{f[0], f[1], f[2], f[3]};
}

template <int LANES, bool BF16_IN, bool BF16_OUT>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_kernel(RopeArgs a) {
    const int64_t token = blockIdx.x / a.per_token;
    const int head = (int)(blockIdx.x % a.per_token) * (kThreads / LANES) + threadIdx.x / LANES;
    const int lane = threadIdx.x % LANES;
    const int64_t pos = a.rot ? a.pos[token] : 0;
    if (a.rot && (pos < 0 || pos >= a.max_pos)) return;     // the row is left as it was
    const bool is_q = head < a.q_heads;
    const bool live = head < a.heads && lane * 8 < a.dim;
    const int h = is_q ? head : head - a.q_heads;
    // its two runs of four elements
    const int half = a.rot >> 1;
    const bool turns = lane * 8 < a.rot;
    const bool split = turns && !a.interleaved;
    const int d0 = split ? lane * 4 : lane * 8;
    const int d1 = split ? half + lane * 4 : lane * 8 + 4;
    float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const float *w = is_q ? a.qw : a.kw;
    if (live) {
        const void *in = is_q ? a.q : a.k;
        const int64_t at = token * (is_q ? a.ldq : a.ldk) + (int64_t)h * a.dim;
        load4<BF16_IN>(in, at + d0, x);
        load4<BF16_IN>(in, at + d1, x + 4);
    }
    if (w) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(x[i], x[i], sum);
#pragma unroll
        for (int step = 1; step < LANES; step <<= 1) sum += __shfl_xor(sum, step);
        const float r = 1.0f / sqrtf(sum * a.inv_dim + a.eps);
        if (live) {
            float g[8];
            load4<false>(w, d0, g);
            load4<false>(w, d1, g + 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = x[i] * r * g[i];
        }
    }
    if (!live) return;
    if (turns) {
        const float *c = a.table + pos * a.rot + lane * 4;
        float cs[4], sn[4];
        load4<false>(c, 0, cs);
        load4<false>(c, half, sn);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float &p = a.interleaved ? x[2 * i] : x[i], &q = a.interleaved ? x[2 * i + 1] : x[4 + i];
            const float u = p * cs[i] - q * sn[i], v = q * cs[i] + p * sn[i];
            p = u;
            q = v;
        }
    }
    void *out = is_q ? a.qo : a.ko;
    const int64_t at = token * (is_q ? a.ldqo : a.ldko) + (int64_t)h * a.dim;
    store4<BF16_OUT>(out, at + d0, x);
    store4<BF16_OUT>(out, at + d1, x + 4);
}

template <int LANES>
void launch_lanes(const RopeArgs &a, bool in, bool out, uint32_t grid, hipStream_t s) {
    if (in && out) qk_norm_rope_kernel<LANES, true, true><<<grid, kThreads, 0, s>>>(a);
    else if (in) qk_norm_rope_kernel<LANES, true, false><<<grid, kThreads, 0, s>>>(a);
    else if (out) qk_norm_rope_kernel<LANES, false, true><<<grid, kThreads, 0, s>>>(a);
    else qk_norm_rope_kernel<LANES, false, false><<<grid, kThreads, 0, s>>>(a);
}

int lanes_of(int dim) {
    int l = 8;
    while (l * 8 < dim) l <<= 1;
    return l;
}

}  // namespace

int64_t qk_norm_rope_grid(int64_t tokens, int32_t heads, int32_t dim) {
    const int per = kThreads / lanes_of(dim);
    return tokens * ((heads + per - 1) / per);
}

hipError_t launch_qk_norm_rope(const void *q, int64_t ldq, const void *k, int64_t ldk, bool bf16_in,
                               const float *qw, const float *kw, float eps, const float *table,
                               const int32_t *pos, int64_t max_pos, int32_t rot, bool interleaved,
                               int64_t tokens, int32_t q_heads, int32_t kv_heads, int32_t dim,
                               void *qo, int64_t ldqo, void *ko, int64_t ldko, bool bf16_out,
                               hipStream_t stream) {
    const int lanes = lanes_of(dim), per = kThreads / lanes, heads = q_heads + kv_heads;
    RopeArgs a{q, k, qo, ko, qw, kw, table, pos, ldq, ldk, ldqo, ldko, tokens, max_pos, eps,
               1.0f / (float)dim, q_heads, heads, dim, rot, interleaved ? 1 : 0,
               (heads + per - 1) / per};
    const uint32_t grid = (uint32_t)qk_norm_rope_grid(tokens, heads, dim);
    if (lanes == 8) launch_lanes<8>(a, bf16_in, bf16_out, grid, stream);
    else if (lanes == 16) launch_lanes<16>(a, bf16_in, bf16_out, grid, stream);
    else launch_lanes<32>(a, bf16_in, bf16_out, grid, stream);
    return hipGetLastError();
}

}  // namespace w4a8

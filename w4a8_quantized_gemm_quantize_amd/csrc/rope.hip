// rope.hip -- RMS norms of queries and keys per head with the position rotation in the same
// pass (w4a8_qk_norm_rope in w4a8.h).
//
// A group of lanes (a power of two, 8 elements each) holds one head: y = x * (1 / sqrt(mean
// x^2 + eps)) * w, the sum of squares over the group by lane swaps, then the pairs (a, b) of
// the first `rot` elements become (a c - b s, b c + a s).  Where pairs are half of rot apart,
// a lane of the rotated part holds four elements of each half instead of eight in a row, so
// that both of a pair are its own.  All in binary32 (the mean of up to 256 squares too), one
// rounding at the end.  Bound by memory for prompts (8192 x 72 heads of 128: 5.1 TB/s in and
// out, what a copy reaches), by launch and load latency in decode.
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

// Sum over aligned groups of LANES (8, 16 or 32) lanes: lane swaps inside a row of 16.
template <int STEP>
__device__ __forceinline__ float swapped(float v) {
    constexpr int kCtrl[] = {0xb1, 0x4e, 0x141, 0x140};   // neighbour, pair, 8, 16 lanes mirrored
    return __uint_as_float(
        (uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), kCtrl[STEP], 0xf, 0xf, false));
}
template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
    v += swapped<0>(v);
    v += swapped<1>(v);
    v += swapped<2>(v);
    if constexpr (LANES >= 16) v += swapped<3>(v);
    if constexpr (LANES >= 32) v += __shfl_xor(v, 16);
    return v;
}

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
// The same for values that are read once.
template <bool BF16>
__device__ __forceinline__ void stream4(const void *p, int64_t at, float f[4]) {
    if constexpr (BF16) {
        const u32x2 w = __builtin_nontemporal_load((const u32x2 *)((const uint16_t *)p + at));
        f[0] = __uint_as_float(w.x << 16);
        f[1] = __uint_as_float(w.x & 0xffff0000u);
        f[2] = __uint_as_float(w.y << 16);
        f[3] = __uint_as_float(w.y & 0xffff0000u);
    } else {
        const f32x4 w = __builtin_nontemporal_load((const f32x4 *)((const float *)p + at));
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

template <int LANES, int TURN, bool BF16_IN, bool BF16_OUT>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_kernel(RopeArgs a) {
    constexpr int kHeads = kThreads / LANES;
    const int64_t token = blockIdx.x / a.per_token;
    const int part = (int)(blockIdx.x - token * a.per_token);
    const int lane = threadIdx.x % LANES;
    const int64_t pos = a.rot ? a.pos[token] : 0;
    if (a.rot && (pos < 0 || pos >= a.max_pos)) return;     // the row is left as it was
    const bool live = lane * 8 < a.dim;
    // its two runs of four elements
    const int half = a.rot >> 1;
    const bool turns = lane * 8 < a.rot;
    const bool split = turns && !a.interleaved;
    const int d0 = split ? lane * 4 : lane * 8;
    const int d1 = split ? half + lane * 4 : lane * 8 + 4;
    float w[2][8], cs[4], sn[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float *p = i ? a.kw : a.qw;
        if (p && live) {
            load4<false>(p, d0, w[i]);
            load4<false>(p, d1, w[i] + 4);
        }
    }
    if (turns) {
        const float *c = a.table + pos * a.rot + lane * 4;
        load4<false>(c, 0, cs);
        load4<false>(c, half, sn);
    }
    const int first = part * (kHeads * TURN) + threadIdx.x / LANES;
    float x[TURN][8];
#pragma unroll
    for (int n = 0; n < TURN; ++n) {
        const int head = first + n * kHeads;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[n][i] = 0.0f;
        if (live && head < a.heads) {
            const bool is_q = head < a.q_heads;
            const void *in = is_q ? a.q : a.k;
            const int64_t at = token * (is_q ? a.ldq : a.ldk) +
                               (int64_t)(is_q ? head : head - a.q_heads) * a.dim;
            stream4<BF16_IN>(in, at + d0, x[n]);
            stream4<BF16_IN>(in, at + d1, x[n] + 4);
        }
    }
#pragma unroll
    for (int n = 0; n < TURN; ++n) {
        const int head = first + n * kHeads;
        const bool is_q = head < a.q_heads;
        if (is_q ? a.qw != nullptr : a.kw != nullptr) {     // the same for a group of lanes
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(x[n][i], x[n][i], sum);
            sum = group_sum<LANES>(sum);
            const float mean = sum * a.inv_dim + a.eps;
            // the instruction takes subnormal numbers for 0
            const float r = mean < 0x1p-126f ? __builtin_amdgcn_rsqf(mean * 0x1p32f) * 0x1p16f
                                             : __builtin_amdgcn_rsqf(mean);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[n][i] = x[n][i] * r * (is_q ? w[0][i] : w[1][i]);
        }
        if (!live || head >= a.heads) continue;
        if (turns) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float &p = a.interleaved ? x[n][2 * i] : x[n][i];
                float &q = a.interleaved ? x[n][2 * i + 1] : x[n][4 + i];
                const float u = p * cs[i] - q * sn[i], v = q * cs[i] + p * sn[i];
                p = u;
                q = v;
            }
        }
        void *out = is_q ? a.qo : a.ko;
        const int64_t at = token * (is_q ? a.ldqo : a.ldko) +
                           (int64_t)(is_q ? head : head - a.q_heads) * a.dim;
        store4<BF16_OUT>(out, at + d0, x[n]);
        store4<BF16_OUT>(out, at + d1, x[n] + 4);
    }
}

template <int LANES, int TURN>
void launch_types(const RopeArgs &a, bool in, bool out, uint32_t grid, hipStream_t s) {
    if (in && out) qk_norm_rope_kernel<LANES, TURN, true, true><<<grid, kThreads, 0, s>>>(a);
    else if (in) qk_norm_rope_kernel<LANES, TURN, true, false><<<grid, kThreads, 0, s>>>(a);
    else if (out) qk_norm_rope_kernel<LANES, TURN, false, true><<<grid, kThreads, 0, s>>>(a);
    else qk_norm_rope_kernel<LANES, TURN, false, false><<<grid, kThreads, 0, s>>>(a);
}
template <int LANES>
void launch_lanes(const RopeArgs &a, int turn, bool in, bool out, uint32_t grid, hipStream_t s) {
    if (turn == 1) launch_types<LANES, 1>(a, in, out, grid, s);
    else launch_types<LANES, 2>(a, in, out, grid, s);
}

int lanes_of(int dim) {
    int l = 8;
    while (l * 8 < dim) l <<= 1;
    return l;
}
// Heads a lane takes: two keep twice the loads in flight and share the weights and the
// table's row (8192 x 72 heads of 128: 59.7 us for 73.3, three 60.9, five 58.3; 24 heads of
// 256: 45.1 for 47.3); while everything fits on the card at once one is the shorter chain
// (1 token 3.1 us for 3.6, 333 tokens 3.5 for 3.7).
int turn_of(int64_t tokens, int64_t heads, int lanes) {
    const int64_t per = kThreads / lanes;
    return tokens * ((heads + per - 1) / per) <= 4 * (int64_t)device_cu_count() ? 1 : 2;
}

}  // namespace

int64_t qk_norm_rope_grid(int64_t tokens, int32_t heads, int32_t dim) {
    const int lanes = lanes_of(dim), per = kThreads / lanes * turn_of(tokens, heads, lanes);
    return tokens * ((heads + per - 1) / per);
}

hipError_t launch_qk_norm_rope(const void *q, int64_t ldq, const void *k, int64_t ldk, bool bf16_in,
                               const float *qw, const float *kw, float eps, const float *table,
                               const int32_t *pos, int64_t max_pos, int32_t rot, bool interleaved,
                               int64_t tokens, int32_t q_heads, int32_t kv_heads, int32_t dim,
                               void *qo, int64_t ldqo, void *ko, int64_t ldko, bool bf16_out,
                               hipStream_t stream) {
    const int heads = q_heads + kv_heads, lanes = lanes_of(dim);
    const int turn = turn_of(tokens, heads, lanes), per = kThreads / lanes * turn;
    RopeArgs a{q, k, qo, ko, qw, kw, table, pos, ldq, ldk, ldqo, ldko, tokens, max_pos, eps,
               1.0f / (float)dim, q_heads, heads, dim, rot, interleaved ? 1 : 0,
               (heads + per - 1) / per};
    const uint32_t grid = (uint32_t)qk_norm_rope_grid(tokens, heads, dim);
    if (lanes == 8) launch_lanes<8>(a, turn, bf16_in, bf16_out, grid, stream);
    else if (lanes == 16) launch_lanes<16>(a, turn, bf16_in, bf16_out, grid, stream);
    else launch_lanes<32>(a, turn, bf16_in, bf16_out, grid, stream);
    return hipGetLastError();
}

}  // namespace w4a8

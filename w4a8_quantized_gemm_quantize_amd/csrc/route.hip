// route.hip -- routing rows to experts: scores, a balance bias, limited groups,
// the top_k experts by key and their weights (moe_route in w4a8.h).
//
// One wavefront per token: lane l holds the V logits of experts l V .. l V + V - 1
// (16-byte loads where the rows allow), so nothing but the results leaves the
// wavefront, and the lower lane, then the lower register, is the lower index.
// Keys are binary32 values mapped to unsigned integers of the same order
// (order_key), so a maximum is one v_max_u32 and an excluded expert is 0.
//
//   score   softmax: p_e = exp(x_e - max), s_e = p_e / fl32(sum p).  The sum is
//           taken in 64 bits: terms of 24 bits then add without a rounding that
//           depends on their order, so a score, and with it the choice between
//           near equals, is the same for every layout of the sum.
//           sigmoid: s_e = 1 / (1 + exp(-x_e)).
//   groups  the two largest keys of a group: in the lane, then over the group's
//           lanes by lane swaps where a group is a power of two of whole lanes,
//           else through LDS; a group's rank is the count of groups that beat it.
//   top k   top_k rounds of a wavefront maximum over all keys.  Which lane and
//           register holds it is scalar work on the comparison masks, beside the
//           vector pipe: 20 vector instructions a round for V = 4.
//
// Bound by instruction issue from a few thousand tokens (the reads take a few
// microseconds at most), by launch and load latency below.
#include "device_common.hpp"
#include "launch.hpp"

namespace w4a8 {
namespace {

// Unsigned integers in the order of the binary32 values, above 0; -0 and +0 are
// equal.  0 is left for what cannot be chosen: excluded experts and NaN or -inf
// keys (`ok` false for both).
__device__ __forceinline__ uint32_t order_key(float v, bool ok) {
    const int u = (int)__float_as_uint(v + 0.0f);      // -0 -> +0
    const uint32_t o = (uint32_t)u ^ ((uint32_t)(u >> 31) | 0x80000000u);
    return ok ? o : 0u;
}
__device__ __forceinline__ bool choosable(float v) { return v > -__builtin_inff(); }
__device__ __forceinline__ float key_value(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? (o ^ 0x80000000u) : ~o);
}

// Lane swaps inside a row of 16 lanes (vector instructions, no LDS traffic): with
// the neighbour, with the next pair, mirrored in 8 lanes, mirrored in 16.  Taken
// in this order each combines two halves that already agree within themselves.
template <int STEP>
__device__ __forceinline__ uint32_t swap_lanes(uint32_t w) {
    constexpr int kCtrl[] = {0xb1, 0x4e, 0x141, 0x140};
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, kCtrl[STEP], 0xf, 0xf, false);
}
template <int STEP>
__device__ __forceinline__ double swap_lanes(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    return __longlong_as_double((long long)(((uint64_t)swap_lanes<STEP>((uint32_t)(u >> 32)) << 32) |
                                            swap_lanes<STEP>((uint32_t)u)));
}
__device__ __forceinline__ double wave_sum_f64(double v) {
    v += swap_lanes<0>(v);
    v += swap_lanes<1>(v);
    v += swap_lanes<2>(v);
    v += swap_lanes<3>(v);
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    return v;
}

struct RouteArgs {
    const void *logits;
    const float *bias;
    int32_t *ids;
    float *weights;
    int64_t tokens, ld;
    int experts, top_k, groups, topk_groups, group_top;
    int per;                  // experts of a group
    uint32_t per_inv;         // e / per = (e * per_inv) >> 20 for e < 1024
    int group_shift;          // log2 of the lanes that rank a group
    int lane_groups;          // a group is that many whole lanes
    float scale;
    int renorm, vector;       // vector: whole V-wide loads stay aligned and in the row
};

constexpr int kRouteWaves = 4;
// Tokens of a launch, 64 work items each: the runtime runs a grid of 2^32 work items or
// more modulo 2^32 and reports no error.
constexpr int64_t kRouteLaunch = (int64_t)1 << 25;

// V values at p + i (clamped to the n there are; the lane's own past the end are
// excluded by the caller).
template <int V, bool BF16>
__device__ __forceinline__ void load_values(const void *p, int64_t base, int i, int n, bool vector,
                                            float (&x)[V]) {
    if constexpr (V >= 4) {
        if (vector) {
            const int at = i < n ? i : n - V;         // n % V == 0: whole vectors
            if constexpr (BF16) {
                const u32x2 *q = (const u32x2 *)((const uint16_t *)p + base + at);
#pragma unroll
                for (int v = 0; v < V / 4; ++v) {
                    const u32x2 w = q[v];
                    x[4 * v] = __uint_as_float(w.x << 16);
                    x[4 * v + 1] = __uint_as_float(w.x & 0xffff0000u);
                    x[4 * v + 2] = __uint_as_float(w.y << 16);
                    x[4 * v + 3] = __uint_as_float(w.y & 0xffff0000u);
                }
            } else {
                const f32x4 *q = (const f32x4 *)((const float *)p + base + at);
#pragma unroll
                for (int v = 0; v < V / 4; ++v) {
                    const f32x4 w = q[v];
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[4 * v + e] = w[e];
                }
            }
            return;
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int at = i + v < n ? i + v : n - 1;
        x[v] = BF16 ? bf16_to_f32(((const uint16_t *)p)[base + at])
                    : ((const float *)p)[base + at];
    }
}

// The two largest of this lane's pair and of the lane that `other` brings it.
template <class F>
__device__ __forceinline__ void merge2(uint32_t &m1, uint32_t &m2, F other) {
    const uint32_t o1 = other(m1), o2 = other(m2);
    m2 = max(max(m2, o2), min(m1, o1));
    m1 = max(m1, o1);
}

template <int V, bool SIGMOID, bool BF16>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(RouteArgs a) {
    // scores, and keys where groups are ranked through LDS, of each wavefront
    __shared__ __attribute__((aligned(16))) float lds_s[kRouteWaves][64 * V];
    __shared__ __attribute__((aligned(16))) uint32_t lds_k[kRouteWaves][64 * V];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
    if (t >= a.tokens) return;           // whole wavefronts; no barrier follows

    const bool use_score = a.bias != nullptr || a.groups > 1;
    const int e0 = lane * V;
    float x[V], b[V];
    load_values<V, BF16>(a.logits, t * a.ld, e0, a.experts, a.vector != 0, x);
#pragma unroll
    for (int v = 0; v < V; ++v) b[v] = 0.0f;
    if (a.bias) load_values<V, false>(a.bias, 0, e0, a.experts, a.experts % V == 0, b);

    // +inf counts as the largest finite value (inf - inf has none); ok: experts that
    // can be chosen
    bool ok[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        ok[v] = e0 + v < a.experts && choosable(x[v]);
        x[v] = __builtin_fminf(x[v], 3.40282347e38f);
    }
    float mx = 0.0f, sum = 1.0f;
    float s[V];
    uint32_t key[V];
    if (!SIGMOID || !use_score) {
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = order_key(x[v], ok[v]);
    }
    if constexpr (!SIGMOID) {
        uint32_t top = key[0];
#pragma unroll
        for (int v = 1; v < V; ++v) top = max(top, key[v]);
        mx = key_value(wave_max_u32(top));
        double part = 0.0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            s[v] = ok[v] ? expf(x[v] - mx) : 0.0f;
            part += (double)s[v];
        }
        sum = (float)wave_sum_f64(part);
    }
    if (use_score) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if constexpr (SIGMOID) s[v] = 1.0f / (1.0f + expf(-x[v]));
            else s[v] = s[v] / sum;
            const float k = s[v] + b[v];          // b is 0 without a bias: s itself
            key[v] = order_key(k, ok[v] && choosable(k));
            lds_s[wave][e0 + v] = s[v];
        }
    }

    if (a.groups > 1) {
        uint32_t m1 = 0u, m2 = 0u;
        const int lanes = 1 << a.group_shift;
        const int g = lane >> a.group_shift;
        if (a.lane_groups) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                m2 = max(m2, min(m1, key[v]));
                m1 = max(m1, key[v]);
            }
            if (lanes >= 2) merge2(m1, m2, [](uint32_t w) { return swap_lanes<0>(w); });
            if (lanes >= 4) merge2(m1, m2, [](uint32_t w) { return swap_lanes<1>(w); });
            if (lanes >= 8) merge2(m1, m2, [](uint32_t w) { return swap_lanes<2>(w); });
            if (lanes >= 16) merge2(m1, m2, [](uint32_t w) { return swap_lanes<3>(w); });
            if (lanes >= 32)
                merge2(m1, m2, [](uint32_t w) { return (uint32_t)__shfl_xor((int)w, 16); });
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) lds_k[wave][e0 + v] = key[v];
            __builtin_amdgcn_wave_barrier();
            if (g < a.groups)
                for (int i = lane & (lanes - 1); i < a.per; i += lanes) {
                    const uint32_t kk = lds_k[wave][g * a.per + i];
                    m2 = max(m2, min(m1, kk));
                    m1 = max(m1, kk);
                }
            for (int off = 1; off < lanes; off <<= 1)
                merge2(m1, m2, [off](uint32_t w) { return (uint32_t)__shfl_xor((int)w, off); });
        }
        // The sum of the group's largest keys; a key that is missing adds nothing.  No
        // key is -inf or NaN, so the sum is no NaN; one that falls to -inf (two keys
        // near the lowest value) still ranks above a group without any, which is 0.
        uint32_t rank_key = m1;
        if (a.group_top == 2 && m2) rank_key = order_key(key_value(m1) + key_value(m2), true);
        // Groups that beat this lane's: a larger sum, or an equal one of a lower
        // group.  Which lanes belong to higher groups is a scalar mask.
        int beaten = 0;
        uint64_t higher = ~0ull << lanes;                   // lanes of groups above o
        for (int o = 0; o < a.groups; ++o) {
            const uint32_t other = (uint32_t)__builtin_amdgcn_readlane((int)rank_key,
                                                                       o << a.group_shift);
            const uint64_t beats = __ballot(rank_key < other) |
                                   (__ballot(rank_key == other) & higher);
            beaten += __builtin_amdgcn_inverse_ballot_w64(beats) ? 1 : 0;
            higher <<= lanes;
        }
        const bool keep = g < a.groups && beaten < a.topk_groups;
        if (a.lane_groups) {
#pragma unroll
            for (int v = 0; v < V; ++v) key[v] = keep ? key[v] : 0u;
        } else {
            const uint64_t kept = __ballot(keep);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const uint32_t eg = ((uint32_t)(e0 + v) * a.per_inv) >> 20;
                const bool in = eg < (uint32_t)a.groups && ((kept >> (eg << a.group_shift)) & 1u);
                key[v] = in ? key[v] : 0u;
            }
        }
    }

    int my_id = -1, my_key = 0;
    uint32_t best = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) best = max(best, key[v]);
    for (int j = 0; j < a.top_k; ++j) {
        const uint32_t m = wave_max_u32(best);
        if (m == 0u) break;                       // nothing left to choose
        uint64_t has[V], any = 0u;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            has[v] = __ballot(key[v] == m);
            any |= has[v];
        }
        const uint64_t win = any & (0ull - any);  // the lowest lane
        uint64_t left = win;
        int reg = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint64_t hit = has[v] & left;   // at most one bit: its lowest register
            left &= ~hit;
            reg = hit ? v : reg;
            key[v] = __builtin_amdgcn_inverse_ballot_w64(hit) ? 0u : key[v];
        }
        best = key[0];
#pragma unroll
        for (int v = 1; v < V; ++v) best = max(best, key[v]);
        // lane j holds choice j
        my_id = lane == j ? (int)__builtin_ctzll(win) * V + reg : my_id;
        my_key = lane == j ? (int)m : my_key;
    }

    __builtin_amdgcn_wave_barrier();
    float w = 0.0f;
    if (my_id >= 0) {
        if (use_score) {
            w = lds_s[wave][my_id];
        } else {
            const float xv = key_value((uint32_t)my_key);
            if constexpr (SIGMOID) w = 1.0f / (1.0f + expf(-xv));
            else w = expf(xv - mx) / sum;
        }
    }
    if (a.renorm) {
        // lanes past top_k hold 0; the sum is the same tree for every top_k
        float total = w;
        total += __uint_as_float(swap_lanes<0>(__float_as_uint(total)));
        total += __uint_as_float(swap_lanes<1>(__float_as_uint(total)));
        total += __uint_as_float(swap_lanes<2>(__float_as_uint(total)));
        if (a.top_k > 8) total += __uint_as_float(swap_lanes<3>(__float_as_uint(total)));
        if (a.top_k > 16) total += __shfl_xor(total, 16);
        w = total > 0.0f ? w / total : 0.0f;
    }
    if (lane < a.top_k) {
        const int64_t i = t * a.top_k + lane;
        a.ids[i] = my_id;
        a.weights[i] = w * a.scale;
    }
}

template <int V, bool SIGMOID>
void launch_route_vt(const RouteArgs &a, bool bf16, unsigned grid, hipStream_t stream) {
    const dim3 block(64 * kRouteWaves);
    RouteArgs p = a;
    p.vector = V >= 4 && a.experts % V == 0 && a.ld % 4 == 0;
    // a group in whole lanes, a power of two of them, at most 32
    const int lanes = a.per / V;
    p.lane_groups = a.groups > 1 && a.per % V == 0 && (lanes & (lanes - 1)) == 0 && lanes <= 32;
    if (p.lane_groups) p.group_shift = __builtin_ctz((unsigned)lanes);
    if (bf16) route_kernel<V, SIGMOID, true><<<grid, block, 0, stream>>>(p);
    else route_kernel<V, SIGMOID, false><<<grid, block, 0, stream>>>(p);
}

template <bool SIGMOID>
void launch_route_v(const RouteArgs &a, bool bf16, hipStream_t stream) {
    const unsigned grid = (unsigned)((a.tokens + kRouteWaves - 1) / kRouteWaves);
    if (a.experts <= 64) launch_route_vt<1, SIGMOID>(a, bf16, grid, stream);
    else if (a.experts <= 128) launch_route_vt<2, SIGMOID>(a, bf16, grid, stream);
    else if (a.experts <= 256) launch_route_vt<4, SIGMOID>(a, bf16, grid, stream);
    else if (a.experts <= 512) launch_route_vt<8, SIGMOID>(a, bf16, grid, stream);
    else launch_route_vt<16, SIGMOID>(a, bf16, grid, stream);
}

}  // namespace

hipError_t launch_route(const void *logits, bool bf16, int64_t ld, const float *bias,
                        int64_t tokens, int32_t experts, int32_t top_k, bool sigmoid,
                        int32_t groups, int32_t topk_groups, int32_t group_top, bool renorm,
                        float scale, int32_t *ids, float *weights, hipStream_t stream) {
    RouteArgs a;
    a.bias = bias;
    a.ld = ld;
    a.experts = experts;
    a.top_k = top_k;
    a.groups = groups;
    a.topk_groups = topk_groups;
    a.group_top = group_top;
    a.per = experts / groups;
    a.per_inv = (uint32_t)(((1u << 20) + a.per - 1) / a.per);
    a.group_shift = 6;
    while ((groups << a.group_shift) > 64) --a.group_shift;
    a.scale = scale;
    a.renorm = renorm;
    for (int64_t t0 = 0; t0 < tokens; t0 += kRouteLaunch) {
        a.logits = (const uint8_t *)logits + t0 * ld * (bf16 ? 2 : 4);
        a.ids = ids + t0 * top_k;
        a.weights = weights + t0 * top_k;
        a.tokens = tokens - t0 < kRouteLaunch ? tokens - t0 : kRouteLaunch;
        if (sigmoid) launch_route_v<true>(a, bf16, stream);
        else launch_route_v<false>(a, bf16, stream);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace w4a8

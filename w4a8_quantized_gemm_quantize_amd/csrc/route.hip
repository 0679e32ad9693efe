// route.hip -- routing rows to experts: scores, a balance bias, limited groups,
// the top_k experts by key and their weights (moe_route in w4a8.h).
//
// One wavefront per token: lane l holds the logits of experts l, l + 64, ... (V
// of them), so loads are whole lines and nothing but the results leaves the
// wavefront.  Keys are binary32 values mapped to unsigned integers of the same
// order (order_key), so a maximum is one v_max_u32 and an excluded expert is 0.
//
//   score   softmax: p_e = exp(x_e - max), s_e = p_e / fl32(sum p).  The sum is
//           taken in 64 bits: terms of 24 bits then add without a rounding that
//           depends on their order, so a score, and with it the choice between
//           near equals, is the same for every layout of the sum.
//           sigmoid: s_e = 1 / (1 + exp(-x_e)).
//   groups  lanes share a group's keys through LDS and keep its two largest; a
//           group's rank is the count of groups that beat it.
//   top k   top_k rounds of a wavefront maximum over all keys; the first lane of
//           the lowest slot that holds it wins, which is the lowest index.
//
// Bound by instruction issue (the reads are a few microseconds at most): about
// 20 instructions per round, 25 per score.
#include "device_common.hpp"
#include "launch.hpp"

namespace w4a8 {
namespace {

// Unsigned integers in the order of the binary32 values; -0 and +0 are equal,
// and every value that cannot be chosen (NaN, -inf) is 0.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);      // -0 -> +0
    const uint32_t o = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return v > -__builtin_inff() ? o : 0u;             // false for NaN
}
__device__ __forceinline__ float key_value(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? (o ^ 0x80000000u) : ~o);
}

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) v += __shfl_xor(v, off);
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
    int lanes_per_group;      // a power of two
    float scale;
    int bf16, renorm;
};

constexpr int kRouteWaves = 4;

template <int V, bool SIGMOID>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(RouteArgs a) {
    // scores, and keys while groups are ranked, of each wavefront's token
    __shared__ float lds_s[kRouteWaves][64 * V];
    __shared__ uint32_t lds_k[kRouteWaves][64 * V];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
    if (t >= a.tokens) return;           // whole wavefronts; no barrier follows

    const bool use_score = a.bias != nullptr || a.groups > 1;
    float x[V], b[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = v * 64 + lane;
        const bool in = e < a.experts;
        x[v] = -__builtin_inff();
        b[v] = 0.0f;
        if (in) {
            const int64_t i = t * a.ld + e;
            x[v] = a.bf16 ? bf16_to_f32(((const uint16_t *)a.logits)[i])
                          : ((const float *)a.logits)[i];
            if (a.bias) b[v] = a.bias[e];
        }
    }
    // +inf counts as the largest finite value (inf - inf has none)
    uint32_t ox[V], top = 0u;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        x[v] = x[v] > 3.40282347e38f ? 3.40282347e38f : x[v];
        ox[v] = order_key(x[v]);
        top = max(top, ox[v]);
    }
    float mx = 0.0f, sum = 1.0f;
    float s[V];
    if constexpr (SIGMOID) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (use_score) s[v] = 1.0f / (1.0f + expf(-x[v]));
    } else {
        mx = key_value(wave_max_u32(top));
        double part = 0.0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            s[v] = ox[v] ? expf(x[v] - mx) : 0.0f;
            part += (double)s[v];
        }
        sum = (float)wave_sum_f64(part);
        if (use_score) {
#pragma unroll
            for (int v = 0; v < V; ++v) s[v] = s[v] / sum;
        }
    }
    uint32_t key[V];
    if (use_score) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            key[v] = ox[v] ? order_key(a.bias ? s[v] + b[v] : s[v]) : 0u;
            lds_s[wave][v * 64 + lane] = s[v];
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = ox[v];
    }

    if (a.groups > 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) lds_k[wave][v * 64 + lane] = key[v];
        __builtin_amdgcn_wave_barrier();
        const int g = lane / a.lanes_per_group, sub = lane & (a.lanes_per_group - 1);
        uint32_t m1 = 0u, m2 = 0u;
        if (g < a.groups)
            for (int i = sub; i < a.per; i += a.lanes_per_group) {
                const uint32_t kk = lds_k[wave][g * a.per + i];
                m2 = max(m2, min(m1, kk));
                m1 = max(m1, kk);
            }
        for (int off = 1; off < a.lanes_per_group; off <<= 1) {
            const uint32_t o1 = (uint32_t)__shfl_xor((int)m1, off);
            const uint32_t o2 = (uint32_t)__shfl_xor((int)m2, off);
            m2 = max(max(m2, o2), min(m1, o1));
            m1 = max(m1, o1);
        }
        // the sum of the group's largest keys; a key that is missing adds nothing
        uint32_t rank_key = m1;
        if (a.group_top == 2 && m2) {
            const float both = key_value(m1) + key_value(m2);
            rank_key = order_key(both);
        }
        int beaten = 0;
        for (int o = 0; o < a.groups; ++o) {
            const uint32_t other =
                (uint32_t)__builtin_amdgcn_readlane((int)rank_key, o * a.lanes_per_group);
            beaten += (other > rank_key || (other == rank_key && o < g)) ? 1 : 0;
        }
        const bool keep = g < a.groups && sub == 0 && beaten < a.topk_groups;
        const uint64_t kept = __ballot(keep);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint32_t eg = ((uint32_t)(v * 64 + lane) * a.per_inv) >> 20;
            const bool in = eg < (uint32_t)a.groups &&
                            ((kept >> (eg * (uint32_t)a.lanes_per_group)) & 1u);
            key[v] = in ? key[v] : 0u;
        }
    }

    int my_id = -1;
    uint32_t my_key = 0u;
    uint32_t best = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) best = max(best, key[v]);
    for (int j = 0; j < a.top_k; ++j) {
        const uint32_t m = wave_max_u32(best);
        if (m == 0u) break;                       // nothing left to choose
        int id = 0;
        bool found = false;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint64_t has = __ballot(key[v] == m);
            if (!found && has) {
                const int l = __builtin_ctzll(has);
                id = v * 64 + l;
                found = true;
                if (lane == l) key[v] = 0u;
            }
        }
        best = key[0];
#pragma unroll
        for (int v = 1; v < V; ++v) best = max(best, key[v]);
        if (lane == j) {
            my_id = id;
            my_key = m;
        }
    }

    // lane j holds choice j
    __builtin_amdgcn_wave_barrier();
    float w = 0.0f;
    if (my_id >= 0) {
        if (use_score) {
            w = lds_s[wave][my_id];
        } else {
            const float xv = key_value(my_key);
            if constexpr (SIGMOID) w = 1.0f / (1.0f + expf(-xv));
            else w = expf(xv - mx) / sum;
        }
    }
    if (a.renorm) {
        float total = w;                          // lanes past top_k hold 0
        for (int off = 1; off < 32; off <<= 1) total += __shfl_xor(total, off);
        w = total > 0.0f ? w / total : 0.0f;
    }
    if (lane < a.top_k) {
        const int64_t i = t * a.top_k + lane;
        a.ids[i] = my_id;
        a.weights[i] = w * a.scale;
    }
}

template <bool SIGMOID>
void launch_route_v(const RouteArgs &a, hipStream_t stream) {
    const unsigned grid = (unsigned)((a.tokens + kRouteWaves - 1) / kRouteWaves);
    const dim3 block(64 * kRouteWaves);
    if (a.experts <= 64) route_kernel<1, SIGMOID><<<grid, block, 0, stream>>>(a);
    else if (a.experts <= 128) route_kernel<2, SIGMOID><<<grid, block, 0, stream>>>(a);
    else if (a.experts <= 256) route_kernel<4, SIGMOID><<<grid, block, 0, stream>>>(a);
    else if (a.experts <= 512) route_kernel<8, SIGMOID><<<grid, block, 0, stream>>>(a);
    else route_kernel<16, SIGMOID><<<grid, block, 0, stream>>>(a);
}

}  // namespace

hipError_t launch_route(const void *logits, bool bf16, int64_t ld, const float *bias,
                        int64_t tokens, int32_t experts, int32_t top_k, bool sigmoid,
                        int32_t groups, int32_t topk_groups, int32_t group_top, bool renorm,
                        float scale, int32_t *ids, float *weights, hipStream_t stream) {
    RouteArgs a;
    a.logits = logits;
    a.bias = bias;
    a.ids = ids;
    a.weights = weights;
    a.tokens = tokens;
    a.ld = ld;
    a.experts = experts;
    a.top_k = top_k;
    a.groups = groups;
    a.topk_groups = topk_groups;
    a.group_top = group_top;
    a.per = experts / groups;
    a.per_inv = (uint32_t)(((1u << 20) + a.per - 1) / a.per);
    a.lanes_per_group = 64;
    while (a.lanes_per_group * groups > 64) a.lanes_per_group >>= 1;
    a.scale = scale;
    a.bf16 = bf16;
    a.renorm = renorm;
    if (sigmoid) launch_route_v<true>(a, stream);
    else launch_route_v<false>(a, stream);
    return hipGetLastError();
}

}  // namespace w4a8

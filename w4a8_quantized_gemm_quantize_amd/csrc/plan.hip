// plan.hip -- sorting rows by the weights they choose and cutting each group
// into row tiles: the table that the products of experts.hip and lora.hip walk.
// The experts' layer quantizes its rows in the same launch.
#include "device_common.hpp"
#include "launch.hpp"

namespace w4a8 {
namespace {

// Workgroup g (0 .. groups) finds on its own what group g needs: how many rows
// each lower group has, so its first sorted row and its first tile, and its own
// rows in order (a stable sort: the result does not depend on timing).  Two passes
// over the ids from L2, counts of the lower groups in LDS, its own by ballots;
// no atomics on global memory and no second launch.  Workgroup `groups` clears the
// rest of the table and writes the entries and rows in use past its end.  rows /
// bm + min(groups, rows) entries are always enough, a count the host has without
// the ids.
//   none_last: ids outside [0, groups - 1) make up group groups - 1; else ids
// outside [0, groups) take no part.
//   Bound by the latency of the id loads: each wavefront requests kIdBatch of
// its 64-id chunks together (one at a time, 16384 rows took 16.8 us).
constexpr int kPlanThreads = 1024;
constexpr int kIdBatch = 8;

struct PlanArgs {
    const int32_t *ids;
    int32_t *order, *src;
    int4 *tiles;
    int rows, groups, none_last, top_k, bm, slots;
};

__device__ __forceinline__ int plan_group(int id, int groups, int none_last) {
    if (none_last) return id >= 0 && id < groups - 1 ? id : groups - 1;
    return id < groups ? id : -1;
}

__device__ __forceinline__ void plan_block(const PlanArgs &p, int g) {
    __shared__ int count[kPlanMaxGroups];
    __shared__ int eq_of[kPlanThreads / 64];
    __shared__ int sums[kPlanThreads / 64][2];
    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int waves = blockDim.x >> 6;
    // a contiguous run of whole 64-row chunks per wavefront
    const int chunks = (p.rows + 63) >> 6;
    const int per = (chunks + waves - 1) / waves;
    const int c0 = wave * per, c1 = c0 + per < chunks ? c0 + per : chunks;
    int id[kIdBatch];
    auto load = [&](int c) {
#pragma unroll
        for (int u = 0; u < kIdBatch; ++u) {
            const int i = (c + u) * 64 + lane;
            id[u] = c + u < c1 && i < p.rows ? p.ids[i] : -1;
        }
#pragma unroll
        for (int u = 0; u < kIdBatch; ++u) {
            const int i = (c + u) * 64 + lane;
            id[u] = c + u < c1 && i < p.rows ? plan_group(id[u], p.groups, p.none_last) : -1;
        }
    };
    load(c0);
    for (int w = tid; w < g; w += blockDim.x) count[w] = 0;
    __syncthreads();
    int eq = 0;
    for (int c = c0; c < c1; c += kIdBatch) {
        if (c > c0) load(c);
#pragma unroll
        for (int u = 0; u < kIdBatch; ++u) {
            if (id[u] >= 0 && id[u] < g) atomicAdd(&count[id[u]], 1);
            eq += __popcll(__ballot(id[u] == g));
        }
    }
    if (lane == 0) eq_of[wave] = eq;
    __syncthreads();
    // rows and tiles of the lower groups
    int part[2] = {0, 0};
    for (int w = tid; w < g; w += blockDim.x) {
        part[0] += count[w];
        part[1] += (count[w] + p.bm - 1) / p.bm;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        for (int off = 1; off < 64; off <<= 1) part[i] += __shfl_xor(part[i], off);
        if (lane == 0) sums[wave][i] = part[i];
    }
    __syncthreads();
    int before = 0, mine = 0, base = 0, first = 0;
    for (int w = 0; w < waves; ++w) {
        if (w == wave) base = mine;
        mine += eq_of[w];
        before += sums[w][0];
        first += sums[w][1];
    }
    if (g == p.groups) {
        for (int s = first + tid; s < p.slots; s += blockDim.x) p.tiles[s] = int4{0, 0, 0, 0};
        if (tid == 0) p.tiles[p.slots] = int4{first, before, 0, 0};
        return;
    }
    if (mine == 0) return;
    for (int s = tid; s * p.bm < mine; s += blockDim.x) {
        const int left = mine - s * p.bm;
        p.tiles[first + s] = int4{g, before + s * p.bm, left < p.bm ? left : p.bm, 0};
    }
    int at = before + base;
    for (int c = c0; c < c1; c += kIdBatch) {
        // one batch holds a short run whole: its ids are still in registers
        if (c1 - c0 > kIdBatch) load(c);
#pragma unroll
        for (int u = 0; u < kIdBatch; ++u) {
            const bool is = id[u] == g;
            const uint64_t m = __ballot(is);
            if (is) {
                const int i = (c + u) * 64 + lane;
                const int q = at + __popcll(m & ((1ull << lane) - 1));
                p.order[q] = i;
                if (p.src) p.src[q] = i / p.top_k;
            }
            at += __popcll(m);
        }
    }
}

__global__ __launch_bounds__(kPlanThreads) void plan_kernel(PlanArgs p) {
    plan_block(p, blockIdx.x);
}

// The plan in workgroups 0 .. groups, then the rows' codes and scales
// (act_scale_pair_rcp), a wavefront per row: neither depends on the other, and
// side by side they cost one launch and the longer of the two.  V vectors (8
// elements) per lane stay in registers; longer rows are read a second time.
template <int V>
__global__ __launch_bounds__(kPlanThreads) void plan_quantize_kernel(
    PlanArgs p, const u32x4 *__restrict__ x, int64_t xrows, int vecs, u32x2 *__restrict__ q,
    float *__restrict__ scales) {
    if ((int)blockIdx.x <= p.groups) {
        plan_block(p, blockIdx.x);
        return;
    }
    const int64_t b = blockIdx.x - p.groups - 1;
    const int64_t row = b * (blockDim.x >> 6) + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (row >= xrows) return;
    const u32x4 *xr = x + row * vecs;
    u32x4 v[V];
#pragma unroll
    for (int u = 0; u < V; ++u) {
        const int i = lane + u * 64;
        v[u] = xr[i < vecs ? i : vecs - 1];
    }
    float amax = 0.0f;
#pragma unroll
    for (int u = 0; u < V; ++u) {
        float f[8];
        bf16x8_to_f32(v[u], f);
        amax = __builtin_fmaxf(amax, absmax_f32x8(f));        // clamped repeats change nothing
    }
    for (int i = lane + V * 64; i < vecs; i += 64) {
        float f[8];
        bf16x8_to_f32(xr[i], f);
        amax = __builtin_fmaxf(amax, absmax_f32x8(f));
    }
    amax = __uint_as_float(wave_max_u32(__float_as_uint(amax)));
    float s, inv;
    act_scale_pair_rcp(amax, s, inv);
    u32x2 *qr = q + row * vecs;
#pragma unroll
    for (int u = 0; u < V; ++u) {
        const int i = lane + u * 64;
        if (i < vecs) {
            float f[8];
            bf16x8_to_f32(v[u], f);
            qr[i] = codes8(f, inv);
        }
    }
    for (int i = lane + V * 64; i < vecs; i += 64) {
        float f[8];
        bf16x8_to_f32(xr[i], f);
        qr[i] = codes8(f, inv);
    }
    if (lane == 0) scales[row] = s;
}

PlanArgs plan_args(const int32_t *ids, int64_t rows, int32_t groups, bool none_last,
                   int32_t top_k, int bm, int32_t *order, int32_t *src, int32_t *tiles) {
    return PlanArgs{ids,    order,     src,   (int4 *)tiles, (int)rows,
                    groups, none_last, top_k, bm,            (int)plan_slots(rows, groups, bm)};
}

// 16 wavefronts once each has a few chunks to read
int plan_threads(int64_t rows) { return rows >= 4096 ? kPlanThreads : 256; }

}  // namespace

int64_t plan_slots(int64_t rows, int64_t groups, int bm) {
    return rows / bm + (rows < groups ? rows : groups);
}

hipError_t launch_plan(const int32_t *ids, int64_t rows, int32_t groups, bool none_last,
                       int32_t top_k, int bm, int32_t *order, int32_t *src, int32_t *tiles,
                       hipStream_t stream) {
    plan_kernel<<<groups + 1, plan_threads(rows), 0, stream>>>(
        plan_args(ids, rows, groups, none_last, top_k, bm, order, src, tiles));
    return hipGetLastError();
}

hipError_t launch_plan_quantize(const int32_t *ids, int64_t rows, int32_t groups, int32_t top_k,
                                int bm, int32_t *order, int32_t *src, int32_t *tiles,
                                const uint16_t *x, int64_t xrows, int64_t cols, int8_t *q,
                                float *scales, hipStream_t stream) {
    const PlanArgs p = plan_args(ids, rows, groups, false, top_k, bm, order, src, tiles);
    const int threads = plan_threads(rows);
    const int64_t per = threads / 64;
    const unsigned grid = (unsigned)(groups + 1 + (xrows + per - 1) / per);
    const u32x4 *xv = (const u32x4 *)x;
    u32x2 *qv = (u32x2 *)q;
    const int vecs = (int)(cols / 8);
    if (vecs <= 64 * 4)
        plan_quantize_kernel<4><<<grid, threads, 0, stream>>>(p, xv, xrows, vecs, qv, scales);
    else if (vecs <= 64 * 8)
        plan_quantize_kernel<8><<<grid, threads, 0, stream>>>(p, xv, xrows, vecs, qv, scales);
    else
        plan_quantize_kernel<16><<<grid, threads, 0, stream>>>(p, xv, xrows, vecs, qv, scales);
    return hipGetLastError();
}

}  // namespace w4a8

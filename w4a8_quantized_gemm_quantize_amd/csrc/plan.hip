// plan.hip -- sorting rows by the weights they choose and cutting each group
// into row tiles: the table that the products of experts.hip and lora.hip walk.
#include "device_common.hpp"
#include "launch.hpp"

namespace w4a8 {
namespace {

// Workgroup g (0 .. groups) finds on its own what group g needs: how many rows
// go to lower groups (its first sorted row), which lower groups have any (its
// first tile) and its own rows in order (a stable sort: the result does not
// depend on timing).  Two passes over the ids from L2 with ballots and
// popcounts; no atomics on global memory and no second launch.
//   Tiles: group g starts at entry rows_before / bm + groups_with_rows_before.
// Since floor(a + b) >= floor(a) + ceil(b) - 1, the next group with rows starts
// at or after the end of g's ceil(rows / bm) tiles, and at most one entry
// between them stays unused (0 rows).  Workgroup `groups` clears the rest of
// the table.  So rows / bm + min(groups, rows) entries are enough, a count the
// host has without the ids.
//   none_last: ids outside [0, groups - 1) make up group groups - 1; else ids
// outside [0, groups) take no part.
constexpr int kPlanThreads = 1024;

__device__ __forceinline__ int plan_group(int id, int groups, int none_last) {
    if (none_last) return id >= 0 && id < groups - 1 ? id : groups - 1;
    return id < groups ? id : -1;
}

__global__ __launch_bounds__(kPlanThreads) void plan_kernel(
    const int32_t *__restrict__ ids, int rows, int groups, int none_last, int top_k, int bm,
    int slots, int32_t *__restrict__ order, int32_t *__restrict__ src, int4 *__restrict__ tiles) {
    __shared__ uint32_t seen[kPlanMaxGroups / 32];
    __shared__ int lt_of[kPlanThreads / 64], eq_of[kPlanThreads / 64];
    const int g = blockIdx.x;
    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int waves = blockDim.x >> 6;
    const int words = (groups + 31) >> 5;
    for (int w = tid; w < words; w += blockDim.x) seen[w] = 0u;
    __syncthreads();
    // a contiguous run of whole 64-row chunks per wavefront
    const int chunks = (rows + 63) >> 6;
    const int per = (chunks + waves - 1) / waves;
    const int c0 = wave * per, c1 = c0 + per < chunks ? c0 + per : chunks;
    int lt = 0, eq = 0;
    for (int c = c0; c < c1; ++c) {
        const int i = c * 64 + lane;
        const int id = i < rows ? plan_group(ids[i], groups, none_last) : -1;
        const bool low = id >= 0 && id < g;
        lt += __popcll(__ballot(low));
        eq += __popcll(__ballot(id == g));
        if (low) {
            const uint32_t bit = 1u << (id & 31);
            if (!(((volatile uint32_t *)seen)[id >> 5] & bit)) atomicOr(&seen[id >> 5], bit);
        }
    }
    if (lane == 0) {
        lt_of[wave] = lt;
        eq_of[wave] = eq;
    }
    __syncthreads();
    int before = 0, mine = 0, base = 0, active = 0;
    for (int w = 0; w < waves; ++w) {
        if (w == wave) base = mine;
        before += lt_of[w];
        mine += eq_of[w];
    }
    for (int w = 0; w < words; ++w) active += __popc(seen[w]);
    const int slot0 = before / bm + active;
    if (g == groups) {
        for (int s = slot0 + tid; s < slots; s += blockDim.x) tiles[s] = int4{0, 0, 0, 0};
        return;
    }
    if (mine == 0) return;
    const int slot1 = (before + mine) / bm + active + 1;
    for (int s = tid; s < slot1 - slot0; s += blockDim.x) {
        const int left = mine - s * bm;
        tiles[slot0 + s] = left > 0 ? int4{g, before + s * bm, left < bm ? left : bm, 0}
                                    : int4{0, 0, 0, 0};
    }
    int at = before + base;
    for (int c = c0; c < c1; ++c) {
        const int i = c * 64 + lane;
        const bool is = i < rows && plan_group(ids[i], groups, none_last) == g;
        const uint64_t m = __ballot(is);
        if (is) {
            const int p = at + __popcll(m & ((1ull << lane) - 1));
            order[p] = i;
            if (src) src[p] = i / top_k;
        }
        at += __popcll(m);
    }
}

}  // namespace

int64_t plan_slots(int64_t rows, int64_t groups, int bm) {
    return rows / bm + (rows < groups ? rows : groups);
}

hipError_t launch_plan(const int32_t *ids, int64_t rows, int32_t groups, bool none_last,
                       int32_t top_k, int bm, int32_t *order, int32_t *src, int32_t *tiles,
                       hipStream_t stream) {
    // 16 wavefronts once each has a few chunks to read
    const int threads = rows >= 4096 ? kPlanThreads : 256;
    plan_kernel<<<groups + 1, threads, 0, stream>>>(ids, (int)rows, groups, none_last, top_k, bm,
                                                    (int)plan_slots(rows, groups, bm), order, src,
                                                    (int4 *)tiles);
    return hipGetLastError();
}

}  // namespace w4a8

// lora.hip -- low-rank adapters of many requests beside a shared projection
// (w4a8_lora_add in w4a8.h): out[t] = y[t] + scale[l] B[l] (A[l] x[t]), l = ids[t].
//
// Both products walk row tiles, up to BM rows that share an adapter, so an adapter's
// A and B are read once per tile however the requests are mixed:
//   shrink  v = A x over one of `slices` parts of K: the four wavefronts split
//           the part, each holding the tile's whole v in accumulators, and add up
//           in LDS; the part's v goes to the workspace in binary32.
//   expand  sums the parts (in order), folds the adapter's scale in, and
//           multiplies by B on the matrix cores with y added in the epilogue.
// v stays binary32 throughout: the matrix cores take bf16, so it is split into
// three bf16 terms, which hold all 24 bits of it, each multiplied by the same B
// operand.  Two terms hold 16 bits: 1 in 450 to 1850 of the bf16 outputs then
// differed from the rounded 64-bit ones, with three 1 in 4000 or fewer, for at most
// 5 % of a call (64 rows, 4096 x 14336, rank 64: 28.3 -> 29.4 us).
//
// v_mfma_f32_16x16x32_bf16: lane (r = l % 16, q = l / 16) supplies row r of the
// first operand and column r of the second, both at k = 8 q .. 8 q + 7 (16
// bytes), and receives elements (4 q + i, r) of the result.  A rows, x rows
// and B rows are contiguous along that k, so every operand is one 16-byte load
// straight from memory.
//
// Row tiles: for up to 64 rows from one ballot (row t leads the tile of the 16 rows
// of its adapter that start with it) and expand sums the parts itself; for more,
// 64-row tiles from the plan (plan.hip; rows without an adapter are a group of
// their own, copied from y), and a pass between the two sums the parts and splits
// them once (every 256 columns of expand read the parts again before: 2.4 times
// the traffic of y itself at 2047 x 28672 x 8192, rank 32).
//   Both are bound by HBM (x once, y once in and out, A and B).
#include "device_common.hpp"
#include "launch.hpp"

namespace w4a8 {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

constexpr int kTerms = 3;                          // bf16 terms of a binary32 v

__device__ __forceinline__ f32x4 mfma_bf16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

struct LoraArgs {
    const uint16_t *x, *a, *b;
    const int32_t *ids;
    const float *scale;
    const void *y;
    void *out;
    float *part;              // [slices][slots][BM][RP]
    uint16_t *terms;          // plan form: v in bf16 terms [slots][kTerms][BM][32 RK]
    const int4 *tiles;        // plan form only
    const int32_t *order;
    int64_t ldx, ldy, ldo, k, n;
    int tokens, adapters, rank, slots, slices, kslice;
    int steps;                // 256-column steps of an expand workgroup
};

constexpr int kLoraWaves = 4;

// Workgroup barrier that waits for this wavefront's LDS operations only: global
// loads stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_s_waitcnt(0xc07f);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// The rows of tile `slot`: their indices into `rows` (LDS, padded with the last
// one), their count and adapter (>= adapters: none).  False: no rows.
template <int BM, bool PLAN>
__device__ __forceinline__ bool tile_rows(const LoraArgs &p, int slot, int *rows, int &count,
                                          int &adapter) {
    const int tid = threadIdx.x;
    if constexpr (PLAN) {
        const int4 t = p.tiles[slot];
        count = t.z;
        adapter = t.x;
        if (count == 0) return false;
        if (tid < BM) rows[tid] = p.order[t.y + (tid < count ? tid : count - 1)];
    } else {
        static_assert(BM == 16, "one ballot");
        const int lane = tid & 63;
        const int id = lane < p.tokens ? p.ids[lane] : -2;
        const int norm = lane < p.tokens ? (id >= 0 && id < p.adapters ? id : p.adapters) : -1;
        adapter = __builtin_amdgcn_readlane(norm, slot);
        const uint64_t same = __ballot(norm == adapter);
        const int before = __popcll(same & ((1ull << slot) - 1));
        if (before & 15) return false;                  // in an earlier row's tile
        const int after = __popcll(same) - before;
        count = after < 16 ? after : 16;
        if (tid < 64) {
            const int rank = __popcll(same & ((1ull << lane) - 1)) - before;
            if (norm == adapter && rank >= 0 && rank < 16) {
                rows[rank] = lane;
                if (rank == count - 1)
                    for (int i = count; i < BM; ++i) rows[i] = lane;
            }
        }
    }
    __syncthreads();
    return true;
}

// ----------------------------------------------------------------- shrink --
// acc += A x over k in [k0, kend) for the tile's rows (LDS) by one wavefront: lane
// (r, q) ends with ranks 16 i + 4 q .. of row 16 j + r.
template <int RT, int MT, int U>
__device__ __forceinline__ void shrink_part(const LoraArgs &p, const int *rows, int adapter,
                                            int64_t k0, int64_t kend, f32x4 (&acc)[RT][MT]) {
    const int lane = threadIdx.x & 63;
    const int r = lane & 15, q = lane >> 4;
    const uint16_t *arow[RT], *xrow[MT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int ar = 16 * i + r < p.rank ? 16 * i + r : p.rank - 1;   // past rank: not used
        arow[i] = p.a + ((int64_t)adapter * p.rank + ar) * p.k + 8 * q;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) xrow[i] = p.x + (int64_t)rows[16 * i + r] * p.ldx + 8 * q;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    struct Batch {
        u32x4 a[U][RT], x[U][MT];
    };
    auto load = [&](Batch &t, int64_t at) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int i = 0; i < RT; ++i) t.a[u][i] = *(const u32x4 *)(arow[i] + at + 32 * u);
#pragma unroll
            for (int i = 0; i < MT; ++i) t.x[u][i] = *(const u32x4 *)(xrow[i] + at + 32 * u);
        }
    };
    auto multiply = [&](const Batch &t) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int j = 0; j < MT; ++j) acc[i][j] = mfma_bf16(t.a[u][i], t.x[u][j], acc[i][j]);
    };
    int64_t kk = k0;
    if (kk + 32 * U <= kend) {
        // two register sets in turn: one is requested before the other is used
        Batch b0, b1;
        load(b0, kk);
        while (true) {
            const bool more1 = kk + 64 * U <= kend;
            if (more1) load(b1, kk + 32 * U);
            __builtin_amdgcn_sched_barrier(0);
            multiply(b0);
            kk += 32 * U;
            if (!more1) break;
            const bool more0 = kk + 64 * U <= kend;
            if (more0) load(b0, kk + 32 * U);
            __builtin_amdgcn_sched_barrier(0);
            multiply(b1);
            kk += 32 * U;
            if (!more0) break;
        }
    }
    for (; kk < kend; kk += 32) {
        const bool in = kk + 8 * q < kend;                     // k % 8 == 0: whole vectors
        const int64_t at = in ? kk : kk - 8 * q;               // a valid place; zeroed below
        u32x4 av[RT], xv[MT];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            av[i] = *(const u32x4 *)(arow[i] + at);
            av[i] = in ? av[i] : u32x4{0u, 0u, 0u, 0u};
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            xv[i] = *(const u32x4 *)(xrow[i] + at);
            xv[i] = in ? xv[i] : u32x4{0u, 0u, 0u, 0u};
        }
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j) acc[i][j] = mfma_bf16(av[i], xv[j], acc[i][j]);
    }

}

template <int RT, int MT, bool PLAN>
__global__ __launch_bounds__(64 * kLoraWaves) void lora_shrink_kernel(LoraArgs p) {
    constexpr int BM = 16 * MT, RP = 16 * RT;
    // steps of 32 along K per load batch; two batches are in flight
    constexpr int U = RT + MT <= 3 ? 4 : RT + MT <= 6 ? 2 : 1;
    __shared__ int rows[BM];
    __shared__ f32x4 red[kLoraWaves][RT][64];
    int count, adapter;
    if (!tile_rows<BM, PLAN>(p, blockIdx.x, rows, count, adapter)) return;
    if (adapter >= p.adapters) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int r = lane & 15, q = lane >> 4;

    // this wavefront's part of the slice
    const int64_t s0 = (int64_t)blockIdx.y * p.kslice;
    const int64_t s1 = s0 + p.kslice < p.k ? s0 + p.kslice : p.k;
    const int wpart = p.kslice / kLoraWaves;                   // a multiple of 32
    const int64_t k0 = s0 + (int64_t)wave * wpart;
    f32x4 acc[RT][MT];
    shrink_part<RT, MT, U>(p, rows, adapter, k0, k0 + wpart < s1 ? k0 + wpart : s1, acc);

    // the four wavefronts' sums, in order; lane (t = r, q) holds ranks 16 i + 4 q ..
    float *part = p.part + ((int64_t)blockIdx.y * p.slots + blockIdx.x) * (BM * RP);
#pragma unroll
    for (int j = 0; j < MT; ++j) {
        if (j > 0) __syncthreads();
#pragma unroll
        for (int i = 0; i < RT; ++i) red[wave][i][lane] = acc[i][j];
        __syncthreads();
        for (int i = wave; i < RT; i += kLoraWaves) {
            f32x4 v = red[0][i][lane];
#pragma unroll
            for (int w = 1; w < kLoraWaves; ++w) {
                const f32x4 o = red[w][i][lane];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = v[e] + o[e];
            }
            *(f32x4 *)(part + (16 * j + r) * RP + 16 * i + 4 * q) = v;
        }
    }
}

// ------------------------------------------------------------------ terms --
// Four ranks of scale * (sum of the parts, in order) as bf16 terms.
__device__ __forceinline__ void split_terms(f32x4 v, float sc, u32x2 (&t)[kTerms]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = v[e] * sc;
#pragma unroll
    for (int m = 0; m < kTerms; ++m) {
        t[m] = u32x2{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3])};
        v[0] = v[0] - __uint_as_float(t[m].x << 16);
        v[1] = v[1] - __uint_as_float(t[m].x & 0xffff0000u);
        v[2] = v[2] - __uint_as_float(t[m].y << 16);
        v[3] = v[3] - __uint_as_float(t[m].y & 0xffff0000u);
    }
}

// Four ranks of the parts, added in order; eight parts' loads in flight at a time.
__device__ __forceinline__ f32x4 sum_parts(const float *src, int slices, int64_t stride) {
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s0 = 0; s0 < slices; s0 += 8) {
        f32x4 o[8];
#pragma unroll
        for (int s = 0; s < 8; ++s)
            o[s] = *(const f32x4 *)(src + (s0 + s < slices ? s0 + s : slices - 1) * stride);
#pragma unroll
        for (int s = 0; s < 8; ++s)
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = s0 + s < slices ? v[e] + o[s][e] : v[e];
    }
    return v;
}

template <int RT>
__global__ __launch_bounds__(256) void lora_terms_kernel(LoraArgs p) {
    constexpr int BM = 64, RP = 16 * RT, RK = (RT + 1) / 2;
    constexpr int VEC = 8 * RK;                    // 4-rank pieces of a row
    const int4 tile = p.tiles[blockIdx.x];
    if (tile.z == 0 || tile.x >= p.adapters) return;
    const float sc = p.scale ? p.scale[tile.x] : 1.0f;
    const int64_t stride = (int64_t)p.slots * (BM * RP);
    const int i = blockIdx.y * 256 + threadIdx.x;
    const int t = i / VEC, c4 = (i - t * VEC) * 4;
    if (t >= tile.z) return;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c4 < p.rank)
        v = sum_parts(p.part + (int64_t)blockIdx.x * (BM * RP) + t * RP + c4, p.slices, stride);
    u32x2 w[kTerms];
    split_terms(v, sc, w);
#pragma unroll
    for (int m = 0; m < kTerms; ++m)
        *(u32x2 *)(p.terms + (((int64_t)blockIdx.x * kTerms + m) * BM + t) * (32 * RK) + c4) = w[m];
}

// ----------------------------------------------------------------- expand --
// Workgroup: 16 MT rows of a row tile (part blockIdx.z of the plan's) x `steps`
// times 256 columns, 64 per wavefront.  The four 16-row operand tiles of a
// wavefront take the B rows in the order (b_row) in which a 16-byte piece of the
// result is 4 consecutive columns of a lane, or 8 of two tiles for bf16, and the four
// lanes of a row hold 64 consecutive bytes: with 64 bytes of a row in one lane,
// written 16 at a time, expand of 2047 x 8192 binary32 took 39 us.  For decode
// batches the time is instructions and latencies as much as bytes (2.4 ns a dependent
// instruction), so B comes through buffer loads whose bounds replace the tests of
// rank and columns, and addresses only advance.
constexpr int kExpandN = 64 * kLoraWaves;

// The B row, of a wavefront's 64, that is row m of its operand tile f.
template <bool BF16>
__device__ __forceinline__ int b_row(int f, int m) {
    return BF16 ? (f >> 1) * 32 + (m >> 2) * 8 + (f & 1) * 4 + (m & 3) : f * 16 + m;
}
// Pieces of a row: piece c of lane q starts PER q columns into the row's c-th 64
// bytes.
constexpr int kPieceBytes = 64;

template <int RT, int MT, bool PLAN, bool BF16>
__global__ __launch_bounds__(64 * kLoraWaves) void lora_expand_kernel(LoraArgs p) {
    constexpr int BM = 16 * MT, RP = 16 * RT;
    constexpr int RK = (RT + 1) / 2;               // steps of 32 along the rank
    constexpr int VS = 32 * RK + 8;                // LDS row stride (bf16)
    constexpr int YV = BF16 ? 2 : 4;               // 16-byte pieces of 16 columns
    constexpr int PER = BF16 ? 8 : 4;              // columns of a piece
    constexpr int ES = BF16 ? 2 : 4;
    __shared__ int rows[PLAN ? 1 : BM];
    __shared__ __attribute__((aligned(16))) uint16_t vs[PLAN ? 1 : kTerms][PLAN ? 1 : BM][VS];
    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int r = lane & 15, q = lane >> 4;
    int count, adapter;
    int row[MT];
    if constexpr (PLAN) {
        const int4 tile = p.tiles[blockIdx.x];
        const int first = blockIdx.z * BM;
        adapter = tile.x;
        count = tile.z - first;
        if (count <= 0) return;
#pragma unroll
        for (int j = 0; j < MT; ++j)
            row[j] = p.order[tile.y + first + (16 * j + r < count ? 16 * j + r : count - 1)];
    } else {
        if (!tile_rows<BM, false>(p, blockIdx.x, rows, count, adapter)) return;
#pragma unroll
        for (int j = 0; j < MT; ++j) row[j] = rows[16 * j + r];
    }
    const bool none = adapter >= p.adapters;
    if (none && p.y == p.out) return;              // nothing to add or move
    int n0 = (int)blockIdx.y * p.steps * kExpandN + wave * 64;
    const int n = (int)p.n;
    const int nend = n0 + p.steps * kExpandN < n ? n0 + p.steps * kExpandN : n;
    const uint8_t *yp[MT];
    uint8_t *op[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) {
        yp[j] = (const uint8_t *)p.y + ((int64_t)row[j] * p.ldy + n0 + PER * q) * ES;
        op[j] = (uint8_t *)p.out + ((int64_t)row[j] * p.ldo + n0 + PER * q) * ES;
    }
    // y of the step's columns; in the row's last, partial step only what is there
    u32x4 yv[MT][YV];
    auto load_y = [&]() {
        if (n0 + 64 <= n) {
#pragma unroll
            for (int j = 0; j < MT; ++j)
#pragma unroll
                for (int c = 0; c < YV; ++c)
                    yv[j][c] = *(const u32x4 *)(yp[j] + c * kPieceBytes);
        } else {
#pragma unroll
            for (int j = 0; j < MT; ++j)
#pragma unroll
                for (int c = 0; c < YV; ++c)
                    if (n0 + (4 * c + q) * PER < n)
                        yv[j][c] = *(const u32x4 *)(yp[j] + c * kPieceBytes);
        }
    };
    auto store = [&](int j, int c, u32x4 v) {
        if (n0 + 64 <= n || n0 + (4 * c + q) * PER < n) *(u32x4 *)(op[j] + c * kPieceBytes) = v;
    };
    auto advance = [&]() {
        n0 += kExpandN;
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            yp[j] += kExpandN * ES;
            op[j] += kExpandN * ES;
        }
    };
    if (none) {                                    // copied
#pragma unroll 1
        while (n0 < nend) {
            load_y();
#pragma unroll
            for (int j = 0; j < MT; ++j)
#pragma unroll
                for (int c = 0; c < YV; ++c)
                    if (16 * j + r < count) store(j, c, yv[j][c]);
            advance();
        }
        return;
    }

    // B of the adapter: rows past n and ranks past the rank read zero
    const __amdgpu_buffer_rsrc_t rb =
        buffer_rsrc(p.b + (int64_t)adapter * n * p.rank, (uint32_t)(n * p.rank * 2));
    uint32_t boff[RK][4];
#pragma unroll
    for (int s = 0; s < RK; ++s)
#pragma unroll
        for (int f = 0; f < 4; ++f) {
            const int kk = 32 * s + 8 * q;         // rank % 8 == 0: whole vectors
            const uint32_t o =
                (uint32_t)((n0 + b_row<BF16>(f, r)) * p.rank + kk) * 2;
            boff[s][f] = kk < p.rank ? o : 0x80000000u;
        }
    const uint32_t bstep = (uint32_t)(kExpandN * p.rank * 2);
    u32x4 bv[RK][4];
    auto load_b = [&]() {
#pragma unroll
        for (int s = 0; s < RK; ++s)
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                bv[s][f] = buffer_load16(rb, (int)boff[s][f], 0);
                boff[s][f] += bstep;
            }
    };
    load_b();
    load_y();
    if constexpr (!PLAN) {
        // v in bf16 terms; zero past the rank
        const float sc = p.scale ? p.scale[adapter] : 1.0f;
        const float *part = p.part + (int64_t)blockIdx.x * (BM * RP);
        constexpr int VEC = 8 * RK;                // 4-rank pieces of a row
        for (int i = tid; i < count * VEC; i += 64 * kLoraWaves) {
            const int t = i / VEC, c4 = (i - t * VEC) * 4;
            f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
            if (c4 < p.rank)
                v = sum_parts(part + t * RP + c4, p.slices, (int64_t)p.slots * (BM * RP));
            u32x2 w[kTerms];
            split_terms(v, sc, w);
#pragma unroll
            for (int m = 0; m < kTerms; ++m) *(u32x2 *)&vs[m][t][c4] = w[m];
        }
        lds_barrier();                             // B and y stay in flight
    }
    const uint16_t *terms =
        p.terms + (int64_t)blockIdx.x * (kTerms * 64 * 32 * RK) + blockIdx.z * (BM * 32 * RK);
#pragma unroll 1
    while (true) {
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            if (16 * j >= count) break;
            f32x4 acc[4];
#pragma unroll
            for (int f = 0; f < 4; ++f) acc[f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            // rows past the count are never stored, and a row of v reaches no
            // other row of the result
            const int t = 16 * j + r < count ? 16 * j + r : count - 1;
#pragma unroll
            for (int m = kTerms - 1; m >= 0; --m)   // smallest terms first
#pragma unroll
                for (int s = 0; s < RK; ++s) {
                    u32x4 vt;
                    if constexpr (PLAN)
                        vt = *(const u32x4 *)(terms + (m * 64 + t) * (32 * RK) + 32 * s + 8 * q);
                    else
                        vt = *(const u32x4 *)&vs[m][t][32 * s + 8 * q];
#pragma unroll
                    for (int f = 0; f < 4; ++f) acc[f] = mfma_bf16(bv[s][f], vt, acc[f]);
                }
            if (16 * j + r >= count) continue;
#pragma unroll
            for (int c = 0; c < YV; ++c) {
                u32x4 o = yv[j][c];
                if constexpr (BF16) {
                    float f[8];
                    bf16x8_to_f32(o, f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = f[e] + acc[2 * c + (e >> 2)][e & 3];
                    o = u32x4{bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]),
                              bf16x2_rne(f[4], f[5]), bf16x2_rne(f[6], f[7])};
                } else {
                    f32x4 f = __builtin_bit_cast(f32x4, o);
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[e] = f[e] + acc[c][e];
                    o = __builtin_bit_cast(u32x4, f);
                }
                store(j, c, o);
            }
        }
        // out may be y: no two steps share a column
        advance();
        if (n0 >= nend) break;
        load_b();
        load_y();
    }
}

// ------------------------------------------------------------------ small --
// Both products of a small decode batch in one launch (one_launch), A of an adapter
// read by every workgroup of its rows (from L2): a row tile x 512 columns, eight
// wavefronts that split K and then the columns.  B and y are on their way while v is
// formed; v never leaves the workgroup.  Latency is all there is: ids, then A, x, B and
// y side by side, then the result.
constexpr int kSmallWaves = 8;
constexpr int kSmallN = 64 * kSmallWaves;

template <int RT, bool BF16>
__global__ __launch_bounds__(64 * kSmallWaves) void lora_small_kernel(LoraArgs p) {
    constexpr int BM = 16, RK = (RT + 1) / 2;
    constexpr int VS = 32 * RK + 8;                // LDS row stride (bf16)
    constexpr int YV = BF16 ? 2 : 4;               // 16-byte pieces of 16 columns
    constexpr int PER = BF16 ? 8 : 4;              // columns of a piece
    constexpr int ES = BF16 ? 2 : 4;
    __shared__ int rows[BM];
    __shared__ f32x4 red[kSmallWaves][RT][64];
    __shared__ __attribute__((aligned(16))) uint16_t vs[kTerms][BM][VS];
    int count, adapter;
    if (!tile_rows<BM, false>(p, blockIdx.x, rows, count, adapter)) return;
    const bool none = adapter >= p.adapters;
    if (none && p.y == p.out) return;              // nothing to add or move
    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int r = lane & 15, q = lane >> 4;
    const int n = (int)p.n;
    const int n0 = (int)blockIdx.y * kSmallN + wave * 64;
    const int col = n0 + PER * q;                  // of piece 0
    const int64_t row = rows[r];

    // B: rows past n and ranks past the rank read zero
    u32x4 bv[RK][4];
    if (!none) {
        const __amdgpu_buffer_rsrc_t rb =
            buffer_rsrc(p.b + (int64_t)adapter * n * p.rank, (uint32_t)(n * p.rank * 2));
#pragma unroll
        for (int s = 0; s < RK; ++s)
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                const int kk = 32 * s + 8 * q;     // rank % 8 == 0: whole vectors
                const uint32_t o =
                    (uint32_t)((n0 + b_row<BF16>(f, r)) * p.rank + kk) * 2;
                bv[s][f] = buffer_load16(rb, kk < p.rank ? (int)o : (int)0x80000000u, 0);
            }
    }
    u32x4 yv[YV];
#pragma unroll
    for (int c = 0; c < YV; ++c)
        if (col + 4 * c * PER < n)
            yv[c] = *(const u32x4 *)((const uint8_t *)p.y + (row * p.ldy + col) * ES +
                                     c * kPieceBytes);
    f32x4 sum[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) sum[f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (!none) {
        const int64_t part = ((p.k + 32 * kSmallWaves - 1) / (32 * kSmallWaves)) * 32;
        const int64_t k0 = wave * part;
        f32x4 acc[RT][1];
        shrink_part<RT, 1, RT == 1 ? 8 : RT == 2 ? 4 : 2>(
            p, rows, adapter, k0, k0 + part < p.k ? k0 + part : p.k, acc);
#pragma unroll
        for (int i = 0; i < RT; ++i) red[wave][i][lane] = acc[i][0];
        lds_barrier();
        // the wavefronts' sums, in order, as bf16 terms; an odd last step of 16
        // ranks is filled with zeros
        const float sc = p.scale ? p.scale[adapter] : 1.0f;
        for (int i = tid; i < 2 * RK * 64; i += 64 * kSmallWaves) {
            f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
            const int it = i >> 6;
            if (it < RT) {
#pragma unroll
                for (int w = 0; w < kSmallWaves; ++w) {
                    const f32x4 o = red[w][it][i & 63];
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = v[e] + o[e];
                }
            }
            u32x2 t[kTerms];
            split_terms(v, sc, t);
#pragma unroll
            for (int m = 0; m < kTerms; ++m)
                *(u32x2 *)&vs[m][i & 15][16 * it + 4 * ((i & 63) >> 4)] = t[m];
        }
        lds_barrier();
#pragma unroll
        for (int m = kTerms - 1; m >= 0; --m)       // smallest terms first
#pragma unroll
            for (int s = 0; s < RK; ++s) {
                const u32x4 vt = *(const u32x4 *)&vs[m][r][32 * s + 8 * q];
#pragma unroll
                for (int f = 0; f < 4; ++f) sum[f] = mfma_bf16(bv[s][f], vt, sum[f]);
            }
    }
    if (r >= count) return;
    uint8_t *dst = (uint8_t *)p.out + (row * p.ldo + col) * ES;
#pragma unroll
    for (int c = 0; c < YV; ++c) {
        if (col + 4 * c * PER >= n) break;
        u32x4 o = yv[c];
        if (!none) {
            if constexpr (BF16) {
                float f[8];
                bf16x8_to_f32(o, f);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = f[e] + sum[2 * c + (e >> 2)][e & 3];
                o = u32x4{bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]),
                          bf16x2_rne(f[4], f[5]), bf16x2_rne(f[6], f[7])};
            } else {
                f32x4 f = __builtin_bit_cast(f32x4, o);
#pragma unroll
                for (int e = 0; e < 4; ++e) f[e] = f[e] + sum[c][e];
                o = __builtin_bit_cast(u32x4, f);
            }
        }
        *(u32x4 *)(dst + c * kPieceBytes) = o;
    }
}

// ---------------------------------------------------------------- launches --
constexpr int64_t kBallotRows = 64;

// One launch (lora_small_kernel) where reading A again in every workgroup costs less
// than the second launch: by the elements of A (ranks padded) that a CU reads, at
// about 64 bytes a clock.  Measured, one launch | two, us per call (two are bound by the
// host at 14.7): 8 rows of rank 16, 4096 x 4096 12.1 | 15.2; 1 row, 8904 x 11040 11.9 |
// 14.9; 20 rows of rank 8, 6384 x 3096 12.2 | 14.8; 8 rows of rank 16, 8192 x 4096 14.2 |
// 14.6, 16384 x 4096 23.6 | 14.8; 4 rows of rank 64, 4096 x 4096 20.9 | 14.8; 32 rows of
// rank 32, 8192 x 8192 43 | 14.8; 64 rows of rank 16, 4096 x 14336 54 | 15.8.
constexpr int64_t kSmallA = 144 * 1024;
bool one_launch(int64_t tokens, int64_t adapters, int64_t rp, int64_t k, int64_t n) {
    if (tokens > kBallotRows || rp > 64) return false;
    const int64_t most = adapters + 1 + tokens / 16;           // row tiles
    const int64_t wgs = (tokens < most ? tokens : most) * ((n + kSmallN - 1) / kSmallN);
    const int64_t ncu = device_cu_count();
    return (wgs + ncu - 1) / ncu * rp * k <= kSmallA;
}

// Whether rows of x (xrow bytes each, xstep apart) and of out share memory.  Views of
// interleaved columns, one step for both, lie in each other's range and share none.
bool rows_overlap(const void *x, int64_t xstep, int64_t xrow, const void *out, int64_t ostep,
                  int64_t orow, int64_t tokens) {
    const int64_t xa = (int64_t)(uintptr_t)x, oa = (int64_t)(uintptr_t)out;
    if (xa + (tokens - 1) * xstep + xrow <= oa || oa + (tokens - 1) * ostep + orow <= xa)
        return false;
    if (xstep != ostep) return true;
    const int64_t d = ((oa - xa) % xstep + xstep) % xstep;      // out's row starts this far in
    return d < xrow || d + orow > xstep;
}

struct LoraSpace {
    bool plan;
    int bm, rp, slices, kslice;
    int64_t slots;
    size_t order, tiles, part, terms, end;
};

LoraSpace lora_space(int64_t tokens, int64_t adapters, int64_t rank, int64_t k) {
    LoraSpace s;
    s.plan = tokens > kBallotRows;
    s.bm = s.plan ? 64 : 16;
    s.rp = rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128;
    s.slots = s.plan ? plan_slots(tokens, adapters + 1, s.bm) : tokens;
    // about 768 workgroups, each wavefront at least 128 of K
    int64_t want = 768 / s.slots;
    const int64_t most = (k + 511) / 512;
    if (want > most) want = most;
    if (want > 16) want = 16;
    if (want < 1) want = 1;
    const int64_t unit = 32 * kLoraWaves;
    s.kslice = (int)(((k + want - 1) / want + unit - 1) / unit * unit);
    s.slices = (int)((k + s.kslice - 1) / s.kslice);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    s.order = take(s.plan ? (size_t)tokens * 4 : 0);
    s.tiles = take(s.plan ? (size_t)(s.slots + 1) * 16 : 0);
    s.part = take((size_t)s.slices * s.slots * s.bm * s.rp * 4);
    // whole steps of 32 ranks
    s.terms = take(s.plan ? (size_t)s.slots * kTerms * s.bm * (s.rp < 32 ? 32 : s.rp) * 2 : 0);
    s.end = at;
    return s;
}

template <bool BF16>
void launch_lora_small(const LoraArgs &p, int rp, hipStream_t stream) {
    const dim3 grid((unsigned)p.slots, (unsigned)((p.n + kSmallN - 1) / kSmallN));
    const dim3 block(64 * kSmallWaves);
    if (rp == 16) lora_small_kernel<1, BF16><<<grid, block, 0, stream>>>(p);
    else if (rp == 32) lora_small_kernel<2, BF16><<<grid, block, 0, stream>>>(p);
    else lora_small_kernel<4, BF16><<<grid, block, 0, stream>>>(p);
}

template <int RT, bool PLAN, bool BF16>
void launch_lora_form(const LoraArgs &p, hipStream_t stream) {
    const dim3 block(64 * kLoraWaves);
    const dim3 shrink((unsigned)p.slots, (unsigned)p.slices);
    const unsigned step_cols = (unsigned)(p.steps * kExpandN);
    const unsigned cols = (unsigned)((p.n + step_cols - 1) / step_cols);
    if constexpr (PLAN) {
        lora_shrink_kernel<RT, 4, true><<<shrink, block, 0, stream>>>(p);
        constexpr int RK = (RT + 1) / 2;
        lora_terms_kernel<RT>
            <<<dim3((unsigned)p.slots, 64 * 8 * RK / 256), 256, 0, stream>>>(p);
        lora_expand_kernel<RT, 2, true, BF16>
            <<<dim3((unsigned)p.slots, cols, 2), block, 0, stream>>>(p);
    } else {
        lora_shrink_kernel<RT, 1, false><<<shrink, block, 0, stream>>>(p);
        lora_expand_kernel<RT, 1, false, BF16>
            <<<dim3((unsigned)p.slots, cols), block, 0, stream>>>(p);
    }
}

template <bool PLAN, bool BF16>
void launch_lora_rank(const LoraArgs &p, int rp, hipStream_t stream) {
    if (rp == 16) launch_lora_form<1, PLAN, BF16>(p, stream);
    else if (rp == 32) launch_lora_form<2, PLAN, BF16>(p, stream);
    else if (rp == 64) launch_lora_form<4, PLAN, BF16>(p, stream);
    else launch_lora_form<8, PLAN, BF16>(p, stream);
}

}  // namespace

size_t lora_workspace_bytes(int64_t tokens, int64_t adapters, int64_t rank, int64_t k) {
    return lora_space(tokens, adapters, rank, k).end;
}

hipError_t launch_lora_add(const uint16_t *x, int64_t ldx, const uint16_t *a, const uint16_t *b,
                           const int32_t *ids, const float *scale, int64_t tokens,
                           int32_t adapters, int32_t rank, int64_t k, int64_t n, const void *y,
                           int64_t ldy, void *out, int64_t ldo, bool bf16, void *workspace,
                           hipStream_t stream) {
    const LoraSpace s = lora_space(tokens, adapters, rank, k);
    uint8_t *ws = (uint8_t *)workspace;
    if (s.plan) {
        const hipError_t err =
            launch_plan(ids, tokens, adapters + 1, true, 1, s.bm, (int32_t *)(ws + s.order),
                        nullptr, (int32_t *)(ws + s.tiles), stream);
        if (err != hipSuccess) return err;
    }
    LoraArgs p;
    p.x = x;
    p.a = a;
    p.b = b;
    p.ids = ids;
    p.scale = scale;
    p.y = y;
    p.out = out;
    p.part = (float *)(ws + s.part);
    p.terms = (uint16_t *)(ws + s.terms);
    p.tiles = (const int4 *)(ws + s.tiles);
    p.order = (const int32_t *)(ws + s.order);
    p.ldx = ldx;
    p.ldy = ldy;
    p.ldo = ldo;
    p.k = k;
    p.n = n;
    p.tokens = (int)tokens;
    p.adapters = adapters;
    p.rank = rank;
    p.slots = (int)s.slots;
    p.slices = s.slices;
    p.kslice = s.kslice;
    // column steps of an expand workgroup: about 1024 workgroups
    const int64_t tiles = s.plan ? 2 * s.slots : s.slots;
    const int64_t steps = s.plan ? 1 : tiles * ((n + kExpandN - 1) / kExpandN) / 1024;
    p.steps = (int)(steps < 1 ? 1 : steps > 8 ? 8 : steps);
    // one launch reads x for other columns while it writes out; with two, x is read
    // before out is written
    const int64_t es = bf16 ? 2 : 4;
    const bool small = one_launch(tokens, adapters, s.rp, k, n) &&
                       !rows_overlap(x, ldx * 2, k * 2, out, ldo * es, n * es, tokens);
    if (small && bf16) launch_lora_small<true>(p, s.rp, stream);
    else if (small) launch_lora_small<false>(p, s.rp, stream);
    else if (s.plan && bf16) launch_lora_rank<true, true>(p, s.rp, stream);
    else if (s.plan) launch_lora_rank<true, false>(p, s.rp, stream);
    else if (bf16) launch_lora_rank<false, true>(p, s.rp, stream);
    else launch_lora_rank<false, false>(p, s.rp, stream);
    return hipGetLastError();
}

}  // namespace w4a8

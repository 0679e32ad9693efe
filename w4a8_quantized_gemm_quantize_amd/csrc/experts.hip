// experts.hip -- the experts' products of rows routed by moe_route, on stacks of
// packed 4-bit weights (w4a8_moe_ffn in w4a8.h):
//   plan     (plan.hip) sorts the (token, slot) rows by expert and cuts each
//            expert's rows into tiles of the products' row block;
//   product  per-token quantization of x, gate and up products with
//            bf16(silu(gate) * up) in the epilogue (kSelGateUp), per-row
//            quantization of that, the down product stored to the rows' own
//            places (kSelScatter);
//   combine  the weighted sum over a token's slots.
// The products are the kernels of gemm_kernels.hpp with a tile table.
#include "gemm_kernels.hpp"

namespace w4a8 {
namespace {

// ---------------------------------------------------------------- combine --
// out[t][c] = sum over the token's slots j, in order, of weights[t][j] *
// y[t top_k + j][c], in binary32; slots without an expert were never written and
// are skipped.  A stream over y, bound by its bytes: 8 columns a thread, four
// slots' loads in flight.  y is binary32 for bf16 outputs too: rounded to bf16 it
// would be half the bytes, but the error of a sum of two to four slots grew from
// 1.7e-3 to 2.4e-3 of its norm, and a token's bits then depended on the batch.
template <bool BF16>
__global__ __launch_bounds__(256) void combine_kernel(const float *__restrict__ y,
                                                      const int32_t *__restrict__ ids,
                                                      const float *__restrict__ weights,
                                                      int64_t tokens, int experts, int top_k,
                                                      int64_t hidden, void *__restrict__ out) {
    const int64_t vecs = hidden / 8;
    const int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t t = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
    if (v >= vecs || t >= tokens) return;
    ids += t * top_k;
    weights += t * top_k;
    const int64_t row0 = t * top_k;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
    for (int j0 = 0; j0 < top_k; j0 += 4) {
        f32x4 a[4], b[4];
        float w[4];
        bool ok[4];
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
            const int j = j0 + jj < top_k ? j0 + jj : top_k - 1;
            const int id = ids[j];
            ok[jj] = j0 + jj < top_k && id >= 0 && id < experts;
            w[jj] = weights[j];
            const f32x4 *p = (const f32x4 *)y + (row0 + j) * 2 * vecs;
            a[jj] = p[2 * v];
            b[jj] = p[2 * v + 1];
        }
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[i] = ok[jj] ? acc[i] + w[jj] * a[jj][i] : acc[i];
                acc[4 + i] = ok[jj] ? acc[4 + i] + w[jj] * b[jj][i] : acc[4 + i];
            }
        }
    }
    if constexpr (BF16) {
        ((u32x4 *)out)[t * vecs + v] =
            u32x4{bf16x2_rne(acc[0], acc[1]), bf16x2_rne(acc[2], acc[3]),
                  bf16x2_rne(acc[4], acc[5]), bf16x2_rne(acc[6], acc[7])};
    } else {
        ((f32x4 *)out)[(t * vecs + v) * 2] = f32x4{acc[0], acc[1], acc[2], acc[3]};
        ((f32x4 *)out)[(t * vecs + v) * 2 + 1] = f32x4{acc[4], acc[5], acc[6], acc[7]};
    }
}

// --------------------------------------------------------------- products --
struct Product {
    const void *a_q;
    const float *a_s;
    const uint8_t *w, *grp;
    const float *ch;
    int64_t rows, n, k;
    void *out;
    int64_t ldo;
    int out_dtype;
    SelArgs sel;
};

// Workgroups of a tiled product: the most tiles there can be, in whole rows of the 8
// XCDs.
int64_t tiled_grid(int64_t slots, int64_t n, int bn) {
    return (slots * ((n + bn - 1) / bn) + 7) / 8 * 8;
}

template <int BM, int BN, int WM, int WN, int SEL>
void launch_sel_tiled(const Product &p, hipStream_t stream) {
    const int64_t grid = tiled_grid(p.sel.slots, p.n, BN);
    gemm_tiled_kernel<kW4Sym, BM, BN, WM, WN, 0, SEL>
        <<<dim3((unsigned)grid, 1), 64 * WM * WN, 0, stream>>>(
            (const int8_t *)p.a_q, p.a_s, p.w, p.grp, p.ch, 0, p.n, p.k, p.out, p.ldo,
            p.out_dtype, p.k, (int64_t)device_cu_count(), p.sel);
}

// Few rows an expert: two 16-channel tiles per workgroup of four wavefronts that
// split K, load batches of two chunks.  Measured on one box (16 tokens of 4 over
// 32 experts of 4096 x 2048; gate-up, down): 8 wavefronts with 4 chunks 57.7, 55.0
// us (registers leave one workgroup per CU); 8 with 2 41.2, 24.4; 4 with 2 35.5,
// 18.8; 2 with 2 36.8, 19.5; one tile per workgroup for the down product 21.2 at
// best.
template <int SEL, bool FUSED, int AV>
void launch_sel_skinny(const Product &p, int bm, hipStream_t stream) {
    constexpr int NT = 2, WAVES = 4, D = 2;
    const unsigned rows = SEL == kSelDirect ? (unsigned)p.rows : (unsigned)p.sel.slots;
    const dim3 grid((unsigned)((p.n / kNTile + NT - 1) / NT), rows);
    const size_t lds = FUSED ? (size_t)bm * (p.k + 16) : 0;
    gemm_skinny_kernel<kW4Sym, 1, NT, WAVES, D, FUSED, AV, 0, false, SEL>
        <<<grid, 64 * WAVES, lds, stream>>>(p.a_q, p.a_s, p.w, p.grp, p.ch, 0, p.n, p.k, p.out,
                                            p.out_dtype, nullptr, nullptr,
                                            (int64_t)device_cu_count(), p.sel);
}

// FUSED: the row vectors a lane holds, for rows of up to kFusedRowMax (kSelDirect) or
// kFusedDownMax (kSelScatter).
constexpr int64_t kFusedRowMax = 8192, kFusedDownMax = 2160;
template <int SEL>
void launch_sel_fused(const Product &p, int bm, hipStream_t stream) {
    if (p.k <= 1024) launch_sel_skinny<SEL, true, 2>(p, bm, stream);
    else if (p.k <= 2048) launch_sel_skinny<SEL, true, 4>(p, bm, stream);
    else if (SEL == kSelScatter || p.k <= 4096) launch_sel_skinny<SEL, true, 8>(p, bm, stream);
    else if constexpr (SEL == kSelDirect) launch_sel_skinny<SEL, true, 16>(p, bm, stream);
}

// ----------------------------------------------------- down, token by token --
// The down product and the weighted sum of a token in one workgroup, 16 output
// columns each (kSelDirect batches: too few rows for two tokens to share an
// expert's weights often).  A wavefront takes one slot, or one of `parts` parts
// of K of a slot: it reads the slot's row of h (from L2) for the maximum, puts the
// codes of its part into LDS of its own, and multiplies; all 16 rows of its MFMA
// are that one row.  The exact int32 sums of a slot's parts meet in LDS; then 16
// threads add the slots up in order.  y is never rounded.
//   Bound by latency: ids, then weights and h side by side, then the sum.  What
// the sum needs is read before it (read after, 8 slots of dependent loads cost
// 3 us), and the codes pass through LDS, which keeps the multiplying loop
// short (rounding at the operand gave 20 KB of straight code: 9.8 us).
constexpr int kTokenWaves = 8;
constexpr int kTokenKMax = 16384;        // LDS: at most 8 parts of K, 128 KB

__global__ __launch_bounds__(64 * kTokenWaves) void token_down_kernel(
    const uint16_t *__restrict__ h, const int32_t *__restrict__ ids,
    const float *__restrict__ weights, const uint8_t *__restrict__ w,
    const uint8_t *__restrict__ grp, const float *__restrict__ ch, int top_k, int experts,
    int64_t n, int k, int parts, int part_bytes, void *__restrict__ out, int bf16) {
    constexpr int D = 2;
    extern __shared__ __attribute__((aligned(16))) uint8_t code_lds[];   // [waves][part_bytes]
    __shared__ int red[32][16];
    __shared__ float sc[32][16];         // channel scales, row scale and weight of a slot
    __shared__ float sa[32], sw[32];
    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int c = lane & 15, kq = lane >> 4;
    const int64_t t = blockIdx.y;
    const int64_t tile = blockIdx.x;
    ids += t * top_k;
    weights += t * top_k;
    (&red[0][0])[tid] = 0;
    (&sc[0][0])[tid] = 0.0f;
    if (tid < 32) sa[tid] = sw[tid] = 0.0f;      // unused slots add nothing
    __syncthreads();

    const int nfull = k >> 7, G = k >> 6, vecs = k >> 3;
    const bool has_half = (k & 64) != 0;
    const int part = wave % parts;
    const int per = (nfull + parts - 1) / parts;
    const int j0 = part * per < nfull ? part * per : nfull;
    const int j1 = j0 + per < nfull ? j0 + per : nfull;
    const bool half_here = has_half && part == parts - 1;
    // this part's vectors of the row (the last part's with the trailing half chunk)
    const int v0 = j0 * 16, v1 = half_here ? vecs : j1 * 16;
    uint8_t *codes = code_lds + wave * part_bytes;
    const WParamSel psel = wparam_selectors<kW4Sym>(c);
    for (int slot = wave / parts; slot < top_k; slot += kTokenWaves / parts) {
        const int e = ids[slot];
        if (e < 0 || e >= experts) continue;
        const int64_t wrow = (int64_t)e * n + tile * kNTile;
        const __amdgpu_buffer_rsrc_t rw = buffer_rsrc(w + wrow * k / 2, (uint32_t)(8 * k));
        const __amdgpu_buffer_rsrc_t rp = buffer_rsrc(grp + wrow * G, (uint32_t)(16 * G));
        const __amdgpu_buffer_rsrc_t rh =
            buffer_rsrc(h + (t * top_k + slot) * (int64_t)k, (uint32_t)(2 * k));
        struct Batch {
            u32x4 w[D];
            uint32_t p[D][2];
        };
        // chunks past the part are clamped to a valid one and not used
        auto load = [&](Batch &b, int jb) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                const int j = jb + d < j1 ? jb + d : nfull - 1;
                b.w[d] = buffer_load16_nt(rw, lane * 16, j * kChunkBytes);
                b.p[d][0] = buffer_load4(rp, c & ~3, 2 * j * kNTile);
                b.p[d][1] = buffer_load4(rp, c & ~3, (2 * j + 1) * kNTile);
            }
        };
        u32x4 v[4];
        auto load_row = [&](int i0) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = i0 + u * 64 + lane;
                v[u] = buffer_load16(rh, (i < vecs ? i : vecs - 1) * 16, 0);
            }
        };
        // the first vectors of h ahead of the weights: loads complete in order
        load_row(0);
        Batch b0, b1;
        load(b0, j0);
        load(b1, j0 + D);
        __builtin_amdgcn_sched_barrier(0);
        float chv = 0.0f, wv = 0.0f;
        if (part == 0) {
            chv = ch[wrow + c];
            wv = weights[slot];
        }
        float amax = 0.0f;
#pragma unroll 1
        for (int i0 = 0; i0 < vecs; i0 += 256) {
            if (i0) load_row(i0);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float f[8];
                bf16x8_to_f32(v[u], f);
                amax = __builtin_fmaxf(amax, absmax_f32x8(f));
            }
        }
        amax = __uint_as_float(wave_max_u32(__float_as_uint(amax)));
        float s, inv;
        act_scale_pair_rcp(amax, s, inv);
#pragma unroll 1
        for (int i = v0 + lane; i < v1; i += 64) {
            float f[8];
            bf16x8_to_f32(buffer_load16(rh, i * 16, 0), f);
            *(u32x2 *)(codes + (i - v0) * 8) = codes8(f, inv);
        }
        // written and read by this wavefront alone: its LDS operations are in order
        __builtin_amdgcn_wave_barrier();
        asm volatile("" ::: "memory");
        v4i acc = {0, 0, 0, 0};
        auto compute = [&](const Batch &b, int jb) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                if (jb + d >= j1) break;
#pragma unroll
                for (int st = 0; st < 2; ++st) {
                    uint32_t mul, add;
                    wparam_consts<kW4Sym>(b.p[d][st], psel, mul, add);
                    const WRec<kW4Sym> rec = {b.w[d]};
                    const v4i a =
                        *(const v4i *)(codes + (jb + d - j0) * 128 + st * 64 + kq * 16);
                    acc = mfma16x16x64(wrec_operand_ma<kW4Sym>(rec, st, mul, add), a, acc);
                }
            }
        };
#pragma unroll 1
        for (int jb = j0; jb < j1; jb += 2 * D) {
            compute(b0, jb);
            load(b0, jb + 2 * D);
            compute(b1, jb + D);
            load(b1, jb + 3 * D);
        }
        if (half_here) {
            // trailing 64-wide chunk: 8-byte records, one K step
            const u32x2 r = *(const u32x2 *)(w + wrow * k / 2 + (int64_t)nfull * kChunkBytes +
                                             lane * 8);
            uint32_t mul, add;
            wparam_consts<kW4Sym>(buffer_load4(rp, c & ~3, 2 * nfull * kNTile), psel, mul, add);
            const v4i a = *(const v4i *)(codes + (nfull - j0) * 128 + kq * 16);
            acc = mfma16x16x64(unpack_step(r.x, r.y, mul, add), a, acc);
        }
        if (c == 0)
#pragma unroll
            for (int i = 0; i < 4; ++i) atomicAdd(&red[slot][4 * kq + i], acc[i]);
        if (part == 0 && lane < 16) {
            sc[slot][lane] = chv;
            if (lane == 0) {
                sa[slot] = s;
                sw[slot] = wv;
            }
        }
    }
    __syncthreads();
    if (tid < 16) {
        const int64_t col = tile * kNTile + tid;
        float sum = 0.0f;
        for (int slot = 0; slot < top_k; ++slot) {
            const float y = (float)red[slot][tid] * sa[slot] * sc[slot][tid];
            sum = sum + sw[slot] * y;
        }
        if (bf16) ((uint16_t *)out)[t * n + col] = (uint16_t)bf16x2_rne(sum, sum);
        else ((float *)out)[t * n + col] = sum;
    }
}

// The tiled products: 64 x 128 tiles of four wavefronts or 256 x 256 tiles.
template <int SEL>
void launch_sel(const Product &p, int bm, hipStream_t stream) {
    if (bm <= 64) launch_sel_tiled<64, 128, 1, 4, SEL>(p, stream);
    else launch_sel_tiled<256, 256, 4, 4, SEL>(p, stream);
}

// Rows an expert has on average, of those that can have any.
int64_t rows_an_expert(int64_t rows, int64_t experts) {
    return rows / (rows < experts ? rows : experts);
}

// Row block of the products for `rows` rows over `experts` experts, by the rows
// an expert has on average.  Up to 16: the skinny kernel, whose operand tile has 16
// rows.  Above, measured on one box, us a call, for blocks of 64 | 256:
//   4096 x 1408, 32 experts: 65 rows an expert 123 | 172, 160 rows 218 | 221, 200 rows
//   253 | 232, 225 rows 279 | 238, 256 rows 307 | 300, 512 rows 565 | 459;
//   2048 x 1024, 64 experts: 131 rows 159 | 195, 187 rows 202 | 207, 212 rows 225 | 216,
//   253 rows 258 | 229;
//   4096 x 14336, 8 experts: 200 rows 554 | 493, 1024 rows 2322 | 1586.
// (128 x 256 tiles were never ahead of both.)
int row_block(int64_t rows, int64_t experts) {
    const int64_t avg = rows_an_expert(rows, experts);
    return avg <= 16 ? 16 : avg < 190 ? 64 : 256;
}

// Whether the skinny down product takes the codes of its rows itself: a launch less, but
// each of a tile's hidden / 32 workgroups repeats them and holds 16 rows of K in LDS (34
// KB at kFusedDownMax, four workgroups per CU).  Measured on one box, us a call, codes taken
// here | from memory, by rows an expert and K: 2 x 768 36.8 | 39.8; 15 x 1024 24.0 | 27.1;
// 10 x 1600 35.5 | 36.4; 2 x 2048 63.7 | 63.4; 4 x 2048 77.8 | 75.8; 6 x 2048 32.1 | 33.7; 10
// x 2112 41.2 | 38.4; 16 x 2048 69.4 | 66.3; with more LDS 2 x 4096 66.8 | 67.2; 15 x 4096
// 46.4 | 43.1; 2 x 8192 82.8 | 75.9; 4 x 8192 93.2 | 81.3.
bool fused_down_pays(int64_t rows, int64_t experts, int64_t inter) {
    return inter <= kFusedDownMax && rows_an_expert(rows, experts) * inter <= 16384;
}

// Whether a batch is taken row by row (kSelDirect, two launches) rather than
// sorted (four): where the weights that two tokens then read separately cost
// less than two launches and their gaps.  Measured on one box, us, row by row |
// sorted, by those bytes: 13 MB (4 tokens, 8 of 64 experts 2048 x 768) 21.3 | 26.8;
// 26 MB (2 tokens, 4 of 16, 4096 x 4096) 41.8 | 44.6; 29 MB (8 tokens, 2 of 8, 2048 x
// 1024) 18.6 | 24.8; 30 MB (8 tokens, 8 of 128, 2048 x 768) 35.1 | 34.5; 36 MB (4
// tokens, 4 of 32, 4096 x 2048) 42.3 | 36.5; 46 MB (2 tokens, 2 of 8, 4096 x 14336) 67.4
// | 58.9; 143 MB (8 tokens, 4 of 32, 4096 x 2048) 77.3 | 50.7.
bool direct_pays(int64_t tokens, int64_t experts, int64_t top_k, int64_t hidden, int64_t inter) {
    if (tokens * top_k > 64 || hidden > kFusedRowMax || hidden < kChunkK || inter < kChunkK ||
        inter > kTokenKMax)
        return false;
    double miss = 1.0;          // an expert that no token chose, choices even
    const double hit = top_k < experts ? (double)top_k / experts : 1.0;
    for (int64_t t = 0; t < tokens; ++t) miss *= 1.0 - hit;
    const double again = (double)(tokens * top_k) - experts * (1.0 - miss);
    return again * 1.55 * hidden * inter < 30e6;       // bytes of an expert's weights
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

enum MoeForm { kMoeDirect, kMoeFew, kMoeTiled };

struct MoeSpace {
    size_t xq, xs, order, src, tiles, h, hq, hs, y, end;
    MoeForm form;
    int bm;
    bool fused_down;          // kMoeFew: the down product takes its rows' codes itself
    int64_t slots;
};

MoeSpace moe_space(int64_t tokens, int64_t experts, int64_t top_k, int64_t hidden,
                   int64_t inter) {
    const size_t t = (size_t)tokens, r = (size_t)(tokens * top_k);
    MoeSpace s;
    s.bm = row_block((int64_t)r, experts);
    // the skinny kernel needs one whole 128-wide chunk of K
    s.form = direct_pays(tokens, experts, top_k, hidden, inter)    ? kMoeDirect
             : s.bm <= 16 && hidden >= kChunkK && inter >= kChunkK ? kMoeFew
                                                                   : kMoeTiled;
    s.fused_down = s.form == kMoeFew && fused_down_pays((int64_t)r, experts, inter);
    s.slots = plan_slots((int64_t)r, experts, s.bm);
    size_t at = 0;
    auto take = [&](bool used, size_t bytes) {
        const size_t here = at;
        at += used ? up256(bytes) : 0;
        return here;
    };
    const bool sorted = s.form != kMoeDirect;
    s.xq = take(sorted, t * hidden);
    s.xs = take(sorted, t * 4);
    s.order = take(sorted, r * 4);
    s.src = take(sorted, r * 4);
    s.tiles = take(sorted, (size_t)(s.slots + 1) * 16);
    s.h = take(true, r * inter * 2);
    s.hq = take(sorted && !s.fused_down, r * inter);
    s.hs = take(sorted && !s.fused_down, r * 4);
    s.y = take(sorted, r * hidden * 4);
    s.end = at;
    return s;
}

}  // namespace

bool moe_fits(int64_t tokens, int64_t experts, int64_t top_k, int64_t hidden, int64_t inter) {
    const MoeSpace s = moe_space(tokens, experts, top_k, hidden, inter);
    if (s.form != kMoeTiled) return true;
    const int64_t n = 2 * inter > hidden ? 2 * inter : hidden;
    const int64_t items = s.bm <= 64 ? tiled_grid(s.slots, n, 128) * 256
                                     : tiled_grid(s.slots, n, 256) * 1024;
    return items < (int64_t)1 << 32;
}

size_t moe_workspace_bytes(int64_t tokens, int64_t experts, int64_t top_k, int64_t hidden,
                           int64_t inter) {
    return moe_space(tokens, experts, top_k, hidden, inter).end;
}

hipError_t launch_moe_ffn(const uint16_t *x, const int32_t *ids, const float *weights,
                          const uint8_t *w13, const uint8_t *g13, const float *c13,
                          const uint8_t *w2, const uint8_t *g2, const float *c2, int64_t tokens,
                          int32_t experts, int32_t top_k, int64_t hidden, int64_t inter,
                          void *out, int out_dtype, void *workspace, hipStream_t stream) {
    const MoeSpace s = moe_space(tokens, experts, top_k, hidden, inter);
    uint8_t *ws = (uint8_t *)workspace;
    const int64_t rows = tokens * top_k;
    int32_t *order = (int32_t *)(ws + s.order), *src = (int32_t *)(ws + s.src);
    Product p{};
    p.a_q = ws + s.xq;
    p.a_s = (const float *)(ws + s.xs);
    p.w = w13;
    p.grp = g13;
    p.ch = c13;
    p.rows = rows;
    p.n = 2 * inter;
    p.k = hidden;
    p.out = ws + s.h;
    p.ldo = inter;
    p.out_dtype = 1;
    if (s.form == kMoeDirect) {
        p.a_q = x;
        p.sel = SelArgs{nullptr, ids, 0u, top_k, experts, inter};
        launch_sel_fused<kSelDirect>(p, 1, stream);
        int parts = 1;                    // wavefronts of a slot, a power of two
        while (parts * 2 * top_k <= kTokenWaves) parts *= 2;
        const int part_bytes =
            (int)(((inter / 128 + parts - 1) / parts) * 128 + 64);   // and a half chunk
        token_down_kernel<<<dim3((unsigned)(hidden / kNTile), (unsigned)tokens),
                            64 * kTokenWaves, (size_t)(kTokenWaves * part_bytes), stream>>>(
            (const uint16_t *)(ws + s.h), ids, weights, w2, g2, c2, top_k, experts, hidden,
            (int)inter, parts, part_bytes, out, out_dtype == 1);
        return hipGetLastError();
    }
    hipError_t err = launch_plan_quantize(ids, rows, experts, top_k, s.bm, order, src,
                                          (int32_t *)(ws + s.tiles), x, tokens, hidden,
                                          (int8_t *)(ws + s.xq), (float *)(ws + s.xs), stream);
    if (err != hipSuccess) return err;
    p.sel = SelArgs{(const int4 *)(ws + s.tiles), src, (uint32_t)(tokens * hidden),
                    (int32_t)s.slots, experts, inter};
    if (s.form == kMoeFew) launch_sel_skinny<kSelGateUp, false, 1>(p, s.bm, stream);
    else launch_sel<kSelGateUp>(p, s.bm, stream);
    p.a_q = ws + s.h;
    if (!s.fused_down) {
        err = launch_quantize_rows((const uint16_t *)(ws + s.h), rows, inter,
                                   (int8_t *)(ws + s.hq), (float *)(ws + s.hs), stream);
        if (err != hipSuccess) return err;
        p.a_q = ws + s.hq;
        p.a_s = (const float *)(ws + s.hs);
    }
    p.w = w2;
    p.grp = g2;
    p.ch = c2;
    p.n = hidden;
    p.k = inter;
    p.out = ws + s.y;
    p.ldo = hidden;
    p.out_dtype = 0;
    p.sel.map = order;
    if (s.fused_down) launch_sel_fused<kSelScatter>(p, s.bm, stream);
    else if (s.form == kMoeFew) launch_sel_skinny<kSelScatter, false, 1>(p, s.bm, stream);
    else launch_sel<kSelScatter>(p, s.bm, stream);
    const int64_t gy = tokens < 32768 ? tokens : 32768;
    const dim3 grid((unsigned)((hidden / 8 + 255) / 256), (unsigned)gy,
                    (unsigned)((tokens + gy - 1) / gy));
    const auto combine = out_dtype == 1 ? combine_kernel<true> : combine_kernel<false>;
    combine<<<grid, 256, 0, stream>>>((const float *)(ws + s.y), ids, weights, tokens, experts,
                                      top_k, hidden, out);
    return hipGetLastError();
}

}  // namespace w4a8

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
// are skipped.  A stream over y: 8 columns a thread, four slots' loads in
// flight.  y has the output's type: for bf16 outputs each product is rounded to
// bf16 once before the sum (halving the largest intermediate; two roundings of
// 2^-8 instead of one).
template <bool BF16>
__global__ __launch_bounds__(256) void combine_kernel(const void *__restrict__ y,
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
        u32x4 a[4], b[4];
        float w[4];
        bool ok[4];
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
            const int j = j0 + jj < top_k ? j0 + jj : top_k - 1;
            const int id = ids[j];
            ok[jj] = j0 + jj < top_k && id >= 0 && id < experts;
            w[jj] = weights[j];
            const u32x4 *p = (const u32x4 *)y + (row0 + j) * (BF16 ? vecs : 2 * vecs);
            if constexpr (BF16) {
                a[jj] = p[v];
            } else {
                a[jj] = p[2 * v];
                b[jj] = p[2 * v + 1];
            }
        }
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
            float f[8];
            if constexpr (BF16) {
                bf16x8_to_f32(a[jj], f);
            } else {
                const f32x4 lo = __builtin_bit_cast(f32x4, a[jj]);
                const f32x4 hi = __builtin_bit_cast(f32x4, b[jj]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f[i] = lo[i];
                    f[4 + i] = hi[i];
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = ok[jj] ? acc[i] + w[jj] * f[i] : acc[i];
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
    const int8_t *a_q;
    const float *a_s;
    const uint8_t *w, *grp;
    const float *ch;
    int64_t rows, n, k;
    void *out;
    int64_t ldo;
    int out_dtype;
    SelArgs sel;
};

template <int BM, int BN, int WM, int WN, int SEL>
void launch_sel_tiled(const Product &p, hipStream_t stream) {
    const int64_t grid = (int64_t)p.sel.slots * ((p.n + BN - 1) / BN);
    gemm_tiled_kernel<kW4Sym, BM, BN, WM, WN, 0, SEL>
        <<<dim3((unsigned)grid, 1), 64 * WM * WN, 0, stream>>>(
            p.a_q, p.a_s, p.w, p.grp, p.ch, 0, p.n, p.k, p.out, p.ldo, p.out_dtype, p.k,
            (int64_t)device_cu_count(), p.sel);
}

template <int SEL>
void launch_sel_skinny(const Product &p, hipStream_t stream) {
    constexpr int NT = SEL == kSelGateUp ? 2 : 1;
    const dim3 grid((unsigned)(p.n / (kNTile * NT)), (unsigned)p.sel.slots);
    gemm_skinny_kernel<kW4Sym, 1, NT, 8, 4, false, 1, 0, false, SEL>
        <<<grid, 512, 0, stream>>>(p.a_q, p.a_s, p.w, p.grp, p.ch, 0, p.n, p.k, p.out,
                                   p.out_dtype, nullptr, nullptr, (int64_t)device_cu_count(),
                                   p.sel);
}

template <int SEL>
void launch_sel(const Product &p, int bm, hipStream_t stream) {
    // the skinny kernel needs one whole 128-wide chunk of K
    if (bm == 16 && p.k >= kChunkK) launch_sel_skinny<SEL>(p, stream);
    else if (bm <= 64) launch_sel_tiled<64, 256, 1, 8, SEL>(p, stream);
    else if (bm == 128) launch_sel_tiled<128, 256, 1, 8, SEL>(p, stream);
    else launch_sel_tiled<256, 256, 4, 4, SEL>(p, stream);
}

// Row block of the products for `rows` rows over `experts` experts.
int row_block(int64_t rows, int64_t experts) {
    const int64_t met = rows < experts ? rows : experts;
    const int64_t avg = rows / met;
    return avg <= 16 ? 16 : avg <= 64 ? 64 : avg <= 512 ? 128 : 256;
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct MoeSpace {
    size_t xq, xs, order, src, tiles, h, hq, hs, y, end;
    int bm;
    int64_t slots;
};

MoeSpace moe_space(int64_t tokens, int64_t experts, int64_t top_k, int64_t hidden, int64_t inter,
                   int out_dtype) {
    const size_t t = (size_t)tokens, r = (size_t)(tokens * top_k);
    MoeSpace s;
    s.bm = row_block((int64_t)r, experts);
    s.slots = plan_slots((int64_t)r, experts, s.bm);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += up256(bytes);
        return here;
    };
    s.xq = take(t * hidden);
    s.xs = take(t * 4);
    s.order = take(r * 4);
    s.src = take(r * 4);
    s.tiles = take((size_t)s.slots * 16);
    s.h = take(r * inter * 2);
    s.hq = take(r * inter);
    s.hs = take(r * 4);
    s.y = take(r * hidden * (out_dtype == 1 ? 2 : 4));
    s.end = at;
    return s;
}

}  // namespace

size_t moe_workspace_bytes(int64_t tokens, int64_t experts, int64_t top_k, int64_t hidden,
                           int64_t inter, int out_dtype) {
    return moe_space(tokens, experts, top_k, hidden, inter, out_dtype).end;
}

hipError_t launch_moe_ffn(const uint16_t *x, const int32_t *ids, const float *weights,
                          const uint8_t *w13, const uint8_t *g13, const float *c13,
                          const uint8_t *w2, const uint8_t *g2, const float *c2, int64_t tokens,
                          int32_t experts, int32_t top_k, int64_t hidden, int64_t inter,
                          void *out, int out_dtype, void *workspace, hipStream_t stream) {
    const MoeSpace s = moe_space(tokens, experts, top_k, hidden, inter, out_dtype);
    uint8_t *ws = (uint8_t *)workspace;
    const int64_t rows = tokens * top_k;
    int32_t *order = (int32_t *)(ws + s.order), *src = (int32_t *)(ws + s.src);
    const int4 *tiles = (const int4 *)(ws + s.tiles);
    hipError_t err = launch_plan(ids, rows, experts, false, top_k, s.bm, order, src,
                                 (int32_t *)(ws + s.tiles), stream);
    if (err != hipSuccess) return err;
    err = launch_quantize_rows(x, tokens, hidden, (int8_t *)(ws + s.xq), (float *)(ws + s.xs),
                               stream);
    if (err != hipSuccess) return err;
    Product p{};
    p.a_q = (const int8_t *)(ws + s.xq);
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
    p.sel = SelArgs{tiles, src, (uint32_t)(tokens * hidden), (int32_t)s.slots, inter};
    launch_sel<kSelGateUp>(p, s.bm, stream);
    err = launch_quantize_rows((const uint16_t *)(ws + s.h), rows, inter, (int8_t *)(ws + s.hq),
                               (float *)(ws + s.hs), stream);
    if (err != hipSuccess) return err;
    p.a_q = (const int8_t *)(ws + s.hq);
    p.a_s = (const float *)(ws + s.hs);
    p.w = w2;
    p.grp = g2;
    p.ch = c2;
    p.n = hidden;
    p.k = inter;
    p.out = ws + s.y;
    p.ldo = hidden;
    p.out_dtype = out_dtype;
    p.sel = SelArgs{tiles, order, 0u, (int32_t)s.slots, 0};
    launch_sel<kSelScatter>(p, s.bm, stream);
    const int64_t gy = tokens < 32768 ? tokens : 32768;
    const dim3 grid((unsigned)((hidden / 8 + 255) / 256), (unsigned)gy,
                    (unsigned)((tokens + gy - 1) / gy));
    if (out_dtype == 1)
        combine_kernel<true><<<grid, 256, 0, stream>>>(ws + s.y, ids, weights, tokens, experts,
                                                       top_k, hidden, out);
    else
        combine_kernel<false><<<grid, 256, 0, stream>>>(ws + s.y, ids, weights, tokens, experts,
                                                        top_k, hidden, out);
    return hipGetLastError();
}

}  // namespace w4a8

// attn.hip -- attention of query rows over the paged 8-bit cache (w4a8_attn_kv8 in w4a8.h).
//
// The G = q_heads / kv_heads query heads of a cache head share its keys and values, so the
// rows of a tile are (row i of the sequence, head g of the group), i G + g, 16 at a time:
// the columns of the matrix products
//   S [token][row] = K Q^T   and   O^T [element][row] += V^T P
// with v_mfma_f32_16x16x32_f16.  K and V are bytes u = code + 128; the half 0x6400 | u is
// 1024 + u, so one byte permutation and one packed subtraction of 1152 make two exact
// codes.  Q enters as halves too, each row scaled by a power of two that puts its largest
// element just below 2^15: exact, but for elements under 2^-29 of that.  The products'
// results arrive in the lanes that the next product's operand needs (kv_index.hpp).
//
// Softmax in base 2 in one pass: with s_j = (scale log2 e) k_scale (q . k_j) of a token in a
// page of value scale sv,
//   t_j = s_j + log2 sv,   m >= max t_j - 8,   p_j = 2^(t_j - m)
//   O = sum p_j codes_j,   l = sum p_j / sv,   out = O / l,   lse = ln 2 (m + log2 l)
// so P needs no factor per page, is at most 2^8, and what its rounding to a half loses
// (2^-11 of each p_j; below 2^-14 absolutely 2^-25) is measured against the largest product
// p_j sv, not against p_j alone.  t, m, l and O are binary32.  m moves only when some t_j
// exceeds it by more than 8, so most tiles rescale nothing.  Where a page's values are all 0
// (sv = 0) any sv does: scales below 2^-100 count as that.
#include "device_common.hpp"
#include "kv_index.hpp"
#include "launch.hpp"

namespace w4a8 {
namespace {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));

struct AttnArgs {
    KvBatch b;
    const uint16_t *q;
    const uint8_t *kv;
    const float *kv_scale;
    uint16_t *out;
    float *lse, *part;             // part: partial results of splits (null: none)
    int64_t ldq, ldo;
    int heads, group, max_rows, causal, window;
    int splits, tiles;             // tiles: of a sequence, or 0 (items found by kv_find_seq)
    int64_t items;
    float scale;                   // times log2 e
};

constexpr float kLn2 = 0.693147180559945f;

// Four bytes u -> halves u - 128 (see above).
__device__ __forceinline__ void codes4(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const half2_t off = {(_Float16)-1152.0f, (_Float16)-1152.0f};
    const half2_t a = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, w, 0x04010400u));
    const half2_t b = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, w, 0x04030402u));
    lo = __builtin_bit_cast(uint32_t, a + off);
    hi = __builtin_bit_cast(uint32_t, b + off);
}
__device__ __forceinline__ half8_t codes8h(uint32_t a, uint32_t b) {
    u32x4 r;
    uint32_t lo, hi;
    codes4(a, lo, hi);
    r.x = lo;
    r.y = hi;
    codes4(b, lo, hi);
    r.z = lo;
    r.w = hi;
    return __builtin_bit_cast(half8_t, r);
}
__device__ __forceinline__ f32x4 mfma16(half8_t a, half8_t b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
// Maximum, sum over the four lanes l % 16 + 16 g.
__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float quad_sum(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

__device__ __forceinline__ bool find_tile(const AttnArgs &a, int64_t item, int shift, KvTile &t) {
    return kv_tile(a.b, item, a.tiles, a.group, shift, a.max_rows, a.causal, a.window, t);
}

// 2^e that brings a row of Q whose largest element has the bits `top` to [2^14, 2^15), with
// the sign of the scale; fac = |scale| / 2^e.
__device__ __forceinline__ float row_scale(uint32_t top, float scale, float &fac) {
    const int e = min(100, 14 + 127 - (int)(top >> 23));
    fac = fabsf(scale) * __uint_as_float((uint32_t)(127 - e) << 23);
    return copysignf(__uint_as_float((uint32_t)(127 + e) << 23), scale);
}
// Of a page: key scale, log2 of the value scale, its inverse.  Without one (sv < 0) log2 is
// -inf, so that every weight is 0.
__device__ __forceinline__ f32x4 page_terms(float sk, float sv) {
    if (!(sv >= 0.0f)) return f32x4{0.0f, -__builtin_inff(), 0.0f, 0.0f};
    sv = fmaxf(sv, 0x1p-100f);
    return f32x4{sk, __builtin_amdgcn_logf(sv), __builtin_amdgcn_rcpf(sv), 0.0f};
}

constexpr int kWaves = 4;

// A wavefront holds all 16 rows and takes every fourth run of 32 tokens of the workgroup's
// range; the four partial results are joined in LDS.  K and V go from memory straight to
// the registers they are multiplied from, the next run's while this one is worked on.
template <int C, bool HALF>                      // full chunks of 64 elements, and a half one
__global__ __launch_bounds__(kWaves * 64, 64 * C + 32 * HALF <= 64 ? 4 : C == 2 && !HALF ? 3 : 2)
void attn_rows_kernel(AttnArgs a) {
    constexpr int kDim = 64 * C + (HALF ? 32 : 0), kTiles = kDim / 16, kSteps = kDim / 32;
    constexpr int kStride = kDim + 4;
    __shared__ __attribute__((aligned(16))) float lds[kWaves * 16 * kStride];
    __shared__ float lds_m[kWaves * 16], lds_l[kWaves * 16];
    const int split = blockIdx.x % a.splits;
    const int head = blockIdx.x / a.splits % a.heads;
    const int64_t item = blockIdx.x / a.splits / a.heads;
    KvTile t;
    if (!find_tile(a, item, 4, t)) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int col = lane & 15, g = lane >> 4;
    const int from = t.seq.len - t.seq.n;

    // this lane's row of Q, scaled
    const int r = t.row0 + col;
    const int i = r / a.group;
    const bool live = col < t.rows;
    half8_t q[kSteps];
    float qfac;
    {
        const uint16_t *p = a.q + (int64_t)(t.seq.first_row + i) * a.ldq +
                            (int64_t)(head * a.group + r - i * a.group) * kDim;
        u32x4 w[kSteps];
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            const int d = k < 2 * C ? (k >> 1) * 64 + 16 * g + 8 * (k & 1) : C * 64 + 8 * g;
            w[k] = live ? *(const u32x4 *)(p + d) : u32x4{0, 0, 0, 0};
            float f[8];
            bf16x8_to_f32(w[k], f);
            top = max(top, __float_as_uint(absmax_f32x8(f)));
        }
        top = max(top, (uint32_t)__shfl_xor((int)top, 16));
        top = max(top, (uint32_t)__shfl_xor((int)top, 32));
        const float up = row_scale(top, a.scale, qfac);
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            float f[8];
            bf16x8_to_f32(w[k], f);
#pragma unroll
            for (int x = 0; x < 8; ++x) q[k][x] = (_Float16)(f[x] * up);
        }
    }
    // tokens this row sees: [see_lo, see_hi)
    const int pos = from + i;
    int see_hi = a.causal ? min(t.hi, pos + 1) : t.hi;
    const int see_lo = a.window ? max(0, pos - a.window + 1) : 0;
    if (!live) see_hi = 0;

    const int u_first = t.lo >> 5, u_all = ((t.hi + 31) >> 5) - u_first;
    const int u0 = u_first + (int)((int64_t)u_all * split / a.splits);
    const int u1 = u_first + (int)((int64_t)u_all * (split + 1) / a.splits);

    f32x4 o[kTiles];
#pragma unroll
    for (int d = 0; d < kTiles; ++d) o[d] = f32x4{0, 0, 0, 0};
    float m = -1e30f, l = 0.0f;

    struct Run {
        u32x4 k[2][C ? C : 1], v[2][C ? C : 1];
        u32x2 kh[2], vh[2];
        float sk[2], sv[2];
    };
    const int page_mask = (1 << a.b.page_shift) - 1;
    auto load = [&](int u, Run &x) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int at = u * 32 + h * 16;
            const int page = at < t.hi ? kv_page(a.b, t.s, at >> a.b.page_shift) : -1;
            if (page >= 0) {
                const int64_t ph = (int64_t)page * a.heads + head;
                const uint8_t *kp = a.kv + (ph * 2 << a.b.page_shift) * kDim + (at & page_mask) * kDim;
                const uint8_t *vp = kp + ((int64_t)kDim << a.b.page_shift);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    x.k[h][c] = *(const u32x4 *)(kp + c * 1024 + lane * 16);
                    x.v[h][c] = *(const u32x4 *)(vp + c * 1024 + lane * 16);
                }
                if constexpr (HALF) {
                    x.kh[h] = *(const u32x2 *)(kp + C * 1024 + lane * 8);
                    x.vh[h] = *(const u32x2 *)(vp + C * 1024 + lane * 8);
                }
                x.sk[h] = a.kv_scale[ph * 2];
                x.sv[h] = a.kv_scale[ph * 2 + 1];
            } else {
                const u32x4 z = {0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u};
#pragma unroll
                for (int c = 0; c < C; ++c) x.k[h][c] = x.v[h][c] = z;
                if constexpr (HALF) x.kh[h] = x.vh[h] = u32x2{z.x, z.x};
                x.sk[h] = 0.0f;
                x.sv[h] = -1.0f;                 // no page: masked
            }
        }
    };

    Run x;
    if (u0 + wave < u1) load(u0 + wave, x);
    for (int u = u0 + wave; u < u1; u += kWaves) {
        // scores of two tiles of 16 tokens
        f32x4 s[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                s[h] = mfma16(codes8h(x.k[h][c].x, x.k[h][c].y), q[2 * c], s[h]);
                s[h] = mfma16(codes8h(x.k[h][c].z, x.k[h][c].w), q[2 * c + 1], s[h]);
            }
            if constexpr (HALF) s[h] = mfma16(codes8h(x.kh[h].x, x.kh[h].y), q[2 * C], s[h]);
        }
        float tv[2][4], inv[2];
        float best = -1e30f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f32x4 pt = page_terms(x.sk[h], x.sv[h]);
            const float f = qfac * pt.x;
            inv[h] = pt.z;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = u * 32 + h * 16 + 4 * g + e;
                tv[h][e] = j >= see_lo && j < see_hi ? __builtin_fmaf(s[h][e], f, pt.y)
                                                     : -__builtin_inff();
                best = fmaxf(best, tv[h][e]);
            }
        }
        if (__any(best > m + 8.0f)) {
            const float n = fmaxf(m, quad_max(best));
            const float down = __builtin_amdgcn_exp2f(m - n);
            m = n;
            l *= down;
#pragma unroll
            for (int d = 0; d < kTiles; ++d) o[d] *= down;
        }
        half8_t p;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float w = __builtin_amdgcn_exp2f(tv[h][e] - m);
                sum += w;
                p[4 * h + e] = (_Float16)w;
            }
            l = __builtin_fmaf(sum, inv[h], l);
        }
        const Run y = x;
        if (u + kWaves < u1) load(u + kWaves, x);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                o[4 * c + j] = mfma16(codes8h(y.v[0][c][j], y.v[1][c][j]), p, o[4 * c + j]);
        if constexpr (HALF) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                o[4 * C + j] = mfma16(codes8h(y.vh[0][j], y.vh[1][j]), p, o[4 * C + j]);
        }
    }
    l = quad_sum(l);
#pragma unroll
    for (int d = 0; d < kTiles; ++d)
        *(f32x4 *)(lds + (wave * 16 + col) * kStride + d * 16 + 4 * g) = o[d];
    if (g == 0) {
        lds_m[wave * 16 + col] = m;
        lds_l[wave * 16 + col] = l;
    }
    __syncthreads();
    // 16 threads a row, 4 elements each at a time
    const int row = threadIdx.x >> 4, at = (threadIdx.x & 15) * 4;
    if (row >= t.rows) return;
    float mm = lds_m[row];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) mm = fmaxf(mm, lds_m[w * 16 + row]);
    float f[kWaves], ll = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        f[w] = __builtin_amdgcn_exp2f(lds_m[w * 16 + row] - mm);
        ll = __builtin_fmaf(f[w], lds_l[w * 16 + row], ll);
    }
    const int rr = t.row0 + row, ri = rr / a.group, qh = head * a.group + rr - ri * a.group;
    const int64_t orow = t.seq.first_row + ri;
    const float by = a.part ? 1.0f : ll > 0.0f ? 1.0f / ll : 0.0f;
    float *part = nullptr;
    if (a.part) {
        part = a.part + (((item * a.heads + head) * a.splits + split) * 16 + row) * (kDim + 4);
        if (at == 0) {
            part[kDim] = mm;
            part[kDim + 1] = ll;
        }
    } else if (at == 0 && a.lse) {
        a.lse[orow * a.heads * a.group + qh] =
            ll > 0.0f ? kLn2 * (mm + __builtin_amdgcn_logf(ll)) : -__builtin_inff();
    }
    for (int d = at; d < kDim; d += 64) {
        f32x4 sum = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const f32x4 v = *(const f32x4 *)(lds + (w * 16 + row) * kStride + d);
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] = __builtin_fmaf(f[w], v[e], sum[e]);
        }
        if (a.part) {
            *(f32x4 *)(part + d) = sum;
        } else {
            *(u32x2 *)(a.out + orow * a.ldo + (int64_t)qh * kDim + d) =
                u32x2{bf16x2_rne(sum[0] * by, sum[1] * by), bf16x2_rne(sum[2] * by, sum[3] * by)};
        }
    }
}

// ---- many rows: 128 packed rows a workgroup, 32 a wavefront ----
//
// Four wavefronts share 64 tokens at a time, converted once to halves in LDS in the order of
// the operands of v_mfma_f32_32x32x16_f16 (A: lane l holds 8 of row l % 32, k = 8 (l / 32) ..;
// result element i of lane l: row 8 (i / 4) + 4 (l / 32) + i % 4, column l % 32):
//   keys    [16 tokens][chunk][half of the record][lane] 16 bytes: step (chunk, s, half) reads
//           the records of quarters 2 s + l / 32, elements 16 (2 s + l / 32) + 8 half ..
//   values  [16 tokens][32 elements][l / 32][element] 16 bytes: tokens 4 (l / 32) .. and
//           8 + 4 (l / 32) .., which are the rows of S that the lane holds.
// Two buffers: while one is multiplied, the next tokens' bytes, loaded a round ago, become the
// other's halves and the loads after them go out; one barrier a round.
typedef float f32x16 __attribute__((ext_vector_type(16)));
__device__ __forceinline__ f32x16 mfma32(half8_t a, half8_t b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
constexpr int kTileShift = 7;                    // packed rows of a tile: 128

template <int C, bool HALF>
__global__ __launch_bounds__(256, (64 * C + 32 * HALF) <= 128 ? 2 : 1) void attn_tile_kernel(AttnArgs a) {
    constexpr int kDim = 64 * C + (HALF ? 32 : 0), kSteps = kDim / 16, kBlocks = kDim / 32;
    constexpr int kSub = 16 * kDim;              // halves of 16 tokens
    __shared__ __attribute__((aligned(16))) _Float16 kbuf[2][4 * kSub], vbuf[2][4 * kSub];
    __shared__ f32x4 page[2][4];                 // of 16 tokens: key scale, log2 value scale, 1 / it
    const int head = blockIdx.x % a.heads;
    const int split = blockIdx.x / a.heads % a.splits;
    const int64_t item = a.items - 1 - blockIdx.x / a.heads / a.splits;
    KvTile t;
    if (!find_tile(a, item, kTileShift, t)) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int col = lane & 31, h = lane >> 5;
    const int from = t.seq.len - t.seq.n;

    const int r = t.row0 + wave * 32 + col;
    const int i = r / a.group;
    const bool live = wave * 32 + col < t.rows;
    half8_t q[kSteps];
    float qfac;
    {
        const uint16_t *p = a.q + (int64_t)(t.seq.first_row + i) * a.ldq +
                            (int64_t)(head * a.group + r - i * a.group) * kDim;
        u32x4 w[kSteps];
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            const int d = k < 4 * C ? (k >> 2) * 64 + 16 * (2 * (k >> 1 & 1) + h) + 8 * (k & 1)
                                    : C * 64 + 8 * (2 * (k & 1) + h);
            w[k] = live ? *(const u32x4 *)(p + d) : u32x4{0, 0, 0, 0};
            float f[8];
            bf16x8_to_f32(w[k], f);
            top = max(top, __float_as_uint(absmax_f32x8(f)));
        }
        top = max(top, (uint32_t)__shfl_xor((int)top, 32));
        const float up = row_scale(top, a.scale, qfac);
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            float f[8];
            bf16x8_to_f32(w[k], f);
#pragma unroll
            for (int x = 0; x < 8; ++x) q[k][x] = (_Float16)(f[x] * up);
        }
    }
    const int pos = from + i;
    const int see_hi = live ? a.causal ? min(t.hi, pos + 1) : t.hi : 0;
    const int see_lo = a.window ? max(0, pos - a.window + 1) : 0;
    // tokens that every row of the wavefront sees
    const bool whole = wave * 32 + 32 <= t.rows;
    const int all_hi = whole ? a.causal ? min(t.hi, from + (t.row0 + wave * 32) / a.group + 1) : t.hi : 0;
    const int all_lo = a.window ? from + (t.row0 + wave * 32 + 31) / a.group - a.window + 1 : 0;

    const int j_first = t.lo >> 6, j_all = ((t.hi + 63) >> 6) - j_first;
    const int j0 = j_first + (int)((int64_t)j_all * split / a.splits);
    const int j1 = j_first + (int)((int64_t)j_all * (split + 1) / a.splits);

    f32x16 o[kBlocks];
#pragma unroll
    for (int d = 0; d < kBlocks; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[d][e] = 0.0f;
    float m = -1e30f, l = 0.0f;

    // this wavefront's 16 of a run of 64 tokens
    u32x4 kr[C ? C : 1], vr[C ? C : 1];
    u32x2 kh, vh;
    float sk, sv;
    const int page_mask = (1 << a.b.page_shift) - 1;
    auto load = [&](int j) {
        const int at = j * 64 + wave * 16;
        const int pg = at < t.hi ? kv_page(a.b, t.s, at >> a.b.page_shift) : -1;
        if (pg >= 0) {
            const int64_t ph = (int64_t)pg * a.heads + head;
            const uint8_t *kp = a.kv + (ph * 2 << a.b.page_shift) * kDim + (at & page_mask) * kDim;
            const uint8_t *vp = kp + ((int64_t)kDim << a.b.page_shift);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                kr[c] = *(const u32x4 *)(kp + c * 1024 + lane * 16);
                vr[c] = *(const u32x4 *)(vp + c * 1024 + lane * 16);
            }
            if constexpr (HALF) {
                kh = *(const u32x2 *)(kp + C * 1024 + lane * 8);
                vh = *(const u32x2 *)(vp + C * 1024 + lane * 8);
            }
            sk = a.kv_scale[ph * 2];
            sv = a.kv_scale[ph * 2 + 1];
        } else {
            const u32x4 z = {0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u};
#pragma unroll
            for (int c = 0; c < C; ++c) kr[c] = vr[c] = z;
            if constexpr (HALF) kh = vh = u32x2{z.x, z.x};
            sk = 0.0f;
            sv = -1.0f;
        }
    };
    auto store = [&](int buf) {
        _Float16 *kb = kbuf[buf] + wave * kSub, *vb = vbuf[buf] + wave * kSub;
        const int g = lane >> 4, e = lane & 15;
        _Float16 *vl = vb + (g & 1) * 256 + e * 8 + (g >> 1) * 4;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            *(half8_t *)(kb + (c * 2) * 512 + lane * 8) = codes8h(kr[c].x, kr[c].y);
            *(half8_t *)(kb + (c * 2 + 1) * 512 + lane * 8) = codes8h(kr[c].z, kr[c].w);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                uint32_t lo, hi;
                codes4(vr[c][x], lo, hi);
                *(u32x2 *)(vl + (c * 2 + (x >> 1)) * 512 + (x & 1) * 128) = u32x2{lo, hi};
            }
        }
        if constexpr (HALF) {
            *(half8_t *)(kb + (C * 2) * 512 + lane * 8) = codes8h(kh.x, kh.y);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                uint32_t lo, hi;
                codes4(vh[x], lo, hi);
                *(u32x2 *)(vl + C * 2 * 512 + x * 128) = u32x2{lo, hi};
            }
        }
        if (lane == 0) page[buf][wave] = page_terms(sk, sv);
    };

    if (j0 < j1) {
        load(j0);
        store(j0 & 1);
        if (j0 + 1 < j1) load(j0 + 1);
    }
    __syncthreads();
    for (int j = j0; j < j1; ++j) {
        if (j + 1 < j1) {
            store((j + 1) & 1);
            if (j + 2 < j1) load(j + 2);
        }
        const _Float16 *kb = kbuf[j & 1], *vb = vbuf[j & 1];
        f32x16 s[2];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int e = 0; e < 16; ++e) s[b][e] = 0.0f;
        const int sub_lane = (lane & 31) >> 4, rec = (h * 16 + (lane & 15)) * 8;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            const int at = k < 4 * C ? ((k >> 2) * 2 + (k & 1)) * 512 + (k >> 1 & 1) * 256
                                     : C * 1024 + (k & 1) * 256;
#pragma unroll
            for (int b = 0; b < 2; ++b)
                s[b] = mfma32(*(const half8_t *)(kb + (2 * b + sub_lane) * kSub + at + rec), q[k], s[b]);
        }
        if (j * 64 + 64 > all_hi || j * 64 < all_lo) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int at = j * 64 + b * 32 + 8 * (e >> 2) + 4 * h + (e & 3);
                    if (at < see_lo || at >= see_hi) s[b][e] = -__builtin_inff();
                }
        }
        f32x4 pt[4];
        float f[4], best = -1e30f;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            pt[x] = page[j & 1][x];
            f[x] = fmaxf(qfac * pt[x].x, 1e-30f);
            float top = s[x >> 1][8 * (x & 1)];
#pragma unroll
            for (int e = 1; e < 8; ++e) top = fmaxf(top, s[x >> 1][8 * (x & 1) + e]);
            best = fmaxf(best, __builtin_fmaf(top, f[x], pt[x].y));
        }
        if (__any(best > m + 8.0f)) {
            const float n = fmaxf(m, fmaxf(best, __shfl_xor(best, 32)));
            const float down = __builtin_amdgcn_exp2f(m - n);
            m = n;
            l *= down;
#pragma unroll
            for (int d = 0; d < kBlocks; ++d) o[d] *= down;
        }
        half8_t p[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const float off = pt[x].y - m;
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[x >> 1][8 * (x & 1) + e], f[x], off));
                sum += w;
                p[x][e] = (_Float16)w;
            }
            l = __builtin_fmaf(sum, pt[x].z, l);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int d = 0; d < kBlocks; ++d)
                o[d] = mfma32(*(const half8_t *)(vb + x * kSub + d * 512 + lane * 8), p[x], o[d]);
        __syncthreads();
    }
    l += __shfl_xor(l, 32);
    const int qh = head * a.group + r - i * a.group;
    const int64_t orow = t.seq.first_row + i;
    if (a.part) {
        if (!live) return;
        float *part = a.part + (((item * a.heads + head) * a.splits + split) * 128 + wave * 32 + col) *
                                   (kDim + 4);
        if (h == 0) {
            part[kDim] = m;
            part[kDim + 1] = l;
        }
#pragma unroll
        for (int d = 0; d < kBlocks; ++d)
#pragma unroll
            for (int x = 0; x < 4; ++x)
                *(f32x4 *)(part + d * 32 + 8 * x + 4 * h) =
                    f32x4{o[d][4 * x], o[d][4 * x + 1], o[d][4 * x + 2], o[d][4 * x + 3]};
        return;
    }
    if (live && h == 0 && a.lse)
        a.lse[orow * a.heads * a.group + qh] =
            l > 0.0f ? kLn2 * (m + __builtin_amdgcn_logf(l)) : -__builtin_inff();
    const float by = l > 0.0f ? 1.0f / l : 0.0f;
    if (!live) return;
    uint16_t *out = a.out + orow * a.ldo + (int64_t)qh * kDim;
#pragma unroll
    for (int d = 0; d < kBlocks; ++d)
#pragma unroll
        for (int x = 0; x < 4; ++x)
            *(u32x2 *)(out + d * 32 + 8 * x + 4 * h) =
                u32x2{bf16x2_rne(o[d][4 * x] * by, o[d][4 * x + 1] * by),
                      bf16x2_rne(o[d][4 * x + 2] * by, o[d][4 * x + 3] * by)};
}

// Joins the splits of a tile: 16 threads a row.
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, int dim, int shift) {
    const int slabs = 1 << (shift - 4), height = 1 << shift;
    const int head = blockIdx.x / slabs % a.heads;
    const int64_t item = blockIdx.x / slabs / a.heads;
    KvTile t;
    if (!find_tile(a, item, shift, t)) return;
    const int row = (int)(blockIdx.x % slabs) * 16 + (threadIdx.x >> 4), at = (threadIdx.x & 15) * 4;
    if (row >= t.rows) return;
    const int64_t step = (int64_t)height * (dim + 4);
    const float *p = a.part + ((item * a.heads + head) * a.splits * height + row) * (dim + 4);
    float mm = -1e30f;
    for (int z = 0; z < a.splits; ++z) mm = fmaxf(mm, p[z * step + dim]);
    float ll = 0.0f;
    for (int z = 0; z < a.splits; ++z)
        ll = __builtin_fmaf(__builtin_amdgcn_exp2f(p[z * step + dim] - mm), p[z * step + dim + 1], ll);
    const float by = ll > 0.0f ? 1.0f / ll : 0.0f;
    const int rr = t.row0 + row, ri = rr / a.group, qh = head * a.group + rr - ri * a.group;
    const int64_t orow = t.seq.first_row + ri;
    if (at == 0 && a.lse)
        a.lse[orow * a.heads * a.group + qh] =
            ll > 0.0f ? kLn2 * (mm + __builtin_amdgcn_logf(ll)) : -__builtin_inff();
    for (int d = at; d < dim; d += 64) {
        f32x4 sum = {0, 0, 0, 0};
        for (int z = 0; z < a.splits; ++z) {
            const float f = __builtin_amdgcn_exp2f(p[z * step + dim] - mm);
            const f32x4 v = *(const f32x4 *)(p + z * step + d);
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] = __builtin_fmaf(f, v[e], sum[e]);
        }
        *(u32x2 *)(a.out + orow * a.ldo + (int64_t)qh * dim + d) =
            u32x2{bf16x2_rne(sum[0] * by, sum[1] * by), bf16x2_rne(sum[2] * by, sum[3] * by)};
    }
}

template <int C, bool HALF>
void launch_dim(const AttnArgs &a, int shift, hipStream_t stream) {
    const dim3 grid((uint32_t)(a.items * a.heads * a.splits));
    if (shift == 4) attn_rows_kernel<C, HALF><<<grid, kWaves * 64, 0, stream>>>(a);
    else attn_tile_kernel<C, HALF><<<grid, 256, 0, stream>>>(a);
}

struct Plan {
    int64_t items;
    int tiles, splits, shift;
};
// The kernel by the packed rows of a sequence, and over how many workgroups the tokens of a
// tile are split: enough of them for the card, at least 256 tokens each.
Plan attn_plan(int64_t rows, int64_t seqs, bool ragged, int64_t max_rows, int64_t max_tokens,
               int q_heads, int kv_heads) {
    const int64_t group = q_heads / kv_heads;
    max_rows = !ragged ? 1 : max_rows < rows ? max_rows : rows;
    Plan p;
    p.shift = max_rows * group <= 32 ? 4 : kTileShift;
    const int64_t height = 1 << p.shift;
    const int64_t tiles = (max_rows * group + height - 1) / height;
    const int64_t loose = kv_tile_items(rows, seqs, group, p.shift);
    p.tiles = !ragged || seqs * tiles <= loose ? (int)tiles : 0;
    p.items = p.tiles ? seqs * tiles : loose;
    const int64_t work = p.items * kv_heads, most = (max_tokens + 255) / 256;
    const int64_t want = p.shift == 4 ? 2048 : 512;
    int64_t splits = work ? (want + work - 1) / work : 1;
    splits = splits < most ? splits : most;
    p.splits = (int)(splits < 1 ? 1 : splits > 128 ? 128 : splits);
    return p;
}

}  // namespace

size_t attn_workspace_bytes(int64_t rows, int64_t seqs, bool ragged, int64_t max_rows,
                            int64_t max_tokens, int q_heads, int kv_heads, int dim) {
    const Plan p = attn_plan(rows, seqs, ragged, max_rows, max_tokens, q_heads, kv_heads);
    return p.splits > 1 ? ((size_t)p.items * kv_heads * p.splits << p.shift) * (dim + 4) * 4 : 0;
}

int64_t attn_grid(int64_t rows, int64_t seqs, bool ragged, int64_t max_rows, int64_t max_tokens,
                  int q_heads, int kv_heads) {
    const Plan p = attn_plan(rows, seqs, ragged, max_rows, max_tokens, q_heads, kv_heads);
    const int64_t slabs = 1 << (p.shift - 4);
    return p.items * kv_heads * (p.splits > slabs ? p.splits : slabs);
}

hipError_t launch_attn(const KvCall &c, const uint16_t *q, int64_t ldq, const uint8_t *kv,
                       const float *kv_scale, int64_t max_rows, int32_t q_heads, bool causal,
                       int32_t window, float scale, uint16_t *out, int64_t ldo, float *lse,
                       void *workspace, hipStream_t stream) {
    const Plan p = attn_plan(c.rows, c.seqs, c.start != nullptr, max_rows,
                             (int64_t)c.blocks * c.page, q_heads, c.kv_heads);
    AttnArgs a;
    a.b = KvBatch{c.start, c.lens, c.table, c.ldb, c.seqs, c.blocks, c.pages, (int32_t)c.rows,
                  __builtin_ctz(c.page)};
    a.q = q;
    a.kv = kv;
    a.kv_scale = kv_scale;
    a.out = out;
    a.lse = lse;
    a.part = p.splits > 1 ? (float *)workspace : nullptr;
    a.ldq = ldq;
    a.ldo = ldo;
    a.heads = c.kv_heads;
    a.group = q_heads / c.kv_heads;
    a.max_rows = (int)(max_rows < c.rows ? max_rows : c.rows);
    a.causal = causal ? 1 : 0;
    a.window = window;
    a.splits = p.splits;
    a.tiles = p.tiles;
    a.items = p.items;
    a.scale = scale * 1.44269504088896f;
    switch (c.dim / 32) {
        case 1: launch_dim<0, true>(a, p.shift, stream); break;
        case 2: launch_dim<1, false>(a, p.shift, stream); break;
        case 3: launch_dim<1, true>(a, p.shift, stream); break;
        case 4: launch_dim<2, false>(a, p.shift, stream); break;
        case 5: launch_dim<2, true>(a, p.shift, stream); break;
        case 6: launch_dim<3, false>(a, p.shift, stream); break;
        case 7: launch_dim<3, true>(a, p.shift, stream); break;
        default: launch_dim<4, false>(a, p.shift, stream); break;
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    attn_join_kernel<<<dim3((uint32_t)(p.items * c.kv_heads << (p.shift - 4))), 256, 0, stream>>>(
        a, c.dim, p.shift);
    return hipGetLastError();
}

}  // namespace w4a8

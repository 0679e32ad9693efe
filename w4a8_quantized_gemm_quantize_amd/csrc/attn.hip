// attn.hip -- attention of query rows over the paged 8-bit cache (w4a8_attn_kv8 in w4a8.h).
//
// The G = q_heads / kv_heads query heads of a cache head share its keys and values, so the
// rows of a tile are (row i of the sequence, head g of the group), i G + g: the columns of
// the matrix products
//   S [token][row] = K Q^T   and   O^T [element][row] += V^T P
// with v_mfma_f32_16x16x32_f16 or _32x32x16_f16.  K and V are bytes u = code + 128; the half 0x6400 | u is
// 1024 + u, so one byte permutation and one packed subtraction of 1152 make two exact
// codes.  Q enters as halves too, each row scaled by a power of two that puts its largest
// element just below 2^15: exact, but for elements under 2^-29 of that.  The products'
// results arrive in the lanes that the next product's operand needs (kv_index.hpp).
//
// Softmax in base 2 in one pass: with s_j = (scale log2 e) k_scale (q . k_j) of a token in a
// page of value scale sv,
//   t_j = s_j + log2 sv,   p_j = 2^(t_j - m),   O = sum p_j codes_j,   l = sum p_j / sv,
//   out = O / l,   lse = ln 2 (m + log2 l)
// so P needs no factor per page, and what its rounding to a half loses (2^-12 of a p_j, or
// 2^-25 where it is below 2^-14) is measured against the largest product p_j sv, not against
// p_j alone.  Few rows, which memory bounds, take what the half leaves of p_j through a second
// product (kLow); prompts, which the products bound, would need half as many again.  t, m, l and O are binary32.  m is no maximum but near one: it moves, to the
// maximum less 4, only when some p_j come out so large that a lane's sum of them exceeds
// 2^14, which a half still holds; so no maximum is taken while nothing overflows, and most
// tiles rescale nothing.  A factor of scores below 1e-30 counts as 1e-30, so that hidden
// tokens' -inf stays one where a page's keys are all 0.
//
// Taking l from the p_j holds while scales lie between 2^-40 and 2^20: then p_j counts in l
// only from 2^-110 on, where exp2 still has it, and l stays in 2^-16 .. 2^84 (2^30 tokens).
// From the first page on that a row of the wavefront sees and whose scale lies outside, zero
// among them, the wavefront takes l's weights by themselves, against a reference of their own:
//   l = sum 2^(s_j - ml),   out = O 2^(m - ml) / l,   lse = ln 2 (ml + log2 l),
// with ml = m before.  Such a page has a log2 sv that makes any weight overflow, so that it is
// found without a test per page, and from there on every sum of weights counts as too large.
// (Values of 1e-10 to 1e8 never get there, and pay nothing up to 128 elements a head; prompts
// of 3000 rows, 32 heads of 192 and 256: 102 -> 105 and 135 -> 140 us, by registers.)
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
    _Float16 *halves;              // the cache as halves (attn_halves_kernel; null: none)
    f32x4 *halves_terms;
    int runs;                      // of 64 tokens, that it has place for a sequence
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

// The largest of a row's bf16 by their bits without the sign, NaN above infinity: even and odd
// elements apart, then of both as binary32.
__device__ __forceinline__ uint32_t max_bits(uint32_t top, uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(v2u16, top),
                                                                  __builtin_bit_cast(v2u16, w & 0x7fff7fffu)));
}
__device__ __forceinline__ uint32_t top_bits(uint32_t top) { return max(top << 16, top & 0xffff0000u); }
// 2^e that brings a row of Q whose largest element has the bits `top` to [2^14, 2^15), with
// the sign of the scale; fac = |scale| / 2^e.  A row with an element that is no finite number
// has the factor NaN, and so has every row where the scale is none; such rows count as zeros
// (row_words).  No weight sees that factor (one is at least 1e-30); it makes NaN of the sum
// in the end, where the row saw anything (row_sum).
__device__ __forceinline__ float row_scale(uint32_t top, float scale, float &fac) {
    const bool none = top >= 0x7f800000u || !(fabsf(scale) < __builtin_inff());
    // 110 at most, so that fac keeps its bits: of smaller rows every element is then a multiple of
    // 2^(110 - 133), which a half holds, and no bit is lost
    const int e = min(110, 14 + 127 - (int)(top >> 23));
    fac = none ? __builtin_nanf("") : fabsf(scale) * __uint_as_float((uint32_t)(127 - e) << 23);
    return copysignf(__uint_as_float((uint32_t)(127 + e) << 23), scale);
}
template <int N>
__device__ __forceinline__ void row_words(u32x4 (&w)[N], float fac) {
    if (!__any(fac != fac)) return;
#pragma unroll
    for (int k = 0; k < N; ++k) w[k] = fac != fac ? u32x4{0, 0, 0, 0} : w[k];
}
__device__ __forceinline__ float row_sum(float l, float fac) { return l > 0.0f && fac != fac ? fac : l; }
// Of a page: key scale, log2 of the value scale, its inverse.  Without one log2 is -inf, so
// that every weight is 0.  For scales that l cannot be taken from p by (see above) log2 is
// kOdd, and the third term what it really is (finite, as weights of 0 are multiplied by it
// where the page is hidden; a scale of 0 has one that no weight survives).  A scale that is
// negative or no finite number must show in the rows that see the page and in no other, so it
// takes neither a product nor an infinity, which hidden tokens' -inf would turn into NaN, but
// a log2 that no weights have: m rises to it.
constexpr float kOdd = 3e38f, kBadScale = 3e38f;
__device__ __forceinline__ f32x4 page_terms(bool have, float sk, float sv) {
    if (!have) return f32x4{0.0f, -__builtin_inff(), 0.0f, 0.0f};
    if (!(fminf(sk, sv) >= 0.0f && sk < __builtin_inff() && sv < __builtin_inff()))
        return f32x4{0.0f, kOdd, kBadScale, 0.0f};
    if (sv >= 0x1p-40f && sv <= 0x1p20f)
        return f32x4{sk, __builtin_amdgcn_logf(sv), __builtin_amdgcn_rcpf(sv), 0.0f};
    // the instruction takes subnormal numbers for 0
    const float log_sv = sv < 1.0f ? __builtin_amdgcn_logf(sv * 0x1p32f) - 32.0f : __builtin_amdgcn_logf(sv);
    return f32x4{sk, kOdd, fmaxf(log_sv, -kOdd), 0.0f};
}
// A row's results from its statistics: x times the factors by and up, which together may be
// out of binary32's range, and its lse.
struct RowEnd {
    float by, up, lse;
    __device__ __forceinline__ float operator()(float x) const { return x * by * up; }
};
__device__ __forceinline__ RowEnd row_end(float m, float ml, float l) {
    if (m >= 1e38f) l = __builtin_nanf("");
    if (l == 0.0f) return RowEnd{0.0f, 0.0f, -__builtin_inff()};
    const float up = __builtin_amdgcn_exp2f(0.5f * (m - ml));
    return RowEnd{1.0f / l * up, up, kLn2 * (ml + __builtin_amdgcn_logf(l))};
}

constexpr float kLimit = 0x1p14f;                // of a lane's sum of weights
constexpr int kWaves = 4;
constexpr int kPairDim = 128;                    // 32 rows a wavefront up to here, by registers

// ---- few rows: 16 MT packed rows a workgroup ----
//
// A wavefront holds all the rows and takes every fourth run of 32 tokens of the workgroup's
// range; the four partial results are joined in LDS.  K and V go from memory straight to
// the registers they are multiplied from: the next run's keys as soon as this one's are
// used, then its values.  Bound by HBM: 64 x 8192 tokens, 8 heads of 128, 180 us or 5.9
// TB/s; with loads that also fill the L2 203 us, with both buffered twice (two wavefronts
// on a SIMD for three) 288 us.
template <int C, bool HALF, int MT>              // full chunks of 64 elements, and a half one
__global__ __launch_bounds__(kWaves * 64, MT == 2 ? 2 : 64 * C + 32 * HALF <= 64 ? 4 : 64 * C + 32 * HALF <= 128 ? 3 : 2)
void attn_rows_kernel(AttnArgs a) {
    constexpr int kDim = 64 * C + (HALF ? 32 : 0), kTiles = kDim / 16, kSteps = kDim / 32;
    constexpr int kStride = kDim + 4, kRows = 16 * MT, kShift = MT == 2 ? 5 : 4;
    // Weights as two halves, 22 bits: free for 16 rows (64 x 8192 tokens 181 us for 182, heads of
    // 96 with three wavefronts a SIMD for four); 24, 40 and 64 rows of the other form would pay
    // 60 -> 63, 75 -> 86 and 74 -> 87 us.
    constexpr bool kLow = MT == 1;
    __shared__ __attribute__((aligned(16))) float lds[kWaves * kRows * kStride];
    __shared__ float lds_m[kWaves * kRows], lds_l[kWaves * kRows], lds_ml[kWaves * kRows];
    const int split = blockIdx.x % a.splits;
    const int head = blockIdx.x / a.splits % a.heads;
    const int64_t item = blockIdx.x / a.splits / a.heads;
    KvTile t;
    if (!find_tile(a, item, kShift, t)) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int col = lane & 15, g = lane >> 4;
    const int from = t.seq.len - t.seq.n;

    // this lane's rows of Q, scaled, and the tokens they see, [see_lo, see_hi)
    half8_t q[MT][kSteps];
    float qfac[MT];
    int see_hi[MT], see_lo[MT];
#pragma unroll
    for (int x = 0; x < MT; ++x) {
        const int r = t.row0 + 16 * x + col, i = r / a.group, pos = from + i;
        const bool live = 16 * x + col < t.rows;
        see_hi[x] = a.causal ? min(t.hi, pos + 1) : t.hi;
        see_lo[x] = a.window ? max(0, pos - a.window + 1) : 0;
        const uint16_t *p = a.q + (int64_t)(t.seq.first_row + i) * a.ldq +
                            (int64_t)(head * a.group + r - i * a.group) * kDim;
        u32x4 w[kSteps];
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            const int d = k < 2 * C ? (k >> 1) * 64 + 16 * g + 8 * (k & 1) : C * 64 + 8 * g;
            w[k] = live ? *(const u32x4 *)(p + d) : u32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 4; ++i) top = max_bits(top, w[k][i]);
        }
        top = top_bits(top);
        top = max(top, (uint32_t)__shfl_xor((int)top, 16));
        top = max(top, (uint32_t)__shfl_xor((int)top, 32));
        const float up = row_scale(top, a.scale, qfac[x]);
        row_words(w, qfac[x]);
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            float f[8];
            bf16x8_to_f32(w[k], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) q[x][k][e] = (_Float16)(f[e] * up);
        }
    }
    // tokens that every row sees
    const int all_hi = a.causal ? min(t.hi, from + t.row0 / a.group + 1) : t.hi;
    const int all_lo = a.window ? from + (t.row0 + t.rows - 1) / a.group - a.window + 1 : 0;

    const int u_first = t.lo >> 5, u_all = ((t.hi + 31) >> 5) - u_first;
    const int u0 = u_first + (int)((int64_t)u_all * split / a.splits) + wave;
    const int u1 = u_first + (int)((int64_t)u_all * (split + 1) / a.splits);

    f32x4 o[MT][kTiles];
    float m[MT], ml[MT], l[MT];
    float limit = kLimit;                        // below 0: l's weights by themselves
#pragma unroll
    for (int r = 0; r < MT; ++r) {
#pragma unroll
        for (int d = 0; d < kTiles; ++d) o[r][d] = f32x4{0, 0, 0, 0};
        m[r] = ml[r] = -1e30f;
        l[r] = 0.0f;
    }

    // Lane x: of this wavefront's run n_in + x, for its two tiles of 16 tokens the place of
    // their keys and the page's terms, 64 runs at a time.  Without a page the place is the
    // cache's first and the weights are 0.
    int n_in = 0;
    int64_t at_in[2];
    f32x4 terms_in[2];
    auto look_up = [&](int n) {
        n_in = n;
        const int64_t u = u0 + (int64_t)(n + lane) * kWaves;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t at = u * 32 + h * 16;
            const int page = u < u1 && at < t.hi ? kv_page(a.b, t.s, at >> a.b.page_shift) : -1;
            at_in[h] = 0;
            float sk = 0.0f, sv = 0.0f;
            if (page >= 0) {
                const int64_t ph = (int64_t)page * a.heads + head;
                at_in[h] = ((ph * 2 << a.b.page_shift) + (at & ((1 << a.b.page_shift) - 1))) * kDim;
                sk = a.kv_scale[ph * 2];
                sv = a.kv_scale[ph * 2 + 1];
            }
            terms_in[h] = page_terms(page >= 0, sk, sv);
        }
    };
    const int64_t to_values = (int64_t)kDim << a.b.page_shift;
    struct Run {
        u32x4 k[2][C ? C : 1], v[2][C ? C : 1];
        u32x2 kh[2], vh[2];
    } x;
    auto lane_value = [](float v, int at) {
        return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), at));
    };
    auto place = [&](int n, int h) {
        const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)at_in[h], n - n_in);
        const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(at_in[h] >> 32), n - n_in);
        return (int64_t)(((uint64_t)hi << 32) | lo);
    };
    auto load_keys = [&](int n) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint8_t *p = a.kv + place(n, h);
#pragma unroll
            for (int c = 0; c < C; ++c) x.k[h][c] = __builtin_nontemporal_load((const u32x4 *)(p + c * 1024 + lane * 16));
            if constexpr (HALF) x.kh[h] = __builtin_nontemporal_load((const u32x2 *)(p + C * 1024 + lane * 8));
        }
    };
    auto load_values = [&](int n) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint8_t *p = a.kv + place(n, h) + to_values;
#pragma unroll
            for (int c = 0; c < C; ++c) x.v[h][c] = __builtin_nontemporal_load((const u32x4 *)(p + c * 1024 + lane * 16));
            if constexpr (HALF) x.vh[h] = __builtin_nontemporal_load((const u32x2 *)(p + C * 1024 + lane * 8));
        }
    };
    auto work = [&](int n) {
        const int first = (u0 + n * kWaves) * 32;
        float sk[2], log_sv[2], inv_sv[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            sk[h] = lane_value(terms_in[h].x, n - n_in);
            log_sv[h] = lane_value(terms_in[h].y, n - n_in);
            inv_sv[h] = lane_value(terms_in[h].z, n - n_in);
        }
        // scores of two tiles of 16 tokens
        f32x4 s[MT][2];
#pragma unroll
        for (int r = 0; r < MT; ++r) s[r][0] = s[r][1] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const half8_t key = codes8h(x.k[h][c][2 * k], x.k[h][c][2 * k + 1]);
#pragma unroll
                    for (int r = 0; r < MT; ++r) s[r][h] = mfma16(key, q[r][2 * c + k], s[r][h]);
                }
        if constexpr (HALF) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const half8_t key = codes8h(x.kh[h].x, x.kh[h].y);
#pragma unroll
                for (int r = 0; r < MT; ++r) s[r][h] = mfma16(key, q[r][2 * C], s[r][h]);
            }
        }
        if (n + 1 - n_in == 64) look_up(n + 1);
        load_keys(n + 1);
        half8_t p[MT], low;
        auto weight = [&](float w, int r, int at) {
            p[r][at] = (_Float16)w;
            if constexpr (kLow) low[at] = (_Float16)(w - (float)p[r][at]);
        };
#pragma unroll
        for (int r = 0; r < MT; ++r) {
            if (first + 32 > all_hi || first < all_lo) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = first + h * 16 + 4 * g + e;
                        if (j < see_lo[r] || j >= see_hi[r]) s[r][h][e] = -__builtin_inff();
                    }
            }
            float f[2], sum[2];
            auto weights = [&]() {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    f[h] = fmaxf(qfac[r] * sk[h], 1e-30f);
                    const float off = log_sv[h] - m[r];
                    sum[h] = 0.0f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r][h][e], f[h], off));
                        sum[h] += w;
                        weight(w, r, 4 * h + e);
                    }
                }
            };
            weights();
            if (__any(!(fmaxf(sum[0], sum[1]) <= limit))) {
                const bool odd = limit < 0.0f || log_sv[0] == kOdd || log_sv[1] == kOdd;
                if (odd) limit = -1.0f;
                float log_v[2] = {log_sv[0], log_sv[1]}, best = -1e30f, best_l = -1e30f;
                if (odd) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (log_sv[h] == kOdd) log_v[h] = inv_sv[h];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (log_sv[h] == -__builtin_inff()) s[r][h][e] = -__builtin_inff();   // no page
                            best_l = fmaxf(best_l, s[r][h][e] * f[h]);
                        }
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        best = fmaxf(best, __builtin_fmaf(s[r][h][e], f[h], log_v[h]));
                const float top = fmaxf(m[r], quad_max(best) - 4.0f);
                const float down = __builtin_amdgcn_exp2f(m[r] - top);
                m[r] = top;
                if (!odd) {
                    ml[r] = top;
                    l[r] *= down;
                    weights();
                } else {
                    const float top_l = fmaxf(ml[r], quad_max(best_l) - 4.0f);
                    l[r] *= __builtin_amdgcn_exp2f(ml[r] - top_l);
                    ml[r] = top_l;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float off = log_v[h] - top;
                        sum[h] = 0.0f;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            weight(__builtin_amdgcn_exp2f(__builtin_fmaf(s[r][h][e], f[h], off)), r, 4 * h + e);
                            l[r] += __builtin_amdgcn_exp2f(__builtin_fmaf(s[r][h][e], f[h], -top_l));
                        }
                    }
                }
#pragma unroll
                for (int d = 0; d < kTiles; ++d) o[r][d] *= down;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) l[r] = __builtin_fmaf(sum[h], inv_sv[h], l[r]);
        }
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const half8_t value = codes8h(x.v[0][c][j], x.v[1][c][j]);
#pragma unroll
                for (int r = 0; r < MT; ++r) o[r][4 * c + j] = mfma16(value, p[r], o[r][4 * c + j]);
                if constexpr (kLow) o[0][4 * c + j] = mfma16(value, low, o[0][4 * c + j]);
            }
        if constexpr (HALF) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const half8_t value = codes8h(x.vh[0][j], x.vh[1][j]);
#pragma unroll
                for (int r = 0; r < MT; ++r) o[r][4 * C + j] = mfma16(value, p[r], o[r][4 * C + j]);
                if constexpr (kLow) o[0][4 * C + j] = mfma16(value, low, o[0][4 * C + j]);
            }
        }
        load_values(n + 1);
    };

    const int runs = u0 < u1 ? (u1 - u0 + kWaves - 1) / kWaves : 0;
    if (runs) {
        look_up(0);
        load_keys(0);
        load_values(0);
        for (int n = 0; n < runs; ++n) work(n);
    }
#pragma unroll
    for (int r = 0; r < MT; ++r) {
        l[r] = row_sum(quad_sum(l[r]), qfac[r]);
        const int row = wave * kRows + 16 * r + col;
#pragma unroll
        for (int d = 0; d < kTiles; ++d) *(f32x4 *)(lds + row * kStride + d * 16 + 4 * g) = o[r][d];
        if (g == 0) {
            lds_m[row] = m[r];
            lds_ml[row] = ml[r];
            lds_l[row] = l[r];
        }
    }
    __syncthreads();
    // 16 threads a row, 4 elements each at a time
#pragma unroll
    for (int x16 = 0; x16 < MT; ++x16) {
        const int row = 16 * x16 + (threadIdx.x >> 4), at = (threadIdx.x & 15) * 4;
        if (row >= t.rows) return;
        float mm = lds_m[row], mml = lds_ml[row];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) {
            mm = fmaxf(mm, lds_m[w * kRows + row]);
            mml = fmaxf(mml, lds_ml[w * kRows + row]);
        }
        float f[kWaves], ll = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            f[w] = __builtin_amdgcn_exp2f(lds_m[w * kRows + row] - mm);
            ll = __builtin_fmaf(__builtin_amdgcn_exp2f(lds_ml[w * kRows + row] - mml),
                                lds_l[w * kRows + row], ll);
        }
        const int rr = t.row0 + row, ri = rr / a.group, qh = head * a.group + rr - ri * a.group;
        const int64_t orow = t.seq.first_row + ri;
        float *part = nullptr;
        const RowEnd end = row_end(mm, mml, ll);
        if (a.part) {
            part = a.part + ((((item * a.heads + head) * a.splits + split) << kShift) + row) * (kDim + 4);
            if (at == 0) {
                part[kDim] = mm;
                part[kDim + 1] = ll;
                part[kDim + 2] = mml;
            }
        } else if (at == 0 && a.lse) {
            a.lse[orow * a.heads * a.group + qh] = end.lse;
        }
        for (int d = at; d < kDim; d += 64) {
            f32x4 sum = {0, 0, 0, 0};
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const f32x4 v = *(const f32x4 *)(lds + (w * kRows + row) * kStride + d);
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[e] = __builtin_fmaf(f[w], v[e], sum[e]);
            }
            if (a.part) {
                *(f32x4 *)(part + d) = sum;
            } else {
                *(u32x2 *)(a.out + orow * a.ldo + (int64_t)qh * kDim + d) =
                    u32x2{bf16x2_rne(end(sum[0]), end(sum[1])), bf16x2_rne(end(sum[2]), end(sum[3]))};
            }
        }
    }
}

// ---- many rows: 128 packed rows a workgroup, 32 a wavefront ----
//
// The wavefronts share 64 tokens at a time, converted once to halves in LDS in the order of
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
// Workgroups of a compute unit, by registers and LDS.  (Workgroups of eight wavefronts and 256
// rows stage half as much each, and gained nothing while every tile converted its tokens: 671
// us for 673 on 5124 and 3067 rows of 64 x 128, 8 us more on short prompts, which have too few.)
constexpr int tile_groups(int dim) { return dim <= 64 ? 3 : dim <= 128 ? 2 : 1; }
constexpr int kTileShift = 7;                    // packed rows of a tile: 128
constexpr int kWaitLoads = 0x0f70;               // s_waitcnt vmcnt(0)

// A run of 64 tokens of a sequence and head as halves: keys, then values as they are in LDS.
__device__ __forceinline__ int64_t halves_run(const AttnArgs &a, int s, int head, int run) {
    return ((int64_t)s * a.heads + head) * a.runs + run;
}
// 16 bytes of keys, 4 of values of a record to their place in the run's image.
template <int C, bool HALF>
struct Halves {
    static constexpr int kDim = 64 * C + (HALF ? 32 : 0), kSub = 16 * kDim;
    static constexpr int kKeyPieces = 2 * C + HALF, kValuePieces = 4 * C + 2 * HALF;
    u32x4 r[C ? C : 1];
    u32x2 h;
    __device__ __forceinline__ void load(const uint8_t *p, int lane) {
#pragma unroll
        for (int c = 0; c < C; ++c) r[c] = *(const u32x4 *)(p + c * 1024 + lane * 16);
        if constexpr (HALF) h = *(const u32x2 *)(p + C * 1024 + lane * 8);
    }
    // n: half a record; `to` the 16 tokens' keys
    __device__ __forceinline__ void key(_Float16 *to, int lane, int n) const {
        const int c = n >> 1, x = 2 * (n & 1);
        *(half8_t *)(to + n * 512 + lane * 8) = n < 2 * C ? codes8h(r[c < C ? c : 0][x], r[c < C ? c : 0][x + 1])
                                                          : codes8h(h.x, h.y);
    }
    static __device__ __forceinline__ int value_lane(int lane) {
        return (lane >> 4 & 1) * 256 + (lane & 15) * 8 + (lane >> 5) * 4;
    }
    // n: 16 elements; `to` the 16 tokens' values and value_lane
    __device__ __forceinline__ void value(_Float16 *to, int n) const {
        uint32_t lo, hi;
        codes4(n < 4 * C ? r[n < 4 * C ? n >> 2 : 0][n & 3] : h[n & 1], lo, hi);
        *(u32x2 *)(to + (n >> 1) * 512 + (n & 1) * 128) = u32x2{lo, hi};
    }
};

// The cache's tokens that the rows see as halves, once, where many tiles read each of them:
// those then copy them straight to LDS.  Converting in every tile costs its wavefronts 77 of
// 285 vector instructions a run, and the card, whose clock falls under this load, a fifth.
template <int C, bool HALF>
__global__ __launch_bounds__(256) void attn_halves_kernel(AttnArgs a) {
    using H = Halves<C, HALF>;
    const int head = blockIdx.x % a.heads;
    const int64_t at = blockIdx.x / a.heads;
    const int s = (int)(at / a.runs), run = (int)(at - (int64_t)s * a.runs);
    const KvSeq q = kv_seq(a.b, s);
    if (!kv_run_seen(a.b, q, run, a.window)) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int token = run * 64 + wave * 16;
    const int page = token < q.len ? kv_page(a.b, s, token >> a.b.page_shift) : -1;
    int64_t place = 0;                           // without a page the cache's first, weights 0
    float sk = 0.0f, sv = 0.0f;
    if (page >= 0) {
        const int64_t ph = (int64_t)page * a.heads + head;
        place = ((ph * 2 << a.b.page_shift) + (token & ((1 << a.b.page_shift) - 1))) * H::kDim;
        sk = a.kv_scale[ph * 2];
        sv = a.kv_scale[ph * 2 + 1];
    }
    H k, v;
    k.load(a.kv + place, lane);
    v.load(a.kv + place + ((int64_t)H::kDim << a.b.page_shift), lane);
    const int64_t r = halves_run(a, s, head, run);
    _Float16 *to = a.halves + r * (8 * H::kSub) + wave * H::kSub;
#pragma unroll
    for (int n = 0; n < H::kKeyPieces; ++n) k.key(to, lane, n);
    to += 4 * H::kSub + H::value_lane(lane);
#pragma unroll
    for (int n = 0; n < H::kValuePieces; ++n) v.value(to, n);
    if (lane == 0) a.halves_terms[r * 4 + wave] = page_terms(page >= 0, sk, sv);
}

// READY: from attn_halves_kernel's halves.
template <int C, bool HALF, bool READY>
__global__ __launch_bounds__(256, tile_groups(64 * C + 32 * HALF)) void attn_tile_kernel(AttnArgs a) {
    constexpr int kDim = 64 * C + (HALF ? 32 : 0), kSteps = kDim / 16, kBlocks = kDim / 32;
    constexpr int kSub = 16 * kDim;              // halves of 16 tokens
    __shared__ __attribute__((aligned(16))) _Float16 kbuf[2][4 * kSub], vbuf[2][4 * kSub];
    __shared__ f32x4 page[4][4];                 // of 16 tokens: page_terms
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
#pragma unroll
            for (int i = 0; i < 4; ++i) top = max_bits(top, w[k][i]);
        }
        top = top_bits(top);
        top = max(top, (uint32_t)__shfl_xor((int)top, 32));
        const float up = row_scale(top, a.scale, qfac);
        row_words(w, qfac);
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            float f[8];
            bf16x8_to_f32(w[k], f);
#pragma unroll
            for (int x = 0; x < 8; ++x) q[k][x] = (_Float16)(f[x] * up);
        }
    }
    const int pos = from + i;
    const int see_hi = a.causal ? min(t.hi, pos + 1) : t.hi;
    const int see_lo = a.window ? max(0, pos - a.window + 1) : 0;
    // tokens that every row of the wavefront sees
    const int row1 = t.row0 + wave * 32, row2 = max(row1, t.row0 + min(t.rows, wave * 32 + 32) - 1);
    const int all_hi = a.causal ? min(t.hi, from + row1 / a.group + 1) : t.hi;
    const int all_lo = a.window ? from + row2 / a.group - a.window + 1 : 0;

    const int j_first = t.lo >> 6, j_all = ((t.hi + 63) >> 6) - j_first;
    const int j0 = j_first + (int)((int64_t)j_all * split / a.splits);
    const int j1 = j_first + (int)((int64_t)j_all * (split + 1) / a.splits);

    f32x16 o[kBlocks];
#pragma unroll
    for (int d = 0; d < kBlocks; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[d][e] = 0.0f;
    float m = -1e30f, ml = -1e30f, l = 0.0f;
    float limit = kLimit;                        // below 0: l's weights by themselves

    // A wavefront stages 16 tokens of each run of 64.  Lane x: of the tokens of run j_in + x
    // the place of their keys and the page's terms, 64 runs at a time (as in attn_rows_kernel).
    int j_in = j0;
    int64_t at_in = 0;
    f32x4 terms_in;
    auto look_up = [&](int j) {
        j_in = j;
        const int64_t at = (int64_t)(j + lane) * 64 + wave * 16;
        const int pg = j + lane < j1 && at < t.hi ? kv_page(a.b, t.s, at >> a.b.page_shift) : -1;
        at_in = 0;
        float sk = 0.0f, sv = 0.0f;
        if (pg >= 0) {
            const int64_t ph = (int64_t)pg * a.heads + head;
            at_in = ((ph * 2 << a.b.page_shift) + (at & ((1 << a.b.page_shift) - 1))) * kDim;
            sk = a.kv_scale[ph * 2];
            sv = a.kv_scale[ph * 2 + 1];
        }
        terms_in = page_terms(pg >= 0, sk, sv);
    };
    auto part_of = [&](int j) -> int64_t {
        const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)at_in, j - j_in);
        const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(at_in >> 32), j - j_in);
        return (int64_t)(((uint64_t)hi << 32) | lo);
    };
    using H = Halves<C, HALF>;
    H kraw, vraw;
    f32x4 terms;
    auto lane_value = [](float v, int at) {
        return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), at));
    };
    const int64_t to_values = (int64_t)kDim << a.b.page_shift;
    auto load_keys = [&](int j) {
        kraw.load(a.kv + part_of(j), lane);
        terms = f32x4{lane_value(terms_in.x, j - j_in), lane_value(terms_in.y, j - j_in),
                      lane_value(terms_in.z, j - j_in), 0.0f};
    };
    auto load_values = [&](int j) { vraw.load(a.kv + part_of(j) + to_values, lane); };
    // What was loaded, as halves, in pieces: keys, then values.
    constexpr int kKeyPieces = H::kKeyPieces, kValuePieces = H::kValuePieces;
    _Float16 *const value_lane = vbuf[0] + wave * kSub + H::value_lane(lane);
    auto store_key = [&](int j, int n) { kraw.key(kbuf[j & 1] + wave * kSub, lane, n); };
    auto store_value = [&](int j, int n) { vraw.value(value_lane + (j & 1) * (4 * kSub), n); };
    auto store_terms = [&](int j) { page[j & 3][wave] = terms; };
    auto store_keys = [&](int j) {
#pragma unroll
        for (int n = 0; n < kKeyPieces; ++n) store_key(j, n);
        store_terms(j);
    };
    auto store_values = [&](int j) {
#pragma unroll
        for (int n = 0; n < kValuePieces; ++n) store_value(j, n);
    };
    // The same from halves that are there: 16 bytes a lane straight to LDS (the wavefront
    // waits for them before the barrier after the next half run).
    auto copy = [&](int j, bool values) {
        const int64_t r = halves_run(a, t.s, head, min(j, j1 - 1));
        const _Float16 *from = a.halves + r * (8 * kSub) + (values ? 4 * kSub : 0) + wave * kSub;
        _Float16 *to = (values ? vbuf[j & 1] : kbuf[j & 1]) + wave * kSub;
#pragma unroll
        for (int n = 0; n < kSub / 512; ++n) global_to_lds16(from + n * 512 + lane * 8, to + n * 512);
        if (!values && wave == 0 && lane < 4) global_to_lds16(a.halves_terms + r * 4 + lane, &page[j & 3][0]);
    };
    const int sub_lane = (lane & 31) >> 4, rec = (h * 16 + (lane & 15)) * 8;
    auto key_operand = [&](int j, int half, int k) {
        const int at = k < 4 * C ? ((k >> 2) * 2 + (k & 1)) * 512 + (k >> 1 & 1) * 256
                                 : C * 1024 + (k & 1) * 256;
        return *(const half8_t *)(kbuf[j & 1] + (2 * half + sub_lane) * kSub + rec + at);
    };
    auto value_operand = [&](int j, int x, int d) {
        return *(const half8_t *)(vbuf[j & 1] + x * kSub + d * 512 + lane * 8);
    };
    // Half a run: the weights p of 32 tokens from their scores s, and beside them, on the
    // matrix cores, the scores `next` of the 32 after and the products of the 32 before.
    auto step = [&](int j, int half, f32x16 &s, f32x16 &next, half8_t (&before)[2], half8_t (&p)[2]) {
        const int first = j * 64 + half * 32;
        if (first + 32 > all_hi || first < all_lo) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int at = first + 8 * (e >> 2) + 4 * h + (e & 3);
                if (at < see_lo || at >= see_hi) s[e] = -__builtin_inff();
            }
        }
        f32x4 pt[2];
        float f[2], sum[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            pt[x] = page[j & 3][2 * half + x];
            f[x] = fmaxf(qfac * pt[x].x, 1e-30f);
        }
        auto weights = [&]() {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float off = pt[x].y - m;
                sum[x] = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[8 * x + e], f[x], off));
                    sum[x] += w;
                    p[x][e] = (_Float16)w;
                }
            }
        };
        // One product at a time with its share of the weights' steps, in this order: the
        // scheduler left to itself puts the products first and the weights behind them.
        constexpr int kAll = 2 * kSteps, kAhead = 4;        // as many sums' as scores': kDim / 16
        auto operand = [&](int n) {              // products in turn: a score's, a sum's
            const int k = n / 2;
            return n % 2 == 0 ? key_operand(j + half, 1 - half, k)
                              : value_operand(j - 1 + half, 2 * (1 - half) + k / kBlocks, k % kBlocks);
        };
        half8_t ring[kAhead];
#pragma unroll
        for (int n = 0; n < kAhead; ++n) ring[n] = operand(n);
        const float off[2] = {pt[0].y - m, pt[1].y - m};
        float u[16], w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) next[e] = 0.0f;
#pragma unroll
        for (int x = 0; x < 2; ++x) sum[x] = 0.0f;
#pragma unroll
        for (int n = 0; n < kAll + 2; ++n) {
            if (n < kAll) {
                const int k = n / 2;
                if (n % 2 == 0) next = mfma32(ring[n % kAhead], q[k], next);
                else o[k % kBlocks] = mfma32(ring[n % kAhead], before[k / kBlocks], o[k % kBlocks]);
                if (n + kAhead < kAll) ring[n % kAhead] = operand(n + kAhead);
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                if (e * kAll / 16 == n) u[e] = __builtin_fmaf(s[e], f[e >> 3], off[e >> 3]);
                if (e * kAll / 16 == n - 1) w[e] = __builtin_amdgcn_exp2f(u[e]);
                if (e * kAll / 16 == n - 2) {
                    sum[e >> 3] += w[e];
                    if (e & 1) {
                        const half2_t c = __builtin_convertvector(f32x2_t{w[e - 1], w[e]}, half2_t);
                        p[e >> 3][(e & 7) - 1] = c[0];
                        p[e >> 3][e & 7] = c[1];
                    }
                }
            }
            if (half && !READY) {
                // and its share of the next tokens' halves
                constexpr int kPieces = kKeyPieces + kValuePieces;
#pragma unroll
                for (int i = 0; i < kPieces; ++i)
                    if (i * kAll / kPieces == n) {
                        if (i < kKeyPieces) store_key(j + 2, i);
                        else store_value(j + 1, i - kKeyPieces);
                    }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (half && !READY) store_terms(j + 2);
        const float most = fmaxf(sum[0], sum[1]);
        if (__builtin_expect(__any(!(most <= limit)), 0)) {
            const bool odd_page = __any(pt[0].y == kOdd || pt[1].y == kOdd);
            const bool odd = limit < 0.0f || odd_page;
            if (odd) limit = -1.0f;
            float log_v[2] = {pt[0].y, pt[1].y}, best = -1e30f, best_l = -1e30f;
            if (odd) {
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    if (pt[x].y == kOdd) log_v[x] = pt[x].z;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    if (pt[e >> 3].y == -__builtin_inff()) s[e] = -__builtin_inff();  // no page
                    best_l = fmaxf(best_l, s[e] * f[e >> 3]);
                }
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) best = fmaxf(best, __builtin_fmaf(s[e], f[e >> 3], log_v[e >> 3]));
            const float n = fmaxf(m, fmaxf(best, __shfl_xor(best, 32)) - 4.0f);
            const float down = __builtin_amdgcn_exp2f(m - n);
            m = n;
#pragma unroll
            for (int d = 0; d < kBlocks; ++d) o[d] *= down;
            if (!odd) {
                ml = n;
                l *= down;
                weights();
            } else {
                const float nl = fmaxf(ml, fmaxf(best_l, __shfl_xor(best_l, 32)) - 4.0f);
                l *= __builtin_amdgcn_exp2f(ml - nl);
                ml = nl;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float off = log_v[x] - n;
                    sum[x] = 0.0f;
                    pt[x].z = 1.0f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        p[x][e] = (_Float16)__builtin_amdgcn_exp2f(__builtin_fmaf(s[8 * x + e], f[x], off));
                        sum[x] += __builtin_amdgcn_exp2f(__builtin_fmaf(s[8 * x + e], f[x], -nl));
                    }
                }
                // Where m and ml are as close as scales between 2^-40 and 2^4 leave them, for
                // all rows, l is taken from p again (a first page of zeros, 5124 and 3067 rows
                // of 64 x 128: 995 us without).
                const float apart = nl - n;
                if (!odd_page && __all(apart >= -4.0f && apart <= 40.0f)) {
                    const float by = __builtin_amdgcn_exp2f(apart);
                    l *= by;
                    ml = n;
                    pt[0].z = pt[1].z = by;
                    limit = kLimit;
                }
            }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) l = __builtin_fmaf(sum[x], pt[x].z, l);
    };

    f32x16 s0, s1;
    half8_t p0[2], p1[2];
    if (j0 < j1) {
        // what the first step multiplies by 0
        for (int x = lane; x < kSub / 8; x += 64)
            *(u32x4 *)(vbuf[(j0 + 1) & 1] + wave * kSub + x * 8) = u32x4{0, 0, 0, 0};
        if constexpr (READY) {
            copy(j0, false);
            copy(j0, true);
            copy(j0 + 1, false);
            __builtin_amdgcn_s_waitcnt(kWaitLoads);
        } else {
            look_up(j0);
            load_keys(j0);
            load_values(j0);
            store_keys(j0);
            store_values(j0);
            load_keys(j0 + 1);
            load_values(j0 + 1);
            store_keys(j0 + 1);
            load_keys(j0 + 2);
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 16; ++e) s0[e] = 0.0f;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) s0 = mfma32(key_operand(j0, 0, k), q[k], s0);
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int e = 0; e < 8; ++e) p1[x][e] = (_Float16)0.0f;
    }
    for (int j = j0; j < j1; ++j) {
        step(j, 0, s0, s1, p1, p0);
        if constexpr (READY) __builtin_amdgcn_s_waitcnt(kWaitLoads);
        __syncthreads();
        if constexpr (READY) {
            copy(j + 2, false);
            copy(j + 1, true);
        }
        step(j, 1, s1, s0, p0, p1);
        if constexpr (!READY) {
            load_values(j + 2);
            if (j + 3 - j_in == 64) look_up(j + 3);
            load_keys(j + 3);
        }
    }
    if constexpr (READY) __builtin_amdgcn_s_waitcnt(kWaitLoads);   // none outlives the wavefront
    if (j0 < j1) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int d = 0; d < kBlocks; ++d) o[d] = mfma32(value_operand(j1 - 1, 2 + x, d), p1[x], o[d]);
    }
    l = row_sum(l + __shfl_xor(l, 32), qfac);
    const int qh = head * a.group + r - i * a.group;
    const int64_t orow = t.seq.first_row + i;
    if (a.part) {
        if (!live) return;
        float *part = a.part + ((((item * a.heads + head) * a.splits + split) << kTileShift) + wave * 32 + col) *
                                   (kDim + 4);
        if (h == 0) {
            part[kDim] = m;
            part[kDim + 1] = l;
            part[kDim + 2] = ml;
        }
#pragma unroll
        for (int d = 0; d < kBlocks; ++d)
#pragma unroll
            for (int x = 0; x < 4; ++x)
                *(f32x4 *)(part + d * 32 + 8 * x + 4 * h) =
                    f32x4{o[d][4 * x], o[d][4 * x + 1], o[d][4 * x + 2], o[d][4 * x + 3]};
        return;
    }
    if (!live) return;
    const RowEnd end = row_end(m, ml, l);
    if (h == 0 && a.lse) a.lse[orow * a.heads * a.group + qh] = end.lse;
    uint16_t *out = a.out + orow * a.ldo + (int64_t)qh * kDim;
#pragma unroll
    for (int d = 0; d < kBlocks; ++d)
#pragma unroll
        for (int x = 0; x < 4; ++x)
            *(u32x2 *)(out + d * 32 + 8 * x + 4 * h) =
                u32x2{bf16x2_rne(end(o[d][4 * x]), end(o[d][4 * x + 1])),
                      bf16x2_rne(end(o[d][4 * x + 2]), end(o[d][4 * x + 3]))};
}

// Joins the splits of a tile, one wavefront a row: lane z holds the factors of splits z and
// z + 64, then groups of dim / 4 lanes sum every group-th split's row.  (16 lanes a row, one
// split after the other: 126 us for 86 splits of 3 x 8 tiles, where the attention took 136.)
constexpr int kMaxSplits = 128;
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, int dim, int shift) {
    const int64_t at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);     // item, head, row
    const int row = (int)(at & ((1 << shift) - 1)), lane = threadIdx.x & 63;
    const int64_t slot = at >> shift, item = slot / a.heads;
    const int head = (int)(slot - item * a.heads);
    KvTile t;
    if (item >= a.items || !find_tile(a, item, shift, t) || row >= t.rows) return;
    const int64_t step = (int64_t)(dim + 4) << shift;
    const float *p = a.part + slot * a.splits * step + row * (dim + 4);
    float m[2], l[2], ml[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int z = lane + 64 * x;
        m[x] = z < a.splits ? p[z * step + dim] : -1e30f;
        l[x] = z < a.splits ? p[z * step + dim + 1] : 0.0f;
        ml[x] = z < a.splits ? p[z * step + dim + 2] : -1e30f;
    }
    float mm = fmaxf(m[0], m[1]), mml = fmaxf(ml[0], ml[1]);
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) {
        mm = fmaxf(mm, __shfl_xor(mm, x));
        mml = fmaxf(mml, __shfl_xor(mml, x));
    }
    const float f0 = __builtin_amdgcn_exp2f(m[0] - mm), f1 = __builtin_amdgcn_exp2f(m[1] - mm);
    float ll = __builtin_fmaf(__builtin_amdgcn_exp2f(ml[0] - mml), l[0],
                              __builtin_amdgcn_exp2f(ml[1] - mml) * l[1]);
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) ll += __shfl_xor(ll, x);
    const int rr = t.row0 + row, ri = rr / a.group, qh = head * a.group + rr - ri * a.group;
    const int64_t orow = t.seq.first_row + ri;
    const RowEnd end = row_end(mm, mml, ll);
    if (lane == 0 && a.lse) a.lse[orow * a.heads * a.group + qh] = end.lse;
    const int cols = dim >> 2, groups = 64 / cols, g = lane / cols, d = (lane - g * cols) * 4;
    f32x4 sum = {0, 0, 0, 0};
    for (int z0 = 0; z0 < a.splits; z0 += groups) {
        const int z = z0 + g;
        const float f = __shfl(z0 < 64 ? f0 : f1, z & 63);
        const float f_next = __shfl(f1, z & 63);        // a round of groups may reach over 64
        if (g < groups && z < a.splits) {
            const f32x4 v = *(const f32x4 *)(p + z * step + d);
            const float w = z0 < 64 && z >= 64 ? f_next : f;
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] = __builtin_fmaf(w, v[e], sum[e]);
        }
    }
    f32x4 all = sum;
    for (int x = 1; x < groups; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) all[e] += __shfl(sum[e], (lane + x * cols) & 63);
    if (g > 0) return;
    *(u32x2 *)(a.out + orow * a.ldo + (int64_t)qh * dim + d) =
        u32x2{bf16x2_rne(end(all[0]), end(all[1])), bf16x2_rne(end(all[2]), end(all[3]))};
}

// The same for few splits of tiles' many rows: 16 lanes a row and all its loads at once.  The
// whole call with a wavefront a row and with this, 8 x 64 rows of 32 heads by 4 splits: 92 and
// 85 us; 512 rows by 4: 65 and 60, by 8: 75.2 and 75.7, by 12: 91 and 99.  The join alone of
// 500 rows of 28 heads of 64 by 6: 10.5 and 6.1 us.
constexpr int kFewSplits = 8;
__global__ __launch_bounds__(256) void attn_join_few_kernel(AttnArgs a, int dim, int shift) {
    const int64_t at = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);    // item, head, row
    const int row = (int)(at & ((1 << shift) - 1)), d0 = (threadIdx.x & 15) * 4;
    // one item for the workgroup: tiles have 16 rows or more
    const int64_t slot = (int64_t)blockIdx.x * 16 >> shift, item = slot / a.heads;
    const int head = (int)(slot - item * a.heads);
    KvTile t;
    if (!find_tile(a, item, shift, t) || row >= t.rows) return;
    const int64_t step = (int64_t)(dim + 4) << shift;
    const float *p = a.part + slot * a.splits * step + row * (dim + 4);
    float f[kFewSplits], l[kFewSplits], ml[kFewSplits], mm = -1e30f, mml = -1e30f, ll = 0.0f;
#pragma unroll
    for (int z = 0; z < kFewSplits; ++z) {
        f[z] = z < a.splits ? p[z * step + dim] : -1e30f;
        l[z] = z < a.splits ? p[z * step + dim + 1] : 0.0f;
        ml[z] = z < a.splits ? p[z * step + dim + 2] : -1e30f;
    }
#pragma unroll
    for (int z = 0; z < kFewSplits; ++z) {
        mm = fmaxf(mm, f[z]);
        mml = fmaxf(mml, ml[z]);
    }
#pragma unroll
    for (int z = 0; z < kFewSplits; ++z) {
        f[z] = __builtin_amdgcn_exp2f(f[z] - mm);
        ll = __builtin_fmaf(__builtin_amdgcn_exp2f(ml[z] - mml), l[z], ll);
    }
    const RowEnd end = row_end(mm, mml, ll);
    const int rr = t.row0 + row, ri = rr / a.group, qh = head * a.group + rr - ri * a.group;
    const int64_t orow = t.seq.first_row + ri;
    if (d0 == 0 && a.lse) a.lse[orow * a.heads * a.group + qh] = end.lse;
    for (int d = d0; d < dim; d += 64) {
        f32x4 v[kFewSplits], sum = {0, 0, 0, 0};
#pragma unroll
        for (int z = 0; z < kFewSplits; ++z)
            v[z] = z < a.splits ? *(const f32x4 *)(p + z * step + d) : f32x4{0, 0, 0, 0};
#pragma unroll
        for (int z = 0; z < kFewSplits; ++z)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] = __builtin_fmaf(f[z], v[z][e], sum[e]);
        *(u32x2 *)(a.out + orow * a.ldo + (int64_t)qh * dim + d) =
            u32x2{bf16x2_rne(end(sum[0]), end(sum[1])), bf16x2_rne(end(sum[2]), end(sum[3]))};
    }
}

template <int C, bool HALF>
void launch_dim(const AttnArgs &a, int shift, hipStream_t stream) {
    const dim3 grid((uint32_t)(a.items * a.heads * a.splits));
    if (shift == 4) {
        attn_rows_kernel<C, HALF, 1><<<grid, kWaves * 64, 0, stream>>>(a);
    } else if (shift == 5) {
        if constexpr (64 * C + 32 * HALF <= kPairDim)
            attn_rows_kernel<C, HALF, 2><<<grid, kWaves * 64, 0, stream>>>(a);
    } else if (a.halves) {
        attn_halves_kernel<C, HALF>
            <<<dim3((uint32_t)((int64_t)a.b.seqs * a.runs * a.heads)), 256, 0, stream>>>(a);
        attn_tile_kernel<C, HALF, true><<<grid, 256, 0, stream>>>(a);
    } else {
        attn_tile_kernel<C, HALF, false><<<grid, 256, 0, stream>>>(a);
    }
}

struct Plan {
    int64_t items;
    int tiles, splits, shift;
    int64_t runs;                  // of the cache as halves, a sequence; 0: none
    size_t part_bytes, halves_bytes, terms_bytes;
};
// The kernel by the packed rows of a sequence: up to 64 go 16 or 32 a workgroup, that is,
// through the cache up to twice (four times past 128 elements a head), from the L2 after the
// first time: 32 x 4000 tokens, 8 heads of 128 with 24, 40, 64 and 80 rows: 60, 79, 84 and
// 165 us, 16 rows a workgroup 67, 127, 132 and 200, 128-row tiles 177, 181, 183 and 146.
// Then over how many workgroups the tokens of a tile are split: the least of a cost in
// microseconds,
//   rounds of workgroups over the card x tokens each x what one takes a token
//   + for more than one split its partial results and the second launch that joins them.
// Few rows: two workgroups a compute unit draw all that memory gives (64 x 8192 tokens, 8
// heads of 128: 183 us unsplit, 203, 197 and 200 us in 2, 3 and 4).  A workgroup alone takes
// 5.5 ns a token (one sequence, 8 heads of 128: 8.0, 16.3 and 27.4 us for 500, 2000 and 4000
// tokens), the join 3.5 us and 0.18 us a split (2000 tokens: 14.5, 12.2, 11.6, 12.3 and 15.5
// us in 2, 4, 8, 16 and 32).
Plan attn_plan(int64_t rows, int64_t seqs, bool ragged, int64_t max_rows, int64_t table_tokens,
               int window, int q_heads, int kv_heads, int dim) {
    const int64_t group = q_heads / kv_heads;
    max_rows = !ragged ? 1 : max_rows < rows ? max_rows : rows;
    int64_t max_tokens = table_tokens;
    Plan p;
    const int64_t packed = max_rows * group;
    p.shift = packed > 64 ? kTileShift : packed > 16 && dim <= kPairDim ? 5 : 4;
    const int64_t height = 1 << p.shift;
    const int64_t tiles = (max_rows * group + height - 1) / height;
    const int64_t loose = kv_tile_items(rows, seqs, group, p.shift);
    p.tiles = !ragged || seqs * tiles <= loose ? (int)tiles : 0;
    p.items = p.tiles ? seqs * tiles : loose;
    // a tile sees its window and as many tokens more as it has rows
    const int64_t seen = window + kv_min(max_rows, height / group + 2);
    if (window && seen < max_tokens) max_tokens = seen;
    const int64_t work = p.items * kv_heads, most = (max_tokens + 127) / 128;
    const int64_t places = device_cu_count() * (p.shift != kTileShift ? 2 : tile_groups(dim));
    const double token = (p.shift != kTileShift ? 5.5e-3 : 3.0e-2) * dim / 128;
    // partial results are written and read at about 4 TB/s (tiles: 512 rows of 4 heads of 96 in
    // 4 parts 14.2 us, unsplit 16.0; 256 rows 12.5 and 11.8)
    const double join = p.shift != kTileShift ? 3.5 : 6.0;
    const double each = 0.18 + 2e-6 * (double)(work << p.shift) * (dim + 4);
    double best = 0;
    p.splits = 1;
    for (int z = 1; z <= kMaxSplits && (z == 1 || z <= most); ++z) {
        const double rounds = (double)((work * z + places - 1) / places);
        const double cost = rounds * token * max_tokens / z + (z > 1 ? join + each * z : 0);
        if (z == 1 || cost < best) {
            best = cost;
            p.splits = z;
        }
    }
    p.part_bytes = p.splits > 1 ? ((size_t)work * p.splits << p.shift) * (dim + 4) * 4 : 0;
    // The cache as halves: where at least eight tiles read a token and the call is long enough
    // for the pass over the tokens (tiles x tokens x heads; 1.05 M: 66 us without, 70 with it,
    // 1.3 M: 122 and 120, 3.1 M: 215 and 207, 3.4 M: 190 and 180, 20 M: 666 and 640), and the
    // space for all tokens that the block tables could name is at most 1 GiB.
    p.runs = (table_tokens + 63) / 64;
    p.halves_bytes = (size_t)seqs * kv_heads * p.runs * 64 * dim * 4;
    p.terms_bytes = (size_t)seqs * kv_heads * p.runs * 64;
    // Of a windowed call a tile sees max_tokens, and a token is seen by so many tiles (5124 and
    // 3067 rows of 64 x 128, window 30: 132 us with it, 124 without, 128: 140 and 129, 1024: 308
    // and 311; 500 rows of 28 x 64, 512: 19.2 and 17.7).
    const int64_t many = rows * group / height;
    const int64_t readers = window ? kv_min(many, seqs * (window * group / height + 1)) : many;
    if (p.shift != kTileShift || readers < 8 * seqs || (double)many * kv_heads * max_tokens < 2e6 ||
        p.halves_bytes > (size_t)1 << 30 || seqs * kv_heads * p.runs >= (1 << 23))
        p.runs = p.halves_bytes = p.terms_bytes = 0;
    return p;
}

}  // namespace

size_t attn_workspace_bytes(int64_t rows, int64_t seqs, bool ragged, int64_t max_rows,
                            int64_t table_tokens, int q_heads, int kv_heads, int dim) {
    const Plan p = attn_plan(rows, seqs, ragged, max_rows, table_tokens, 0, q_heads, kv_heads, dim);
    return p.part_bytes + p.halves_bytes + p.terms_bytes;
}

int64_t attn_grid(int64_t rows, int64_t seqs, bool ragged, int64_t max_rows, int64_t table_tokens,
                  int q_heads, int kv_heads, int dim) {
    const Plan p = attn_plan(rows, seqs, ragged, max_rows, table_tokens, 0, q_heads, kv_heads, dim);
    return p.items * kv_heads * (p.splits == 1 ? 1 : p.splits > 1 << p.shift ? p.splits : 1 << p.shift);
}

hipError_t launch_attn(const KvCall &c, const uint16_t *q, int64_t ldq, const uint8_t *kv,
                       const float *kv_scale, int64_t max_rows, int32_t q_heads, bool causal,
                       int32_t window, float scale, uint16_t *out, int64_t ldo, float *lse,
                       void *workspace, hipStream_t stream) {
    const int64_t tokens = (int64_t)c.blocks * c.page;
    Plan p = attn_plan(c.rows, c.seqs, c.start != nullptr, max_rows, tokens, 0, q_heads, c.kv_heads,
                       c.dim);
    if (window) {                                // the workspace knows no window: never more of it
        const Plan w = attn_plan(c.rows, c.seqs, c.start != nullptr, max_rows, tokens, window, q_heads,
                                 c.kv_heads, c.dim);
        p.splits = w.splits < p.splits ? w.splits : p.splits;
        p.runs = w.runs < p.runs ? w.runs : p.runs;
    }
    AttnArgs a;
    a.b = KvBatch{c.start, c.lens, c.table, c.ldb, c.seqs, c.blocks, c.pages, (int32_t)c.rows,
                  __builtin_ctz(c.page)};
    a.q = q;
    a.kv = kv;
    a.kv_scale = kv_scale;
    a.out = out;
    a.lse = lse;
    a.part = p.splits > 1 ? (float *)workspace : nullptr;
    a.runs = (int)p.runs;
    a.halves = p.runs ? (_Float16 *)((uint8_t *)workspace + p.part_bytes) : nullptr;
    a.halves_terms = (f32x4 *)((uint8_t *)workspace + p.part_bytes + p.halves_bytes);
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
    const int64_t joins = p.items * c.kv_heads << p.shift;               // rows
    if (p.splits <= kFewSplits && p.shift == kTileShift)
        attn_join_few_kernel<<<dim3((uint32_t)(joins / 16)), 256, 0, stream>>>(a, c.dim, p.shift);
    else
        attn_join_kernel<<<dim3((uint32_t)(joins / 4)), 256, 0, stream>>>(a, c.dim, p.shift);
    return hipGetLastError();
}

}  // namespace w4a8

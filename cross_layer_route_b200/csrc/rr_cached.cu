// rr_cached.cu -- attention of a sequence's newest tokens over the paged cache
// (declared in include/rr_cache.h).
//
// A CTA takes a share of one sequence's tokens for one key head and up to 8 NT
// rows (query token, query head) that read it; its warps take 16 tokens at a
// time in turn, each with its own running softmax, so nothing in the loop waits
// for another warp.  Both products put the cache on the 16-row side of
// mma.sync m16n8k16, where none of it is wasted on padding, and take it straight
// from global memory:
//   S^T = K Q^T   A = 16 tokens x 16 dims.  A lane's 16-byte load of a token's
//                 row holds dims that need not be the ones of the standard
//                 fragment: the query fragments use the same order.
//   O^T = V^T P^T A = 16 dims x 16 tokens.  A lane holds 4 tokens' bytes of the
//                 same dims; bytes of two tokens are paired with prmt.
// Codes become f16 exactly.  The scales are powers of two: a row's goes to its
// score (keys) or its weight (values); with one for every 32 elements a code is
// multiplied by its group's scale over the row's largest, exact down to 2^-35.
// Weights are f16 and relative to the largest weight * scale seen so far, which
// stands at 2^7 (and at 2^15 before it is noticed), so neither a wide spread of
// scales nor a long tail of small weights is lost; the sum of the weights is
// fp32 and not rounded.  That reference is kept relative to the running maximum
// of the scores: a score of 2^24 or more would swallow a scale added to it.
// The references move only when a score passes them by 2^8: most steps then
// cost one vote and no shuffles.
// The loop is bound by HBM: a step's bytes are loaded one step ahead.
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>

#include "rr_cache.cuh"

namespace rr_cache {

using namespace rr_attn;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kAttnWarps = 8;
constexpr float kLift = 7.f;     // weights are 2^7 at the maximum
constexpr float kSlack = 8.f;    // ... and 2^15 at most
constexpr int kGroupLift = 12;   // codes of 4 bits carry 2^12
constexpr int kState = 4;        // floats beside a partial row: max, sum, value reference, nearest

struct Cached {
    rr_cache_config c;
    rr_cache_pool pool;
    rr_cached_attn_config n;
    rr_cached_attn_args a;
    float *part;       // [batch * heads, splits, rows, dh + kState]
    int shift;         // log2(chunk)
    int group, rows;   // query heads per key head, rows per key head
    int splits;
    float s1, s2;      // as in the masked attention
};

template <int FMT, int DH>
struct Words {
    static constexpr int kK = FMT == RR_E4M3 ? DH / 16 : DH / 32;   // 32-bit words of one key row a lane holds
    static constexpr int kV = FMT == RR_E4M3 ? DH / 32 : DH / 64;
    static constexpr int kRowBytes = FMT == RR_E4M3 ? DH : DH / 2;
    static constexpr int kGroups = FMT == RR_E4M3 ? 1 : DH / 32;
};

// One step's bytes: 16 tokens of a page.
template <int FMT, int DH>
struct Step {
    uint32_t k[2][Words<FMT, DH>::kK];   // tokens g, g + 8
    uint32_t v[4][Words<FMT, DH>::kV];   // tokens 2t, 2t + 1, 2t + 8, 2t + 9
    uint32_t ks[2], vs[2];               // scale bytes of tokens g, g + 8
    int pos;                             // position of token 0; < 0: skipped
};

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], const unsigned char *x) {
    if constexpr (N == 4) {
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(x));
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    } else if constexpr (N == 2) {
        const uint2 a = __ldg(reinterpret_cast<const uint2 *>(x));
        w[0] = a.x, w[1] = a.y;
    } else {
        w[0] = __ldg(reinterpret_cast<const uint32_t *>(x));
    }
}

template <int FMT, int DH>
__device__ __forceinline__ uint32_t load_scales(const unsigned char *scales, size_t row) {
    if constexpr (FMT == RR_E4M3) return __ldg(scales + row);
    else if constexpr (DH == 64) return __ldg(reinterpret_cast<const uint16_t *>(scales) + row);
    else return __ldg(reinterpret_cast<const uint32_t *>(scales) + row);
}

template <int FMT, int DH>
__device__ __forceinline__ void load_step(Step<FMT, DH> &s, const Cached &p, int head, int page, int pos, int len) {
    using W = Words<FMT, DH>;
    s.pos = pos;
    if (pos < 0) return;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int place = pos & (p.c.chunk - 1);
    const size_t krow = ((size_t)page * p.c.heads + head) * 2 * p.c.chunk + place, vrow = krow + p.c.chunk;
    const unsigned char *codes = static_cast<const unsigned char *>(p.pool.codes);
    const unsigned char *scales = static_cast<const unsigned char *>(p.pool.scales);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const unsigned char *x = codes + (krow + g + 8 * i) * W::kRowBytes;
        if constexpr (W::kK == 8) {
            uint32_t a[4], b[4];
            load_words(a, x + 16 * t);
            load_words(b, x + 64 + 16 * t);
#pragma unroll
            for (int j = 0; j < 4; ++j) s.k[i][j] = a[j], s.k[i][4 + j] = b[j];
        } else {
            load_words(s.k[i], x + 4 * W::kK * t);
        }
        s.ks[i] = load_scales<FMT, DH>(scales, krow + g + 8 * i);
        s.vs[i] = load_scales<FMT, DH>(scales, vrow + g + 8 * i);
    }
    // values behind the sequence's end are whatever the page held: a NaN code
    // there would meet a weight of zero in the product
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int tok = 2 * t + (i & 1) + 8 * (i >> 1);
        if (pos + tok < len) {
            load_words(s.v[i], codes + (vrow + tok) * W::kRowBytes + 4 * W::kV * g);
        } else {
#pragma unroll
            for (int j = 0; j < W::kV; ++j) s.v[i][j] = 0u;
        }
    }
}

__device__ __forceinline__ uint32_t f16x2_of_e4m3(uint32_t two) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
    return (uint32_t)h.x | (uint32_t)h.y << 16;
}
__device__ __forceinline__ uint32_t f16x2_of_e2m1(uint32_t two) {
    const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)two, __NV_E2M1);
    return (uint32_t)h.x | (uint32_t)h.y << 16;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    const __half2 c = __hmul2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&c);
}
// The 8x8 matrix of 16-bit elements a warp holds (row g, columns 2t, 2t + 1), transposed.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// Largest of a row's scale bytes that are not NaN (0 if all are).
template <int G>
__device__ __forceinline__ int top_scale(uint32_t w) {
    int m = 0;
#pragma unroll
    for (int i = 0; i < G; ++i) {
        const int b = (w >> (8 * i)) & 255;
        m = max(m, b == 255 ? 0 : b);
    }
    return m;
}
template <int G>
__device__ __forceinline__ bool has_nan(uint32_t w) {
    bool y = false;
#pragma unroll
    for (int i = 0; i < G; ++i) y = y || ((w >> (8 * i)) & 255) == 255;
    return y;
}
// 2^(byte - top + kGroupLift) in f16; zero below 2^-24 and for NaN bytes.
__device__ __forceinline__ uint32_t group_factor(uint32_t byte, int top) {
    const int e = (int)byte - top + kGroupLift;
    if (byte == 255 || e < -24) return 0;
    return e >= -14 ? (uint32_t)(e + 15) << 10 : 1u << (e + 24);
}

// Bits of one query row, as f16 scaled by a power of two that leaves its
// largest element in [2^13, 2^14) (elements 2^-37 below that are lost, which
// is 2^13 below the rounding of the scores' fp32 sums); returns the power.
__device__ __forceinline__ int query_shift(unsigned amax_bits) {
    const int e = (int)(amax_bits >> 23);
    return e == 0 || e == 255 ? 0 : 13 - (e - 127);
}

template <int FMT, int DH, int NT>
__global__ void __launch_bounds__(32 * kAttnWarps, NT <= 2 ? 2 : 1) cached_attention_kernel(const __grid_constant__ Cached p) {
    using W = Words<FMT, DH>;
    constexpr int kRows = 8 * NT, kQRow = DH + 4;      // padded query rows: lanes 8 banks apart
    constexpr int kMT = DH / 16;                       // 16-dim tiles of the values
    constexpr int kKeep = kMT * 4 * NT + 6 * NT;       // floats of a warp's state per lane
    extern __shared__ __align__(16) unsigned char smem[];
    __half *s_q = reinterpret_cast<__half *>(smem);                                   // [kRows][kQRow]
    float *s_row = reinterpret_cast<float *>(smem + kRows * kQRow * 2);               // [kRows] score factor
    int *s_near = reinterpret_cast<int *>(s_row + kRows);
    float *s_merge = reinterpret_cast<float *>(smem + kRows * kQRow * 2 + kRows * 4 + 16);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int head = blockIdx.y % p.c.heads, b = blockIdx.y / p.c.heads, row0 = blockIdx.z * kRows;
    const int len = p.a.seq_lens[b];
    const int32_t *table = p.a.page_table + (size_t)b * p.n.table_stride;
    const int32_t *route = p.a.route ? p.a.route + ((size_t)b * p.c.heads + head) * p.n.route_stride : nullptr;
    const int entries = len <= 0 ? 0 : route ? p.n.width : min(p.n.table_width, ((len - 1) >> p.shift) + 1);
    const int sub_shift = p.shift - 4;                 // steps per chunk
    const long long all = (long long)entries << sub_shift;
    const int begin = (int)(all * blockIdx.x / p.splits), end = (int)(all * (blockIdx.x + 1) / p.splits);

    // queries
    for (int r = warp; r < kRows; r += kAttnWarps) {
        const int row = row0 + r;
        float x[DH / 32];
        unsigned amax = 0;
#pragma unroll
        for (int i = 0; i < DH / 32; ++i) {
            x[i] = 0.f;
            if (row < p.rows) {
                const int64_t at = b * p.n.q_stride[0] + (row / p.group) * p.n.q_stride[1] +
                                   (head * p.group + row % p.group) * p.n.q_stride[2] + lane + 32 * i;
                x[i] = p.n.dtype == RR_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p.a.q)[at])
                                            : __half2float(static_cast<const __half *>(p.a.q)[at]);
            }
            amax = max(amax, __float_as_uint(x[i]) & 0x7fffffffu);
        }
        amax = __reduce_max_sync(kFull, amax);
        const int shift = query_shift(amax);
#pragma unroll
        for (int i = 0; i < DH / 32; ++i) s_q[r * kQRow + lane + 32 * i] = __float2half_rn(ldexpf(x[i], shift));
        if (lane == 0) s_row[r] = ldexpf(p.s1, -shift - (FMT == RR_E2M1 ? kGroupLift : 0));
    }
    // The distance that the bias is taken relative to: the newest token's to the
    // nearest key that has a page (see `nearest` of the masked attention).
    if (warp == 0) {
        int best = INT_MAX;
        if (p.a.slopes && len > 0) {
            for (int e0 = 0; e0 < entries; e0 += 32) {
                const int e = e0 + lane;
                if (e < entries) {
                    const int id = route ? route[e] : entries - 1 - e;
                    if (id >= 0 && id < p.n.table_width && (id << p.shift) < len) {
                        const int page = table[id];
                        if (page >= 0 && page < p.c.pages)
                            best = min(best, max(0, len - 1 - ((id << p.shift) + p.c.chunk - 1)));
                    }
                }
                if (!route && __any_sync(kFull, best != INT_MAX)) break;   // entries come nearest first
            }
            best = __reduce_min_sync(kFull, best);
        }
        if (lane == 0) *s_near = best == INT_MAX ? 0 : best;
    }
    __syncthreads();

    uint32_t qf[NT <= 2 ? NT : 1][DH / 16][2];
    auto query = [&](int nt, int j, uint32_t &b0, uint32_t &b1) {
        const int dim = FMT == RR_E2M1 ? (DH / 4) * t + 4 * j : 64 * (j / 4) + 16 * t + 4 * (j % 4);
        const uint2 w = *reinterpret_cast<const uint2 *>(s_q + (nt * 8 + g) * kQRow + dim);
        b0 = w.x;
        b1 = w.y;
    };
    if constexpr (NT <= 2) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < DH / 16; ++j) query(nt, j, qf[nt][j][0], qf[nt][j][1]);
    }

    // this lane's rows of every tile of 8: 2t, 2t + 1
    float rowf[NT][2], slope[NT][2];
    int pos_r[NT][2], near_r[NT][2];
    const bool bias = p.a.slopes != nullptr, cap = p.n.soft_cap > 0.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = nt * 8 + 2 * t + i, row = row0 + r;
            const int back = p.n.q_tokens - 1 - (row < p.rows ? row / p.group : 0);   // tokens after it
            rowf[nt][i] = s_row[r];
            pos_r[nt][i] = row < p.rows ? len - 1 - back : -1;
            near_r[nt][i] = max(0, *s_near - back);
            slope[nt][i] = bias && row < p.rows ? p.a.slopes[head * p.group + row % p.group] * kLog2e : 0.f;
        }

    float o[kMT][NT][4];
#pragma unroll
    for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
    float m1[NT][2], m2[NT][2], l[NT][2];
    uint32_t broken = 0;    // (row of the lane, group): a visible value's scale is NaN
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) m1[nt][0] = m1[nt][1] = m2[nt][0] = m2[nt][1] = -INFINITY, l[nt][0] = l[nt][1] = 0.f;

    // A warp's steps begin + warp, + kAttnWarps, ...; lane i looks up the page of the i-th of 32.
    const int mine = begin + warp < end ? (end - begin - warp + kAttnWarps - 1) / kAttnWarps : 0;
    int page_l = -1, pos_l = -1;
    auto fetch = [&](Step<FMT, DH> &s, int i) {
        if ((i & 31) == 0) {
            page_l = pos_l = -1;
            if (i + lane < mine) {
                const int step = begin + warp + (i + lane) * kAttnWarps;
                const int entry = step >> sub_shift;
                const int id = route ? route[entry] : entry;
                if (id >= 0 && id < p.n.table_width) {
                    const int at = (id << p.shift) + ((step & ((1 << sub_shift) - 1)) << 4);
                    if (at < len) {
                        page_l = table[id];
                        if (page_l >= 0 && page_l < p.c.pages) pos_l = at;
                    }
                }
            }
        }
        load_step(s, p, head, __shfl_sync(kFull, page_l, i & 31), __shfl_sync(kFull, pos_l, i & 31), len);
    };

    Step<FMT, DH> cur, nxt;
    if (mine > 0) fetch(nxt, 0);
    for (int i = 0; i < mine; ++i) {
        cur = nxt;
        if (i + 1 < mine) fetch(nxt, i + 1);
        if (cur.pos < 0) continue;

        // S^T: tokens g, g + 8 by rows 2t, 2t + 1
        float s[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
        float kf[2], ev[2];
        uint32_t gf[2] = {0, 0};
        if constexpr (FMT == RR_E4M3) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                kf[h] = power_of_two(cur.ks[h]);
                ev[h] = cur.vs[h] == 255 ? NAN : (float)((int)cur.vs[h] - 127);
            }
        } else {
            const int grp = DH == 128 ? t : t / 2;    // the scale group of this lane's dims
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int kt = top_scale<W::kGroups>(cur.ks[h]);
                kf[h] = has_nan<W::kGroups>(cur.ks[h]) ? NAN : power_of_two(kt);
                const uint32_t f = group_factor((cur.ks[h] >> (8 * grp)) & 255, kt);
                gf[h] = f | f << 16;
                ev[h] = (float)(top_scale<W::kGroups>(cur.vs[h]) - 127 - kGroupLift);
            }
        }
#pragma unroll
        for (int j = 0; j < DH / 16; ++j) {
            uint32_t a[4];
            if constexpr (FMT == RR_E4M3) {
                a[0] = f16x2_of_e4m3(cur.k[0][j] & 0xffffu);
                a[1] = f16x2_of_e4m3(cur.k[1][j] & 0xffffu);
                a[2] = f16x2_of_e4m3(cur.k[0][j] >> 16);
                a[3] = f16x2_of_e4m3(cur.k[1][j] >> 16);
            } else {
                const uint32_t w0 = cur.k[0][j / 2] >> (16 * (j & 1)), w1 = cur.k[1][j / 2] >> (16 * (j & 1));
                a[0] = mul_f16x2(f16x2_of_e2m1(w0 & 255u), gf[0]);
                a[1] = mul_f16x2(f16x2_of_e2m1(w1 & 255u), gf[1]);
                a[2] = mul_f16x2(f16x2_of_e2m1((w0 >> 8) & 255u), gf[0]);
                a[3] = mul_f16x2(f16x2_of_e2m1((w1 >> 8) & 255u), gf[1]);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                uint32_t b0, b1;
                if constexpr (NT <= 2) b0 = qf[nt][j][0], b1 = qf[nt][j][1];
                else query(nt, j, b0, b1);
                mma_f16(s[nt], a, b0, b1);
            }
        }

        // scores in base 2 and their masks; c: token g + 8 (c >> 1), row c & 1
        bool grow = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int key = cur.pos + g + 8 * (c >> 1), r = c & 1;
                float x = s[nt][c] * rowf[nt][r] * kf[c >> 1];
                if (cap) x = p.s2 * tanhf(x);
                if (bias) x -= slope[nt][r] * (float)(pos_r[nt][r] - key - near_r[nt][r]);
                const bool see = key <= pos_r[nt][r];
                if (!see) x = -INFINITY;
                s[nt][c] = x;
                grow = grow || x > m1[nt][r] + kSlack || (see && x - m1[nt][r] + ev[c >> 1] > m2[nt][r] + kSlack);
                if constexpr (FMT == RR_E2M1) {
                    if (see && has_nan<W::kGroups>(cur.vs[c >> 1])) {
#pragma unroll
                        for (int grp = 0; grp < W::kGroups; ++grp)
                            if (((cur.vs[c >> 1] >> (8 * grp)) & 255) == 255)
                                broken |= 1u << ((nt * 2 + r) * W::kGroups + grp);
                    }
                }
            }
        if (__any_sync(kFull, grow)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float a = fmaxf(m1[nt][r], fmaxf(s[nt][r], s[nt][2 + r]));
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) a = fmaxf(a, __shfl_xor_sync(kFull, a, d));
                    const float base = a == -INFINITY ? 0.f : a, down = m1[nt][r] - base;
                    float c = fmaxf(s[nt][r] - base + ev[0], s[nt][2 + r] - base + ev[1]);
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) c = fmaxf(c, __shfl_xor_sync(kFull, c, d));
                    const float was = m2[nt][r] + down;
                    c = fmaxf(c, was);
                    l[nt][r] *= exp2f(down);
                    const float corr = c == -INFINITY ? 1.f : exp2f(was - c);
                    m1[nt][r] = a;
                    m2[nt][r] = c;
#pragma unroll
                    for (int i2 = 0; i2 < kMT; ++i2) {
                        o[i2][nt][r] *= corr;
                        o[i2][nt][2 + r] *= corr;
                    }
                }
        }

        // weights: P^T fragments by transposing 8x8 blocks
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float w[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int r = c & 1;
                const float x = s[nt][c];
                const bool none = x == -INFINITY;
                l[nt][r] += none ? 0.f : exp2f(x - m1[nt][r]);
                w[c] = none ? 0.f : exp2f(x - m1[nt][r] + (ev[c >> 1] - m2[nt][r] + kLift));
            }
            pb[nt][0] = transpose_8x8(pack_f16(w[0], w[1]));
            pb[nt][1] = transpose_8x8(pack_f16(w[2], w[3]));
        }

        // O^T: dims (DH / 8) g + 2 i (rows g) and + 1 (rows g + 8) of tile i
        uint32_t vf[2] = {0, 0};
        if constexpr (FMT == RR_E2M1) {
            const int grp = DH == 128 ? g / 2 : g / 4;
            uint32_t f[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t w = __shfl_sync(kFull, cur.vs[q >> 1], 4 * (2 * t + (q & 1)));
                f[q] = group_factor((w >> (8 * grp)) & 255, top_scale<W::kGroups>(w));
            }
            vf[0] = f[0] | f[1] << 16;
            vf[1] = f[2] | f[3] << 16;
        }
#pragma unroll
        for (int j = 0; j < W::kV; ++j) {
            if constexpr (FMT == RR_E4M3) {
                const uint32_t x0 = __byte_perm(cur.v[0][j], cur.v[1][j], 0x5140), x1 = __byte_perm(cur.v[2][j], cur.v[3][j], 0x5140);
                const uint32_t y0 = __byte_perm(cur.v[0][j], cur.v[1][j], 0x7362), y1 = __byte_perm(cur.v[2][j], cur.v[3][j], 0x7362);
                const uint32_t a[4] = {f16x2_of_e4m3(x0 & 0xffffu), f16x2_of_e4m3(x0 >> 16),
                                       f16x2_of_e4m3(x1 & 0xffffu), f16x2_of_e4m3(x1 >> 16)};
                const uint32_t c[4] = {f16x2_of_e4m3(y0 & 0xffffu), f16x2_of_e4m3(y0 >> 16),
                                       f16x2_of_e4m3(y1 & 0xffffu), f16x2_of_e4m3(y1 >> 16)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma_f16(o[2 * j][nt], a, pb[nt][0], pb[nt][1]);
                    mma_f16(o[2 * j + 1][nt], c, pb[nt][0], pb[nt][1]);
                }
            } else {
                // byte i of a row holds dims 2i (low half) and 2i + 1
                const uint32_t lo0 = (cur.v[0][j] & 0x0f0f0f0fu) | (cur.v[1][j] & 0x0f0f0f0fu) << 4;
                const uint32_t hi0 = ((cur.v[0][j] >> 4) & 0x0f0f0f0fu) | (cur.v[1][j] & 0xf0f0f0f0u);
                const uint32_t lo1 = (cur.v[2][j] & 0x0f0f0f0fu) | (cur.v[3][j] & 0x0f0f0f0fu) << 4;
                const uint32_t hi1 = ((cur.v[2][j] >> 4) & 0x0f0f0f0fu) | (cur.v[3][j] & 0xf0f0f0f0u);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t a[4] = {mul_f16x2(f16x2_of_e2m1((lo0 >> (8 * q)) & 255u), vf[0]),
                                           mul_f16x2(f16x2_of_e2m1((hi0 >> (8 * q)) & 255u), vf[0]),
                                           mul_f16x2(f16x2_of_e2m1((lo1 >> (8 * q)) & 255u), vf[1]),
                                           mul_f16x2(f16x2_of_e2m1((hi1 >> (8 * q)) & 255u), vf[1])};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_f16(o[4 * j + q][nt], a, pb[nt][0], pb[nt][1]);
                }
            }
        }
    }

    // the lanes of a row's 8 tokens: sums, and marks of NaN scales
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[nt][r] += __shfl_xor_sync(kFull, l[nt][r], d);
    if constexpr (FMT == RR_E2M1) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) broken |= __shfl_xor_sync(kFull, broken, d);
        if (broken) {
            const int grp = DH == 128 ? g / 2 : g / 4;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    if (broken >> ((nt * 2 + r) * W::kGroups + grp) & 1)
#pragma unroll
                        for (int i = 0; i < kMT; ++i) o[i][nt][r] = o[i][nt][2 + r] = NAN;
        }
    }

    // the warps' results, joined in pairs: the upper half hands its state to the lower
    for (int half = kAttnWarps / 2; half; half >>= 1) {
        float *at = s_merge + (warp - half) * 32 * kKeep + lane;
        if (warp >= half && warp < 2 * half) {
            int k = 0;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int i = 0; i < kMT; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) at[32 * k++] = o[i][nt][c];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    at[32 * k++] = m1[nt][r];
                    at[32 * k++] = m2[nt][r];
                    at[32 * k++] = l[nt][r];
                }
            }
        }
        __syncthreads();
        if (warp < half) {
            at = s_merge + warp * 32 * kKeep + lane;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float *os = at + 32 * (nt * (kMT * 4 + 6)), *st = os + 32 * kMT * 4;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float a = st[32 * 3 * r], c = st[32 * (3 * r + 1)], ls = st[32 * (3 * r + 2)];
                    const float n1 = fmaxf(m1[nt][r], a), b1 = n1 == -INFINITY ? 0.f : n1;
                    l[nt][r] = l[nt][r] * exp2f(m1[nt][r] - b1) + ls * exp2f(a - b1);
                    const float r0 = m2[nt][r] + (m1[nt][r] - b1), r1 = c + (a - b1), n2 = fmaxf(r0, r1);
                    const float b2 = n2 == -INFINITY ? 0.f : n2;
                    const float f0 = exp2f(r0 - b2), f1 = exp2f(r1 - b2);
                    m1[nt][r] = n1;
                    m2[nt][r] = n2;
#pragma unroll
                    for (int i = 0; i < kMT; ++i) {
                        o[i][nt][r] = o[i][nt][r] * f0 + os[32 * (4 * i + r)] * f1;
                        o[i][nt][2 + r] = o[i][nt][2 + r] * f0 + os[32 * (4 * i + 2 + r)] * f1;
                    }
                }
            }
        }
        __syncthreads();
    }
    if (warp != 0) return;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = row0 + nt * 8 + 2 * t + r;
            if (row >= p.rows) continue;
            const int dim = (DH / 8) * g;
            if (p.splits > 1) {
                float *at = p.part + (((size_t)blockIdx.y * p.splits + blockIdx.x) * p.rows + row) * (DH + kState);
#pragma unroll
                for (int i = 0; i < kMT; ++i)
                    *reinterpret_cast<float2 *>(at + dim + 2 * i) = make_float2(o[i][nt][r], o[i][nt][2 + r]);
                if (g == 0) *reinterpret_cast<float4 *>(at + DH) = make_float4(m1[nt][r], l[nt][r], m2[nt][r], (float)near_r[nt][r]);
            } else {
                const bool none = l[nt][r] == 0.f;
                const float f = none ? 0.f : exp2f(m2[nt][r] - kLift) / l[nt][r];
                const size_t orow = ((size_t)b * p.n.q_tokens + row / p.group) * p.n.q_heads + head * p.group + row % p.group;
                uint32_t *out = static_cast<uint32_t *>(p.a.out) + (orow * DH + dim) / 2;
#pragma unroll
                for (int i = 0; i < kMT; ++i) {
                    const float x = none ? 0.f : o[i][nt][r] * f, y = none ? 0.f : o[i][nt][2 + r] * f;
                    out[i] = p.n.dtype == RR_BF16 ? pack_bf16(x, y) : pack_f16(x, y);
                }
                if (p.a.lse && g == 0)
                    p.a.lse[orow] = none ? -INFINITY
                                         : (m1[nt][r] + log2f(l[nt][r])) * kLn2 - (bias ? slope[nt][r] * kLn2 * (float)near_r[nt][r] : 0.f);
            }
        }
}

// Joins the splits of one row: a warp per row, a lane DH / 32 dims.
template <int DH>
__global__ void __launch_bounds__(128) cached_join_kernel(const __grid_constant__ Cached p, long long rows) {
    constexpr int E = DH / 32;
    const int lane = threadIdx.x & 31;
    const long long r = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (r >= rows) return;
    const long long bh = r / p.rows;
    const int row = (int)(r % p.rows), head = (int)(bh % p.c.heads);
    const long long b = bh / p.c.heads;
    const float *at = p.part + ((size_t)bh * p.splits * p.rows + row) * (DH + kState);
    const size_t stride = (size_t)p.rows * (DH + kState);
    float n1 = -INFINITY, n2 = -INFINITY;
    for (int s = lane; s < p.splits; s += 32) n1 = fmaxf(n1, at[s * stride + DH]);
#pragma unroll
    for (int d = 16; d; d >>= 1) n1 = fmaxf(n1, __shfl_xor_sync(kFull, n1, d));
    const float b1 = n1 == -INFINITY ? 0.f : n1;
    for (int s = lane; s < p.splits; s += 32) n2 = fmaxf(n2, at[s * stride + DH + 2] + (at[s * stride + DH] - b1));
#pragma unroll
    for (int d = 16; d; d >>= 1) n2 = fmaxf(n2, __shfl_xor_sync(kFull, n2, d));
    const float b2 = n2 == -INFINITY ? 0.f : n2;
    float l = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s) {
        const float4 st = *reinterpret_cast<const float4 *>(at + s * stride + DH);
        l += st.y * exp2f(st.x - b1);
        const float f = exp2f(st.z + (st.x - b1) - b2);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += at[s * stride + lane * E + e] * f;
    }
    const bool none = l == 0.f;
    const float f = none ? 0.f : exp2f(n2 - kLift) / l;
    const size_t orow = ((size_t)b * p.n.q_tokens + row / p.group) * p.n.q_heads + head * p.group + row % p.group;
    uint32_t *out = static_cast<uint32_t *>(p.a.out) + (orow * DH + lane * E) / 2;
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        const float x = none ? 0.f : o[e] * f, y = none ? 0.f : o[e + 1] * f;
        out[e / 2] = p.n.dtype == RR_BF16 ? pack_bf16(x, y) : pack_f16(x, y);
    }
    if (p.a.lse && lane == 0) {
        const float near = at[DH + 3];
        p.a.lse[orow] = none ? -INFINITY
                             : (n1 + log2f(l)) * kLn2 - (p.a.slopes ? p.a.slopes[head * p.group + row % p.group] * near : 0.f);
    }
}

bool config_ok(const rr_cache_config *c, const rr_cached_attn_config *n) {
    if (!config_ok(c) || !n) return false;
    if (n->batch < 0 || n->q_tokens < 0 || n->q_heads < 1 || n->q_heads % c->heads != 0) return false;
    if ((long long)n->q_heads / c->heads * n->q_tokens > 256) return false;
    if ((long long)n->batch * c->heads > 65535) return false;
    if (n->dtype != RR_BF16 && n->dtype != RR_F16) return false;
    if (n->table_width < 0 || n->table_stride < (n->table_width > 1 ? n->table_width : 1)) return false;
    if ((long long)n->table_width * c->chunk > 1 << 24) return false;
    if (n->width < 0 || n->route_stride < (n->width > 1 ? n->width : 1) || n->width > 1 << 20) return false;
    if (!(n->scale >= 0.f && n->scale <= 1e30f)) return false;
    if (n->soft_cap != 0.f && !(n->soft_cap >= 1e-3f && n->soft_cap <= 1e30f)) return false;
    for (int64_t x : n->q_stride)
        if (x < 0 || x % 8 != 0 || x > (1ll << 40)) return false;
    return true;
}

int tiles_of(const rr_cache_config *c, const rr_cached_attn_config *n) {
    const int rows = n->q_heads / c->heads * n->q_tokens;
    return rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
}

// CTAs that share a sequence's tokens: enough of them for four waves of two
// CTAs on each of 148 SMs, so that ragged lengths even out, but at least one
// step of 16 tokens for each of a CTA's warps.
int splits_of(const rr_cache_config *c, const rr_cached_attn_config *n, bool route) {
    const long long rows = (long long)(n->q_heads / c->heads) * n->q_tokens;
    const long long blocks = (long long)n->batch * c->heads * ((rows + 8 * tiles_of(c, n) - 1) / (8 * tiles_of(c, n)));
    const long long steps = (long long)(route ? n->width : n->table_width) * (c->chunk / 16);
    if (blocks == 0) return 1;
    const long long want = (4 * 296 + blocks - 1) / blocks, most = steps / kAttnWarps;
    const long long s = want < most ? want : most;
    return s < 1 ? 1 : (int)s;
}

template <int FMT, int DH, int NT>
cudaError_t launch(const Cached &p, cudaStream_t s) {
    constexpr int kKeep = DH / 16 * 4 * NT + 6 * NT;
    const int smem = 8 * NT * (DH + 4) * 2 + 8 * NT * 4 + 16 + kAttnWarps / 2 * 32 * kKeep * 4;
    auto kern = cached_attention_kernel<FMT, DH, NT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const dim3 grid(p.splits, p.n.batch * p.c.heads, (p.rows + 8 * NT - 1) / (8 * NT));
    kern<<<grid, 32 * kAttnWarps, smem, s>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess || p.splits == 1) return e;
    const long long rows = (long long)p.n.batch * p.c.heads * p.rows;
    cached_join_kernel<DH><<<(unsigned)((rows + 3) / 4), 128, 0, s>>>(p, rows);
    return cudaGetLastError();
}

template <int FMT, int DH>
cudaError_t launch_rows(const Cached &p, cudaStream_t s) {
    switch (tiles_of(&p.c, &p.n)) {
        case 1: return launch<FMT, DH, 1>(p, s);
        case 2: return launch<FMT, DH, 2>(p, s);
    }
    return launch<FMT, DH, 4>(p, s);
}

}  // namespace rr_cache

extern "C" size_t rr_cached_attention_workspace_bytes(const rr_cache_config *cfg, const rr_cached_attn_config *attn,
                                                      int32_t routed) {
    using namespace rr_cache;
    if (!config_ok(cfg, attn)) return 0;
    const int splits = splits_of(cfg, attn, routed != 0);
    if (splits == 1) return 0;
    return (size_t)attn->batch * attn->q_heads * attn->q_tokens * splits * (cfg->dh + kState) * sizeof(float);
}

extern "C" rr_status rr_cached_attention(const rr_cache_config *cfg, const rr_cache_pool *pool,
                                         const rr_cached_attn_config *attn, const rr_cached_attn_args *args,
                                         void *workspace, size_t workspace_bytes, void *stream) {
    using namespace rr_cache;
    if (!config_ok(cfg, attn) || !pool || !args) return RR_EINVAL;
    const rr_cached_attn_args &a = *args;
    if (attn->batch == 0 || attn->q_tokens == 0) return RR_OK;
    if (!a.q || !a.out || !aligned(a.q, 16) || !aligned(a.out, 16)) return RR_EINVAL;
    if (cfg->pages > 0 && (!pool->codes || !pool->scales || !aligned(pool->codes, 16) || !aligned(pool->scales, 16)))
        return RR_EINVAL;
    if (!a.seq_lens || !aligned(a.seq_lens, 4) || !aligned(a.route, 4) || !aligned(a.slopes, 4) || !aligned(a.lse, 4))
        return RR_EINVAL;
    if (attn->table_width > 0 && (!a.page_table || !aligned(a.page_table, 4))) return RR_EINVAL;
    const size_t need = rr_cached_attention_workspace_bytes(cfg, attn, a.route != nullptr);
    if (need > 0 && (!workspace || !aligned(workspace, 256))) return RR_EINVAL;
    if (workspace_bytes < need) return RR_ENOMEM;
    Cached p;
    p.c = *cfg;
    p.pool = *pool;
    p.n = *attn;
    p.a = a;
    p.part = static_cast<float *>(workspace);
    p.shift = chunk_shift(cfg->chunk);
    p.group = attn->q_heads / cfg->heads;
    p.rows = p.group * attn->q_tokens;
    p.splits = splits_of(cfg, attn, a.route != nullptr);
    const float scale = attn->scale > 0.f ? attn->scale : 1.0f / sqrtf((float)cfg->dh);
    p.s1 = attn->soft_cap > 0.f ? scale / attn->soft_cap : scale * kLog2e;
    p.s2 = attn->soft_cap * kLog2e;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (cfg->format == RR_E4M3) e = cfg->dh == 64 ? launch_rows<RR_E4M3, 64>(p, s) : launch_rows<RR_E4M3, 128>(p, s);
    else e = cfg->dh == 64 ? launch_rows<RR_E2M1, 64>(p, s) : launch_rows<RR_E2M1, 128>(p, s);
    return e == cudaSuccess ? RR_OK : RR_ECUDA;
}

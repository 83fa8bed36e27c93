// rr_cache.cu -- quantising keys and values into the paged cache, and reading
// them back (declared in include/rr_cache.h).
//
// A warp takes up to 32 tokens, one after another, and of each up to 8 * 32 /
// (dh / 8) (key or value, head) rows, 8 elements a lane, so that a lane has up to
// eight independent 16-byte loads in flight; both kernels are bound by HBM.  The
// places of its tokens are looked up side by side, one by each lane; a warp with
// one token (few tokens: the time to the first load counts) searches cu 32 ways
// at a time.  The group's largest
// magnitude comes from shuffles over its lanes (dh / 8 lanes, or 4 lanes for 32
// elements), its exponent from the magnitude's bits:
//   a = f 2^E, f in [1, 2); M = 1.75 2^8 (e4m3) or 1.5 2^2 (e2m1)
//   least e with a <= M 2^e:  e = E - 8 + (f > 1.75)  or  E - 2 + (f > 1.5)
// x 2^-e is exact in fp32 wherever its rounding can matter (what falls below
// 2^-126 rounds to zero in either format), so each element is rounded once.
//
// Measured on a B200: writing 8 prompts of up to 8191 tokens (8 heads of 128, bf16 to
// e4m3, 266 MB in all) 54 us, 4.9 TB/s; reading 4 histories of up to 32000 tokens
// (e2m1 to bf16, 574 MB) 109 us, 5.3 TB/s; a copy reaches 6.5.  Addresses by fixed
// steps and packed maxima took the write from 84 us and the read from 127, where
// both were bound by instructions; two thirds of the issue slots are still taken.
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "../../include/rr_cache.h"
#include "rr_cache.cuh"

namespace rr_cache {

constexpr int kWarps = 8;

struct Rows {
    rr_cache_config c;
    rr_cache_pool pool;
    rr_cache_rows r;
    void *k, *v;                       // the row arrays (read by the write, written by the read)
    int64_t k_stride[2], v_stride[2];
    int shift;                         // log2(chunk)
    int tokens;                        // per warp, 1 .. 32
    int parts;                         // warps that share the rows of a token
};

// How many of cu[0..n-1] are <= row, by the warp.
__device__ __forceinline__ int count_le(const int32_t *cu, int n, int row) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = n;
    while (lo < hi) {
        const int step = (int)(((unsigned)(hi - lo) + 31u) / 32u);
        const long long at = lo + (long long)(lane + 1) * step - 1;
        const int c = __popc(__ballot_sync(0xffffffffu, at < hi && cu[at < hi ? at : lo] <= row));
        lo += c * step;
        hi = min(hi, lo + step - 1);
    }
    return lo;
}

// The same, by one thread.
__device__ __forceinline__ int count_le_alone(const int32_t *cu, int n, int row) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = lo + (hi - lo) / 2;
        if (cu[mid] <= row) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

// Where a row of the batch lies, n of cu being <= the row: its page (kNoPage: its
// position has none; kNoSequence: it belongs to none) and its place in the page.
constexpr int kNoPage = -1, kNoSequence = -2;
__device__ __forceinline__ int page_of(const Rows &p, int row, int n, int &place) {
    place = 0;
    if (n < 1 || n > p.r.batch) return kNoSequence;
    const long long pos = (long long)p.r.start[n - 1] + row - p.r.cu[n - 1];
    place = (int)(pos & (p.c.chunk - 1));
    const long long entry = pos >> p.shift;
    if (pos < 0 || entry >= p.r.table_width) return kNoPage;
    const int page = p.r.page_table[(size_t)(n - 1) * p.r.table_stride + entry];
    return page >= 0 && page < p.c.pages ? page : kNoPage;
}

// The places of the warp's tokens row0, row0 + kWarps, ..., n of them, lane i that
// of token i.
__device__ __forceinline__ int pages_of(const Rows &p, int row0, int n, int &place) {
    const int lane = threadIdx.x & 31;
    int page = kNoSequence;
    place = 0;
    if (n == 1) {
        page = page_of(p, row0, count_le(p.r.cu, p.r.batch + 1, row0), place);
    } else if (lane < n) {
        const int row = row0 + lane * kWarps;
        page = page_of(p, row, count_le_alone(p.r.cu, p.r.batch + 1, row), place);
    }
    return page;
}

// Eight elements of a row, as loaded.
template <typename T>
struct Eight {
    static constexpr int kUnroll = 8;     // rows a lane holds at once
    uint4 w;
    __device__ __forceinline__ void load(const T *x) { w = __ldcs(reinterpret_cast<const uint4 *>(x)); }
    __device__ __forceinline__ void zero() { w = make_uint4(0u, 0u, 0u, 0u); }
    // bits of the largest magnitude, ordered like it (an infinity or a NaN above all
    // numbers), and the fp32 bits they stand for
    __device__ __forceinline__ unsigned top() const {
        const unsigned m = __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu),
                                    __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
        return max(m & 0xffffu, m >> 16);
    }
    static __device__ __forceinline__ unsigned wide(unsigned top) {
        const uint16_t h = (uint16_t)top;
        return __float_as_uint(rr_attn::Half<T>::up(*reinterpret_cast<const T *>(&h)));
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const T *h = reinterpret_cast<const T *>(&w);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = rr_attn::Half<T>::up(h[i]);
    }
    static __device__ __forceinline__ void store(T *x, const float (&f)[8]) {
        uint4 w;
        uint32_t *u = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = rr_attn::Half<T>::pack(f[2 * i], f[2 * i + 1]);
        *reinterpret_cast<uint4 *>(x) = w;
    }
};
template <>
struct Eight<float> {
    static constexpr int kUnroll = 4;
    float4 a, b;
    __device__ __forceinline__ void load(const float *x) {
        a = __ldcs(reinterpret_cast<const float4 *>(x));
        b = __ldcs(reinterpret_cast<const float4 *>(x) + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ unsigned top() const {
        float f[8];
        get(f);
        unsigned m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
        return m;
    }
    static __device__ __forceinline__ unsigned wide(unsigned top) { return top; }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
    static __device__ __forceinline__ void store(float *x, const float (&f)[8]) {
        reinterpret_cast<float4 *>(x)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4 *>(x)[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
};

// A lane's share of a token: `which` 0 or 1 (key or value) and heads head0,
// head0 + kStep, ..., elements 8 sub ..; all of its addresses are a base and a
// fixed step.
template <int FMT, int DH>
struct Lane {
    static constexpr int kLanes = DH / 8;                     // lanes of a row
    static constexpr int kStep = 16 / kLanes;                 // heads a warp takes at once, key and value of each
    static constexpr int kRowBytes = FMT == RR_E4M3 ? DH : DH / 2;
    static constexpr int kGroups = FMT == RR_E4M3 ? 1 : DH / 32;
    int sub, which, head0;
    __device__ __forceinline__ Lane(int first_head) {
        const int lane = threadIdx.x & 31, r = lane / kLanes;
        sub = lane % kLanes;
        which = r & 1;
        head0 = first_head + (r >> 1);
    }
    // row of the pool
    __device__ __forceinline__ size_t row(const Rows &p, int page, int place) const {
        return (((size_t)page * p.c.heads + head0) * 2 + which) * p.c.chunk + place;
    }
};

template <int FMT, typename T, int DH>
__global__ void __launch_bounds__(32 * kWarps) cache_write_kernel(const __grid_constant__ Rows p) {
    using L = Lane<FMT, DH>;
    constexpr int kGroupLanes = FMT == RR_E4M3 ? L::kLanes : 4, kUnroll = Eight<T>::kUnroll;
    // the block's warps take neighbouring tokens, whose rows are neighbours in the pool
    const int part = blockIdx.x % p.parts;
    const long long first = (long long)(blockIdx.x / p.parts) * p.tokens * kWarps + (threadIdx.x >> 5);
    if (first >= p.r.rows) return;
    const int row0 = (int)first, tokens = min(p.tokens, (p.r.rows - row0 - 1) / kWarps + 1);
    const L l(part * kUnroll * L::kStep);
    const int64_t x_token = l.which ? p.v_stride[0] : p.k_stride[0];
    const int64_t x_step = (l.which ? p.v_stride[1] : p.k_stride[1]) * L::kStep;
    const T *x = static_cast<const T *>(l.which ? p.v : p.k) + row0 * x_token +
                 l.head0 * (l.which ? p.v_stride[1] : p.k_stride[1]) + l.sub * 8;
    const size_t rows_step = (size_t)2 * p.c.chunk * L::kStep;
    int page_l = kNoPage, place_l = 0;
    for (int tok = 0; tok < tokens; ++tok, x += x_token * kWarps) {
        // the first token's rows are on their way while its place is looked up
        Eight<T> x8[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            if (l.head0 + i * L::kStep < p.c.heads) x8[i].load(x + i * x_step);
            else x8[i].zero();
        }
        if (tok == 0) page_l = pages_of(p, row0, tokens, place_l);
        const int page = __shfl_sync(0xffffffffu, page_l, tok), place = __shfl_sync(0xffffffffu, place_l, tok);
        if (page < 0) continue;
        const size_t at = l.row(p, page, place);
        unsigned char *codes = static_cast<unsigned char *>(p.pool.codes) + at * L::kRowBytes + l.sub * (L::kRowBytes / L::kLanes);
        unsigned char *scales = static_cast<unsigned char *>(p.pool.scales) + at * L::kGroups + (FMT == RR_E4M3 ? 0 : l.sub / 4);
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            if (part * kUnroll * L::kStep + i * L::kStep >= p.c.heads) break;      // the same for the whole warp
            unsigned a = x8[i].top();
#pragma unroll
            for (int d = 1; d < kGroupLanes; d <<= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, d));
            a = Eight<T>::wide(a);
            const bool finite = a < 0x7f800000u;
            const unsigned mant = a & 0x7fffffu;
            int e = (int)(a >> 23) - 127;
            e = FMT == RR_E4M3 ? e - 8 + (mant > 0x600000u) : e - 2 + (mant > 0x400000u);
            e = max(e, -127);
            const float inv = __uint_as_float((unsigned)(127 - e) << 23);   // 2^-e; e <= 126
            const bool mine = l.head0 + i * L::kStep < p.c.heads;
            float f[8];
            x8[i].get(f);
            if constexpr (FMT == RR_E4M3) {
                uint32_t h[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    h[j] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * j] * inv, f[2 * j + 1] * inv), __NV_SATFINITE,
                                                    __NV_E4M3);
                uint2 w = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
                if (!finite) w = make_uint2(0u, 0u);
                if (mine) *reinterpret_cast<uint2 *>(codes + i * rows_step * L::kRowBytes) = w;
            } else {
                uint32_t w = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w |= (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(f[2 * j] * inv, f[2 * j + 1] * inv), __NV_E2M1,
                                                            cudaRoundNearest)
                         << (8 * j);
                if (!finite) w = 0;
                if (mine) *reinterpret_cast<uint32_t *>(codes + i * rows_step * L::kRowBytes) = w;
            }
            if (mine && l.sub % kGroupLanes == 0)
                scales[i * rows_step * L::kGroups] = finite ? (unsigned char)(e + 127) : 255;
        }
    }
}

template <int FMT, typename T, int DH>
__global__ void __launch_bounds__(32 * kWarps) cache_read_kernel(const __grid_constant__ Rows p) {
    using L = Lane<FMT, DH>;
    constexpr int kUnroll = Eight<T>::kUnroll;
    const int part = blockIdx.x % p.parts;
    const long long first = (long long)(blockIdx.x / p.parts) * p.tokens * kWarps + (threadIdx.x >> 5);
    if (first >= p.r.rows) return;
    const int row0 = (int)first, tokens = min(p.tokens, (p.r.rows - row0 - 1) / kWarps + 1);
    const L l(part * kUnroll * L::kStep);
    T *out = static_cast<T *>(l.which ? p.v : p.k);
    const int64_t x_token = l.which ? p.v_stride[0] : p.k_stride[0];
    const int64_t x_step = (l.which ? p.v_stride[1] : p.k_stride[1]) * L::kStep;
    T *x = out + row0 * x_token + l.head0 * (l.which ? p.v_stride[1] : p.k_stride[1]) + l.sub * 8;
    const size_t rows_step = (size_t)2 * p.c.chunk * L::kStep;
    const int heads = out ? p.c.heads : 0;      // nothing to read for an output that is not asked for
    int place_l;
    const int page_l = pages_of(p, row0, tokens, place_l);
    for (int tok = 0; tok < tokens; ++tok, x += x_token * kWarps) {
        const int page = __shfl_sync(0xffffffffu, page_l, tok), place = __shfl_sync(0xffffffffu, place_l, tok);
        if (page == kNoSequence) continue;
        const size_t at = l.row(p, max(page, 0), place);
        const unsigned char *codes = static_cast<const unsigned char *>(p.pool.codes) + at * L::kRowBytes + l.sub * (L::kRowBytes / L::kLanes);
        const unsigned char *scales = static_cast<const unsigned char *>(p.pool.scales) + at * L::kGroups + (FMT == RR_E4M3 ? 0 : l.sub / 4);
        uint2 code[kUnroll];
        unsigned scale[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            code[i] = make_uint2(0u, 0u);
            scale[i] = 0;
            if (page >= 0 && l.head0 + i * L::kStep < heads) {
                if constexpr (FMT == RR_E4M3) code[i] = __ldcs(reinterpret_cast<const uint2 *>(codes + i * rows_step * L::kRowBytes));
                else code[i].x = __ldcs(reinterpret_cast<const uint32_t *>(codes + i * rows_step * L::kRowBytes));
                scale[i] = __ldg(scales + i * rows_step * L::kGroups);
            }
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            if (l.head0 + i * L::kStep >= heads) continue;
            const float two = power_of_two(scale[i]);
            float f[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                __half2_raw h;
                if constexpr (FMT == RR_E4M3) {
                    const uint32_t w = j < 2 ? code[i].x : code[i].y;
                    h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * (j & 1))), __NV_E4M3);
                } else {
                    h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(code[i].x >> (8 * j)), __NV_E2M1);
                }
                const float2 y = __half22float2(__half2(h));
                f[2 * j] = y.x * two;
                f[2 * j + 1] = y.y * two;
            }
            Eight<T>::store(x + i * x_step, f);
        }
    }
}

template <int FMT, typename T>
cudaError_t launch(const Rows &p, bool write, unsigned blocks, cudaStream_t s) {
    if (p.c.dh == 64) {
        if (write) cache_write_kernel<FMT, T, 64><<<blocks, 32 * kWarps, 0, s>>>(p);
        else cache_read_kernel<FMT, T, 64><<<blocks, 32 * kWarps, 0, s>>>(p);
    } else {
        if (write) cache_write_kernel<FMT, T, 128><<<blocks, 32 * kWarps, 0, s>>>(p);
        else cache_read_kernel<FMT, T, 128><<<blocks, 32 * kWarps, 0, s>>>(p);
    }
    return cudaGetLastError();
}

template <int FMT>
cudaError_t launch_type(const Rows &p, int dtype, bool write, unsigned blocks, cudaStream_t s) {
    if (dtype == RR_F32) return launch<FMT, float>(p, write, blocks, s);
    if (dtype == RR_BF16) return launch<FMT, __nv_bfloat16>(p, write, blocks, s);
    return launch<FMT, __half>(p, write, blocks, s);
}

rr_status run(const rr_cache_config *cfg, const rr_cache_pool *pool, const rr_cache_rows *rows, void *k,
              const int64_t *k_stride, void *v, const int64_t *v_stride, int32_t dtype, bool write, void *stream) {
    if (!config_ok(cfg) || !pool || !rows) return RR_EINVAL;
    if (dtype != RR_F32 && dtype != RR_BF16 && dtype != RR_F16) return RR_EINVAL;
    if (rows->batch < 0 || rows->batch == 0x7fffffff || rows->rows < 0 || rows->table_width < 0 ||
        rows->table_stride < (rows->table_width > 1 ? rows->table_width : 1))
        return RR_EINVAL;
    const int64_t size = dtype == RR_F32 ? 4 : 2;
    const void *ptr[2] = {k, v};
    const int64_t *stride[2] = {k_stride, v_stride};
    for (int i = 0; i < 2; ++i) {
        if (!ptr[i]) {
            if (write && rows->rows > 0) return RR_EINVAL;
            continue;
        }
        if (!stride[i] || !aligned(ptr[i], 16)) return RR_EINVAL;
        for (int j = 0; j < 2; ++j) {
            const int64_t x = stride[i][j];
            if ((j == 0 ? rows->rows : cfg->heads) <= 1) continue;
            if (x < 0 || x > (1ll << 40) || x * size % 16 != 0) return RR_EINVAL;
        }
        const int32_t sizes[2] = {rows->rows, cfg->heads};
        if (!write && !rr_attn::rows_apart(sizes, stride[i], 2, cfg->dh)) return RR_EINVAL;
    }
    if (rows->rows == 0 || rows->batch == 0 || (!k && !v)) return RR_OK;
    if (cfg->pages > 0 && (!pool->codes || !pool->scales || !aligned(pool->codes, 16) || !aligned(pool->scales, 16)))
        return RR_EINVAL;
    if (!rows->cu || !rows->start || !aligned(rows->cu, 4) || !aligned(rows->start, 4)) return RR_EINVAL;
    if (rows->table_width > 0 && (!rows->page_table || !aligned(rows->page_table, 4))) return RR_EINVAL;
    Rows p;
    p.c = *cfg;
    p.pool = *pool;
    p.r = *rows;
    p.k = k;
    p.v = v;
    for (int j = 0; j < 2; ++j) {
        const bool counts = (j == 0 ? rows->rows : cfg->heads) > 1;
        p.k_stride[j] = k && counts ? k_stride[j] : 0;
        p.v_stride[j] = v && counts ? v_stride[j] : 0;
    }
    p.shift = chunk_shift(cfg->chunk);
    const int per_warp = (dtype == RR_F32 ? Eight<float>::kUnroll : Eight<__half>::kUnroll) * 128 / cfg->dh;   // heads
    p.parts = (cfg->heads + per_warp - 1) / per_warp;
    // as many tokens a warp as leave two waves of 32 warps on each SM
    const long long tokens = (long long)rows->rows * p.parts / (148 * 64);
    p.tokens = (int)(tokens < 1 ? 1 : tokens < 32 ? tokens : 32);
    const long long blocks = ((long long)rows->rows + p.tokens * kWarps - 1) / (p.tokens * kWarps) * p.parts;
    if (blocks > 0x7fffffffLL) return RR_EINVAL;
    const unsigned grid = (unsigned)blocks;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = cfg->format == RR_E4M3 ? launch_type<RR_E4M3>(p, dtype, write, grid, s)
                                                 : launch_type<RR_E2M1>(p, dtype, write, grid, s);
    return e == cudaSuccess ? RR_OK : RR_ECUDA;
}

}  // namespace rr_cache

extern "C" size_t rr_cache_codes_bytes(const rr_cache_config *cfg) {
    if (!rr_cache::config_ok(cfg)) return 0;
    return (size_t)cfg->pages * cfg->heads * 2 * cfg->chunk * (cfg->format == RR_E4M3 ? cfg->dh : cfg->dh / 2);
}

extern "C" size_t rr_cache_scales_bytes(const rr_cache_config *cfg) {
    if (!rr_cache::config_ok(cfg)) return 0;
    return (size_t)cfg->pages * cfg->heads * 2 * cfg->chunk * (cfg->format == RR_E4M3 ? 1 : cfg->dh / 32);
}

extern "C" rr_status rr_cache_write(const rr_cache_config *cfg, const rr_cache_pool *pool, const rr_cache_rows *rows,
                                    const void *d_k, const int64_t k_stride[2], const void *d_v,
                                    const int64_t v_stride[2], int32_t dtype, void *stream) {
    return rr_cache::run(cfg, pool, rows, const_cast<void *>(d_k), k_stride, const_cast<void *>(d_v), v_stride, dtype,
                         true, stream);
}

extern "C" rr_status rr_cache_read(const rr_cache_config *cfg, const rr_cache_pool *pool, const rr_cache_rows *rows,
                                   void *d_k, const int64_t k_stride[2], void *d_v, const int64_t v_stride[2],
                                   int32_t dtype, void *stream) {
    return rr_cache::run(cfg, pool, rows, d_k, k_stride, d_v, v_stride, dtype, false, stream);
}

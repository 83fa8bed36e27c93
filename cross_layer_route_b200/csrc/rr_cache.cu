// rr_cache.cu -- quantising keys and values into the paged cache, and reading
// them back (declared in include/rr_cache.h).
//
// A warp takes one token and up to 4 * 32 / (dh / 8) of its (key or value, head)
// rows, 8 elements a lane, so that a lane has up to four independent 16-byte
// loads in flight; both kernels are bound by HBM.  The group's largest
// magnitude comes from shuffles over its lanes (dh / 8 lanes, or 4 lanes for 32
// elements), its exponent from the magnitude's bits:
//   a = f 2^E, f in [1, 2); M = 1.75 2^8 (e4m3) or 1.5 2^2 (e2m1)
//   least e with a <= M 2^e:  e = E - 8 + (f > 1.75)  or  E - 2 + (f > 1.5)
// x 2^-e is exact in fp32 wherever its rounding can matter (what falls below
// 2^-126 rounds to zero in either format), so each element is rounded once.
// The token's sequence is found by a 32-way search over cu by the whole warp.
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "../../include/rr_cache.h"
#include "rr_cache.cuh"

namespace rr_cache {

constexpr int kWarps = 8;
constexpr int kUnroll = 4;

struct Rows {
    rr_cache_config c;
    rr_cache_pool pool;
    rr_cache_rows r;
    void *k, *v;                       // the row arrays (read by the write, written by the read)
    int64_t k_stride[2], v_stride[2];
    int shift;                         // log2(chunk)
    int parts;                         // warps per token
    long long tasks;                   // rows * parts
};

// How many of cu[0..n-1] are <= row, by the warp.
__device__ __forceinline__ int count_le(const int32_t *cu, int n, int row) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = n;
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32;
        const long long at = lo + (long long)(lane + 1) * step - 1;
        const int c = __popc(__ballot_sync(0xffffffffu, at < hi && cu[at < hi ? at : lo] <= row));
        lo += c * step;
        hi = min(hi, lo + step - 1);
    }
    return lo;
}

// Where a row of the batch lies: false if it belongs to no sequence; page < 0
// if its position has no page.
__device__ __forceinline__ bool place_of(const Rows &p, int row, int &page, int &place) {
    const int n = count_le(p.r.cu, p.r.batch + 1, row);
    if (n < 1 || n > p.r.batch) return false;
    const long long pos = (long long)p.r.start[n - 1] + row - p.r.cu[n - 1];
    page = -1;
    place = (int)(pos & (p.c.chunk - 1));
    const long long entry = pos >> p.shift;
    if (pos >= 0 && entry < p.r.table_width) {
        page = p.r.page_table[(size_t)(n - 1) * p.r.table_stride + entry];
        if (page >= p.c.pages) page = -1;
    }
    return true;
}

template <typename T>
struct Eight;   // 8 elements of a row, as fp32
template <>
struct Eight<float> {
    static __device__ __forceinline__ void load(const float *x, float (&f)[8]) {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(x)), b = __ldg(reinterpret_cast<const float4 *>(x) + 1);
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
    static __device__ __forceinline__ void store(float *x, const float (&f)[8]) {
        reinterpret_cast<float4 *>(x)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4 *>(x)[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
};
template <typename T>
struct Eight {
    static __device__ __forceinline__ void load(const T *x, float (&f)[8]) {
        const uint4 w = __ldg(reinterpret_cast<const uint4 *>(x));
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

template <int FMT, typename T, int DH>
__global__ void __launch_bounds__(32 * kWarps) cache_write_kernel(const __grid_constant__ Rows p) {
    constexpr int kLanes = DH / 8, kRows = 32 / kLanes;
    constexpr int kGroupLanes = FMT == RR_E4M3 ? kLanes : 4;
    const int lane = threadIdx.x & 31, sub = lane % kLanes;
    for (long long task = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); task < p.tasks;
         task += (long long)gridDim.x * kWarps) {
        const int row = (int)(task / p.parts), part = (int)(task % p.parts);
        int page, place;
        if (!place_of(p, row, page, place) || page < 0) continue;
        float f[kUnroll][8];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int pair = (part * kUnroll + i) * kRows + lane / kLanes;   // keys' heads, then values'
            if (pair < 2 * p.c.heads) {
                const int which = pair >= p.c.heads, head = pair - which * p.c.heads;
                const T *x = which ? static_cast<const T *>(p.v) + row * p.v_stride[0] + head * p.v_stride[1]
                                   : static_cast<const T *>(p.k) + row * p.k_stride[0] + head * p.k_stride[1];
                Eight<T>::load(x + sub * 8, f[i]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) f[i][e] = 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            unsigned a = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) a = max(a, __float_as_uint(f[i][e]) & 0x7fffffffu);
#pragma unroll
            for (int d = 1; d < kGroupLanes; d <<= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, d));
            const bool finite = a < 0x7f800000u;
            const unsigned mant = a & 0x7fffffu;
            int e = (int)(a >> 23) - 127;
            e = FMT == RR_E4M3 ? e - 8 + (mant > 0x600000u) : e - 2 + (mant > 0x400000u);
            e = max(e, -127);
            const float inv = __uint_as_float((unsigned)(127 - e) << 23);   // 2^-e; e <= 126
            const int pair = (part * kUnroll + i) * kRows + lane / kLanes;
            if (pair >= 2 * p.c.heads) continue;
            const int which = pair >= p.c.heads, head = pair - which * p.c.heads;
            const size_t at = (((size_t)page * p.c.heads + head) * 2 + which) * p.c.chunk + place;
            const unsigned char byte = finite ? (unsigned char)(e + 127) : 255;
            if constexpr (FMT == RR_E4M3) {
                uint2 w = make_uint2(0u, 0u);
                if (finite) {
                    uint16_t h[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        h[j] = __nv_cvt_float2_to_fp8x2(make_float2(f[i][2 * j] * inv, f[i][2 * j + 1] * inv),
                                                        __NV_SATFINITE, __NV_E4M3);
                    w = make_uint2(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16);
                }
                *reinterpret_cast<uint2 *>(static_cast<unsigned char *>(p.pool.codes) + at * DH + sub * 8) = w;
                if (sub == 0) static_cast<unsigned char *>(p.pool.scales)[at] = byte;
            } else {
                uint32_t w = 0;
                if (finite) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        w |= (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(f[i][2 * j] * inv, f[i][2 * j + 1] * inv),
                                                                __NV_E2M1, cudaRoundNearest)
                             << (8 * j);
                }
                *reinterpret_cast<uint32_t *>(static_cast<unsigned char *>(p.pool.codes) + at * (DH / 2) + sub * 4) = w;
                if (sub % 4 == 0) static_cast<unsigned char *>(p.pool.scales)[at * (DH / 32) + sub / 4] = byte;
            }
        }
    }
}

template <int FMT, typename T, int DH>
__global__ void __launch_bounds__(32 * kWarps) cache_read_kernel(const __grid_constant__ Rows p) {
    constexpr int kLanes = DH / 8, kRows = 32 / kLanes;
    const int lane = threadIdx.x & 31, sub = lane % kLanes;
    for (long long task = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); task < p.tasks;
         task += (long long)gridDim.x * kWarps) {
        const int row = (int)(task / p.parts), part = (int)(task % p.parts);
        int page, place;
        if (!place_of(p, row, page, place)) continue;
        uint2 code[kUnroll];
        unsigned scale[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int pair = (part * kUnroll + i) * kRows + lane / kLanes;
            code[i] = make_uint2(0u, 0u);
            scale[i] = 0;
            if (pair >= 2 * p.c.heads || page < 0) continue;
            const int which = pair >= p.c.heads, head = pair - which * p.c.heads;
            const size_t at = (((size_t)page * p.c.heads + head) * 2 + which) * p.c.chunk + place;
            const unsigned char *codes = static_cast<const unsigned char *>(p.pool.codes);
            const unsigned char *scales = static_cast<const unsigned char *>(p.pool.scales);
            if constexpr (FMT == RR_E4M3) {
                code[i] = __ldg(reinterpret_cast<const uint2 *>(codes + at * DH + sub * 8));
                scale[i] = __ldg(scales + at);
            } else {
                code[i].x = __ldg(reinterpret_cast<const uint32_t *>(codes + at * (DH / 2) + sub * 4));
                scale[i] = __ldg(scales + at * (DH / 32) + sub / 4);
            }
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int pair = (part * kUnroll + i) * kRows + lane / kLanes;
            if (pair >= 2 * p.c.heads) continue;
            const int which = pair >= p.c.heads, head = pair - which * p.c.heads;
            T *x = static_cast<T *>(which ? p.v : p.k);
            if (!x) continue;
            x += which ? row * p.v_stride[0] + head * p.v_stride[1] : row * p.k_stride[0] + head * p.k_stride[1];
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
            Eight<T>::store(x + sub * 8, f);
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
            if (x < 0 || x > (1ll << 40) || x * size % 16 != 0) return RR_EINVAL;
            if (!write && x < cfg->dh && (j == 0 ? rows->rows : cfg->heads) > 1) return RR_EINVAL;
        }
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
        p.k_stride[j] = k ? k_stride[j] : 0;
        p.v_stride[j] = v ? v_stride[j] : 0;
    }
    p.shift = chunk_shift(cfg->chunk);
    const int per_warp = kUnroll * 32 / (cfg->dh / 8);
    p.parts = (int)((2ll * cfg->heads + per_warp - 1) / per_warp);
    p.tasks = (long long)rows->rows * p.parts;
    const long long blocks = (p.tasks + kWarps - 1) / kWarps;
    const unsigned grid = (unsigned)(blocks < 0x7fffffffLL ? blocks : 0x7fffffffLL);
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

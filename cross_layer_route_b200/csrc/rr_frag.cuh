// rr_frag.cuh -- warp-level matrix fragments and asynchronous copies shared by
// the attention kernels on mma.sync.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace rr_attn {

constexpr int kMaxWidth = 1024;     // route entries read per query chunk
constexpr unsigned kFull = 0xffffffffu;

// Lets a kernel have `bytes` of dynamic shared memory, on the current device, the
// first time it is asked for there (`done`: a bit for each of 64 devices).
inline cudaError_t allow_smem(const void *kernel, int bytes, std::atomic<uint64_t> &done) {
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const uint64_t bit = device < 64 ? 1ull << device : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Whether the rows (of `row` elements) of an output lie apart: by dimensions (at most
// 3, strides >= 0) from the smallest stride up, each steps over all that the ones
// before it span.  A size of one counts nothing.
inline bool rows_apart(const int32_t *size, const int64_t *stride, int dims, int64_t row) {
    bool used[3] = {};
    __int128 span = row;
    for (int n = 0; n < dims; ++n) {
        int least = -1;
        for (int i = 0; i < dims; ++i)
            if (!used[i] && size[i] > 1 && (least < 0 || stride[i] < stride[least])) least = i;
        if (least < 0) break;
        if (stride[least] < span) return false;
        used[least] = true;
        span += (__int128)(size[least] - 1) * stride[least];
    }
    return true;
}

__device__ __forceinline__ uint32_t smem_u32(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;\n" ::: "memory");
}

// Waits until at most one committed group is still in flight.
__device__ __forceinline__ void cp_async_wait_one() {
    asm volatile("cp.async.wait_group 1;\n" ::: "memory");
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t &r0, uint32_t &r1, uint32_t &r2,
                                            uint32_t &r3) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr));
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t &r0, uint32_t &r1, uint32_t &r2,
                                                  uint32_t &r3) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr));
}

// d += a (16x16 bf16, row) * b (16x8 bf16, col), fp32 accumulate.
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two floats as a bf16 pair, `lo` in the low half (round to nearest even).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
}

// The same with 16-byte copies that a zero `bytes` turns into zero fill.
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
}

// 2^x by the special function unit (relative error 2^-22; results below 2^-126 are zero).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
    return d;
}
__device__ __forceinline__ void unpack2(uint64_t d, float &x, float &y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(d));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// tanh z.  Up to |z| = 1 z P(z^2), P the polynomial of degree 6 of least largest
// relative error (5e-8, by exchange in double); beyond that 1 - 2 / (1 + e^2z),
// where the difference loses no bit.  Relative error below 2^-21 throughout, so a
// cap far above the scores leaves them as they are.
__device__ __forceinline__ float tanh_within_one(float z) {
    const float y = z * z;
    float s = fmaf(y, 0.00104102263f, -0.00620337910f);
    s = fmaf(y, s, 0.0202899804f);
    s = fmaf(y, s, -0.0534570296f);
    s = fmaf(y, s, 0.133252041f);
    s = fmaf(y, s, -0.333328392f);
    s = fmaf(y, s, 0.99999995f);
    return z * s;
}
__device__ __forceinline__ float tanh_f32(float z) {
    const float far = 1.f - __fdividef(2.f, 1.f + ex2(z * 2.8853900817779268f));
    return fabsf(z) < 1.f ? tanh_within_one(z) : far;
}

// tanh(x s1) of two scores with |x s1| < 1: tanh_within_one, two at a time.
__device__ __forceinline__ void tanh_pair(float *x, float s1) {
    const uint64_t z = mul2(pack2(x[0], x[1]), pack2(s1, s1)), y = mul2(z, z);
    uint64_t s = fma2(y, pack2(0.00104102263f, 0.00104102263f), pack2(-0.00620337910f, -0.00620337910f));
    s = fma2(y, s, pack2(0.0202899804f, 0.0202899804f));
    s = fma2(y, s, pack2(-0.0534570296f, -0.0534570296f));
    s = fma2(y, s, pack2(0.133252041f, 0.133252041f));
    s = fma2(y, s, pack2(-0.333328392f, -0.333328392f));
    s = fma2(y, s, pack2(0.99999995f, 0.99999995f));
    unpack2(mul2(z, s), x[0], x[1]);
}

// The two 16-bit types of the operators that take either.
template <typename T>
struct Half;
template <>
struct Half<__nv_bfloat16> {
    static constexpr bool kBf16 = true;
    static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        mma_bf16(d, a, b0, b1);
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return pack_bf16(lo, hi); }
    static __device__ __forceinline__ uint32_t pack_mean(float lo, float hi) { return pack_bf16(lo, hi); }
    static __device__ __forceinline__ float up(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __forceinline__ __nv_bfloat16 down(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Half<__half> {
    static constexpr bool kBf16 = false;
    static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        mma_f16(d, a, b0, b1);
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return pack_f16(lo, hi); }
    // Means of finite values, which are at most 65504.  Weights rounded up by 2^-11 at most
    // can carry them past 65520, from where on f16 has infinities.  A NaN stays one.  (In
    // bf16 the sums of such values are infinite before.)
    static __device__ __forceinline__ uint32_t pack_mean(float lo, float hi) {
        const __half2 top = __float2half2_rn(65504.f);
        const __half2 x = __hmax2_nan(__hmin2_nan(__floats2half2_rn(lo, hi), top), __hneg2(top));
        return *reinterpret_cast<const uint32_t *>(&x);
    }
    static __device__ __forceinline__ float up(__half x) { return __half2float(x); }
    static __device__ __forceinline__ __half down(float x) { return __float2half_rn(x); }
};

}  // namespace rr_attn

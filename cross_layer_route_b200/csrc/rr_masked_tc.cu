// rr_masked_tc.cu -- masked attention over a route on tcgen05 (declared in
// include/rr_attention.h; the masks and the list of key chunks in rr_masked.cuh).
//
// One CTA = up to 256 rows of a unit in two tiles of 128 (the query heads that
// share a key head times the chunk's tokens), so that a 128-key tile of K and V
// fetched from L2 serves 256 rows: at 4 dh flops a pair that is what L2 can feed.
//   warps 0-3, 4-7  softmax of tile 0 and 1, a thread per row (TMEM lane): S is
//                   read from TMEM into registers, scores and masks are applied,
//                   P goes back to TMEM in 16 bits over the first half of S;
//   warp 8          issues tcgen05.mma: S = Q K^T (both operands in shared
//                   memory), O += P V (P from TMEM, V as it lies in memory, an
//                   N-major operand);
//   warp 9          TMA producer: key chunks gathered by the route into tiles of
//                   128 keys, K and V in turn through a ring of stages.
// While one tile's softmax runs, the tensor cores work for the other.  TMEM: two
// S tiles and two O tiles of 128 columns.  P aliases S: the product that reads it
// is issued before the one that writes the next S, and they execute in order.
//
// The running maximum moves only when it would grow by more than 2^8 (in the
// weights), so O is seldom rescaled: the weights then reach 2^8, times the 2^7
// that keeps small ones away from f16's subnormals, and all sums are fp32.
//
// Every wait is bounded; when one runs out the CTA stops, drains its copies,
// waits for its last MMA, frees TMEM and leaves its rows NaN.
#include "rr_masked.cuh"
#include "rr_tc.cuh"

namespace rr_masked {

using namespace rr::tc;

constexpr int kTileRows = 128;
constexpr int kTileKeys = 128;
constexpr int kTiles = 2;
constexpr int kSoftWarps = 4 * kTiles;
constexpr int kTcThreads = 32 * (kSoftWarps + 4);   // two warps of the last group are idle
// Registers: launched with 168 a thread (384 threads: 64512 in all), then the two
// softmax groups take 224 and the third keeps 56: 2 * 128 * 224 + 128 * 56 = 64512.
constexpr int kSoftRegs = 224, kOtherRegs = 56;
constexpr float kSlack = 8.f;     // growth of the maximum that is let pass
constexpr float kLift = 7.f;      // weights are 2^7 at the maximum
constexpr int kSubBytes = kTileRows * 128;    // 128 rows of 64 elements

template <int DH>
struct TcShape {
    static constexpr int kSubs = DH / 64;
    static constexpr int kTileBytes = kSubs * kSubBytes;          // a Q, K or V tile
    static constexpr int kStages = DH == 128 ? 4 : 8;
    static constexpr int kHead = kMaxWidth * 4 + 16;
    static constexpr int kBars = 2 * kStages + 4 * kTiles + 2;
    static constexpr int kMisc = 256;
    static constexpr int kSmem = 1024 + kHead + kBars * 8 + kMisc + (kTiles + kStages) * kTileBytes;
};

// fp32 accumulator; A K-major; B K-major (keys) or N-major (values).
template <typename T>
__host__ __device__ constexpr uint32_t idesc_of(int n, bool b_n_major) {
    const uint32_t type = Half<T>::kBf16 ? 1u : 0u;
    return (1u << 4) | (type << 7) | (type << 10) | ((b_n_major ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(kTileRows >> 4) << 24);
}

// N-major operand in 128-byte swizzled rows of 64 N elements: rows of a group of
// 8 keys 128 bytes apart, groups 1024, the next 64 N elements kSubBytes on.
__device__ __forceinline__ uint64_t n_major_desc(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(kSubBytes >> 4) << 16) | ((uint64_t)(1024u >> 4) << 32) |
           ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}

__device__ __forceinline__ void tma_load_4d_elect(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1,
                                                  int c2, int c3) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(saddr(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

__device__ __forceinline__ void tma_store_4d(const CUtensorMap *map, uint32_t src, int c0, int c1, int c2, int c3) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
                 : "memory");
}

// Tensor maps of the operands; axes: see tensor_map.
struct Maps {
    CUtensorMap q, k, v, out;
    int axes[4];
};

// 32 columns of this thread's TMEM lane; the values may be used after wait_ld32.
__device__ __forceinline__ void ld32(uint32_t taddr, float *v) {
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
        "%30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
// Waits for the loads before it; names the registers, so that no use moves ahead.
__device__ __forceinline__ void wait_ld32(float *v) {
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                   "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void st32(uint32_t taddr, const float *v) {
    const uint32_t *r = reinterpret_cast<const uint32_t *>(v);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// (NaN if any of them is)
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <typename T, int DH>
__global__ void __launch_bounds__(kTcThreads, 1)
masked_attention_tc_kernel(const __grid_constant__ Masked p, const __grid_constant__ Maps maps) {
    using S = TcShape<DH>;
    extern __shared__ unsigned char raw[];
    unsigned char *smem = align_smem_1024(raw);
    unsigned char *q_s = smem, *kv_s = smem + kTiles * S::kTileBytes;
    int32_t *s_list = reinterpret_cast<int32_t *>(kv_s + S::kStages * S::kTileBytes);
    int32_t *s_n = s_list + kMaxWidth;
    uint64_t *full = reinterpret_cast<uint64_t *>(s_list + kMaxWidth + 4);
    uint64_t *empty = full + S::kStages, *s_full = empty + S::kStages, *p_ready = s_full + kTiles;
    uint64_t *o_done = p_ready + 2 * kTiles, *q_ready = o_done + kTiles, *mma_done = q_ready + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Unit u = unit_of(p, blockIdx.x);
    const int rows = p.group << p.shift, row0 = u.tile * kTiles * kTileRows;
    const int tiles = min(kTiles, (rows - row0 + kTileRows - 1) / kTileRows);
    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int t = 0; t < kTiles; ++t) {
            mbar_init(&s_full[t], 1);
            mbar_init(&p_ready[2 * t], 4);
            mbar_init(&p_ready[2 * t + 1], 4);
            mbar_init(&o_done[t], 1);
        }
        mbar_init(q_ready, 1);
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kSoftWarps) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tmem_slot)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    const int n_list = build_list(p, u, s_list, s_n);    // ends with a barrier
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int slots = n_list << p.shift, n = (slots + kTileKeys - 1) / kTileKeys;

    if (warp < kSoftWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        if ((warp >> 2) < tiles) {
            // ---- softmax: one row per thread ----
            const int t = warp >> 2;
            const int row = row0 + threadIdx.x;              // of the unit
            const bool in_unit = row < rows;
            const int head = u.route_head * p.group + (in_unit ? row >> p.shift : 0), tok = row & (p.c.chunk - 1);
            const bool valid = in_unit && tok < u.tokens;
            const int64_t token = ((int64_t)u.i << p.shift) + tok;
            const int pos = u.p_first + tok;
            const bool docs = p.a.doc_q != nullptr, bias = p.a.slopes != nullptr, cap = p.c.soft_cap > 0.f;
            const int doc = docs && valid ? p.a.doc_q[(size_t)u.b * p.c.nq_tokens + token] : -1;
            const int32_t *doc_k = docs ? p.a.doc_k + (size_t)u.b * p.c.nk_tokens : nullptr;
            // keys below this are in sight; none to a row without a document
            const int limit = docs && doc < 0 ? 0 : min(p.c.nk_tokens, p.c.causal ? max(pos + 1, u.prefix) : p.c.nk_tokens);
            const float slope = bias ? p.a.slopes[head] * kLog2e : 0.f;
            int near = 0;
            if (bias) {
                near = nearest(p, u, s_list, n_list, pos, doc, 0, 1);
                if (near == INT_MAX) near = 0;
            }
            const uint32_t lanes = (uint32_t)(warp & 3) << 21;    // TMEM lane 32 (warp mod 4), in bits 16-31
            const uint32_t s_at = tmem + lanes + t * 128, o_at = tmem + lanes + 256 + t * 128;
            float m = -INFINITY, l = 0.f;
            bool ok = true;
            for (int j = 0; j < n; ++j) {
                // what the tile's chunks are to the unit: lane e looks at chunk e; lane i
                // fetches the documents of keys 4i .. 4i + 3 while S is computed
                const int per = kTileKeys >> p.shift;
                const int mine = j * per + lane < n_list ? s_list[j * per + lane] : -1;
                const bool plain = __all_sync(kFull, lane >= per || (mine >= 0 && (mine & kChunkFull)));
                int dk[4];
                if (docs && !plain) {
                    const int entry = __shfl_sync(kFull, mine, (4 * lane) >> p.shift);
                    const int at = ((entry & kChunkId) << p.shift) + ((4 * lane) & (p.c.chunk - 1));
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        dk[c] = entry >= 0 && at + c < p.c.nk_tokens ? doc_k[at + c] : -1;
                }
                ok = mbar_wait_warp(&s_full[t], j & 1, abort_flag);
                if (!ok) break;
                tc_fence_after();
                float s[kTileKeys];
#pragma unroll
                for (int c = 0; c < kTileKeys; c += 32) ld32(s_at + c, s + c);
#pragma unroll
                for (int c = 0; c < kTileKeys; c += 32) wait_ld32(s + c);
                if (cap) {
                    // z = s1 s; the polynomial alone while no score of the warp reaches the cap
                    float tops[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < kTileKeys; c += 8)
#pragma unroll
                        for (int i = 0; i < 4; ++i) tops[i] = max3(tops[i], fabsf(s[c + 2 * i]), fabsf(s[c + 2 * i + 1]));
                    const float most = max3(max3(tops[0], tops[1], tops[2]), tops[3], tops[3]);
                    if (__all_sync(kFull, most * p.s1 < 1.f)) {
#pragma unroll
                        for (int c = 0; c < kTileKeys; ++c) s[c] = p.s2 * rr_attn::tanh_within_one(s[c] * p.s1);
                    } else {
#pragma unroll
                        for (int c = 0; c < kTileKeys; ++c) s[c] = p.s2 * rr_attn::tanh_f32(s[c] * p.s1);
                    }
                }
                const float scale = cap ? 1.f : p.s1;
                if (bias) {
#pragma unroll
                    for (int c0 = 0; c0 < kTileKeys; c0 += 16) {
                        const int entry = __shfl_sync(kFull, mine, c0 >> p.shift) & kChunkId;
                        const float from = (float)(pos - ((entry << p.shift) + (c0 & (p.c.chunk - 1))));
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            s[c0 + c] = s[c0 + c] * scale - slope * (fabsf(from - (float)c) - (float)near);
                    }
                }
                if (!plain) {
#pragma unroll
                    for (int c0 = 0; c0 < kTileKeys; c0 += 16) {
                        const int entry = __shfl_sync(kFull, mine, c0 >> p.shift);
                        if (entry >= 0 && (entry & kChunkFull)) continue;
                        const int base = entry < 0 ? 0 : ((entry & kChunkId) << p.shift) + (c0 & (p.c.chunk - 1));
                        const int left = entry < 0 ? 0 : limit - base;
#pragma unroll
                        for (int c = 0; c < 16; ++c) s[c0 + c] = c < left ? s[c0 + c] : -INFINITY;
                    }
                    if (docs) {
#pragma unroll
                        for (int c = 0; c < kTileKeys; ++c)
                            if (__shfl_sync(kFull, dk[c & 3], c >> 2) != doc) s[c] = -INFINITY;
                    }
                }
                const float mul = bias ? 1.f : scale;
                float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < kTileKeys; c += 8)
#pragma unroll
                    for (int i = 0; i < 4; ++i) tops[i] = max3(tops[i], s[c + 2 * i], s[c + 2 * i + 1]);
                const float top = max3(max3(tops[0], tops[1], tops[2]), tops[3], tops[3]) * mul;
                if (__any_sync(kFull, top > m + kSlack)) {
                    const float was = m;
                    m = fmaxf(m, top);
                    if (j > 0) {
                        const float corr = was == -INFINITY ? 0.f : rr_attn::ex2(was - m);
                        l *= corr;
                        ok = mbar_wait_warp(&o_done[t], (j - 1) & 1, abort_flag);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int c = 0; c < DH; c += 32) {
                            float o[32];
                            ld32(o_at + c, o);
                            wait_ld32(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] *= corr;
                            st32(o_at + c, o);
                        }
                    }
                }
                // an infinite or NaN score makes the row NaN
                const float ref = !(top < INFINITY) ? NAN : m == -INFINITY ? 0.f : kLift - m;
                float sums[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int half = 0; half < 2; ++half) {
#pragma unroll
                    for (int c0 = half * 64; c0 < half * 64 + 64; c0 += 32) {
                        uint32_t w[16];
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            const float x = rr_attn::ex2(fmaf(s[c0 + 2 * c], mul, ref));
                            const float y = rr_attn::ex2(fmaf(s[c0 + 2 * c + 1], mul, ref));
                            sums[2 * (c & 1)] += x;
                            sums[2 * (c & 1) + 1] += y;
                            w[c] = Half<T>::pack(x, y);
                        }
                        st16(s_at + c0 / 2, w);
                    }
                    wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_ready[2 * t + half]);
                }
                l += (sums[0] + sums[1]) + (sums[2] + sums[3]);
            }
            if (ok && n > 0) {
                ok = mbar_wait_warp(&o_done[t], (n - 1) & 1, abort_flag);
                tc_fence_after();
            }
            // Rows go out by TMA from where Q lay (every product that read it is done), a
            // warp's 32 rows by itself.  A row that saw nothing is zero whatever its
            // accumulators hold.
            const float inv = l == 0.f ? 0.f : 1.f / l;
            bool bad = false;
            unsigned char *dst = q_s + t * S::kTileBytes + (threadIdx.x & 127) * 128;
#pragma unroll
            for (int c0 = 0; c0 < DH; c0 += 32) {
                float o[32];
                if (ok && n > 0) {
                    ld32(o_at + c0, o);
                    wait_ld32(o);
                }
                uint32_t w[16];
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    if (!ok) o[2 * c] = o[2 * c + 1] = NAN;
                    else if (l == 0.f) o[2 * c] = o[2 * c + 1] = 0.f;
                    bad = bad || !isfinite(o[2 * c]) || !isfinite(o[2 * c + 1]);
                    w[c] = Half<T>::pack(o[2 * c] * inv, o[2 * c + 1] * inv);
                }
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    *reinterpret_cast<uint4 *>(dst + (c0 >> 6) * kSubBytes + ((((c0 & 63) / 8 + c) ^ (lane & 7)) << 4)) =
                        make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
                const int rows_out = min(32, p.c.chunk);
                for (int r = 0; r < 32; r += rows_out) {
                    const int ur = row0 + warp * 32 + r;       // of the unit; 32 warp: tile and row
                    if (ur >= rows) break;
                    for (int sub = 0; sub < S::kSubs; ++sub)
                        tma_store_4d(&maps.out, saddr(q_s) + t * S::kTileBytes + sub * kSubBytes + ((warp & 3) * 32 + r) * 128,
                                     sub * 64, (u.i << p.shift) + (ur & (p.c.chunk - 1)),
                                     u.route_head * p.group + (ur >> p.shift), u.b);
                }
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
            if (valid && p.a.lse)
                p.a.lse[((size_t)u.b * p.c.q_heads + head) * p.c.nq_tokens + token] =
                    !ok ? NAN
                        : l == 0.f ? -INFINITY
                                   : (m - kLift + log2f(l)) * kLn2 - (bias ? p.a.slopes[head] * (float)near : 0.f);
            // (where the sum is a NaN, a score that the row sees is one, and so is the row)
            unsigned again = __ballot_sync(kFull, ok && bad && valid && l == l);
            if (lane == 0) {
                if (again) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
                else asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            }
            __syncwarp();
            while (again) {
                const int r = __ffs(again) - 1;
                again &= again - 1;
                row_alone<T, DH>(p, u, s_list, n_list, row0 + (warp << 5) + r, __shfl_sync(kFull, near, r));
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == kSoftWarps + 1) {
            // ---- producer: K_0, V_0, K_1, V_1, ... ----
            const int box = p.c.chunk, per = kTileKeys >> p.shift;
            const int kh = maps.axes[1] & 1 ? u.kv_head : 0, kb = maps.axes[1] & 2 ? u.b : 0;
            const int vh = maps.axes[2] & 1 ? u.kv_head : 0, vb = maps.axes[2] & 2 ? u.b : 0;
            if (n > 0) {
                // the heads of the tiles' rows; rows past the unit as tokens past the last, which read as zeros
                mbar_expect_tx_elect(q_ready, tiles * S::kTileBytes);
                for (int e = 0; e < tiles * per; ++e) {
                    const int h = (row0 >> p.shift) + e;
                    const int head = maps.axes[0] & 1 ? u.route_head * p.group + min(h, p.group - 1) : 0;
                    const int token = h < p.group ? u.i << p.shift : p.c.nq_tokens;
                    for (int sub = 0; sub < S::kSubs; ++sub)
                        tma_load_4d_elect(saddr(q_s) + e / per * S::kTileBytes + sub * kSubBytes + e % per * box * 128,
                                          &maps.q, q_ready, sub * 64, token, head, maps.axes[0] & 2 ? u.b : 0);
                }
            }
            int issued = 0;
            for (int g = 0; g < 2 * n; ++g) {
                const int s = g % S::kStages;
                if (g >= S::kStages && !mbar_wait_warp(&empty[s], ((g / S::kStages) & 1) ^ 1, abort_flag)) break;
                mbar_expect_tx_elect(&full[s], S::kTileBytes);
                const CUtensorMap *map = g & 1 ? &maps.v : &maps.k;
                const uint32_t dst = saddr(kv_s) + s * S::kTileBytes;
                for (int e = 0; e < per; ++e) {
                    // past the route: a box past the tokens, which reads as zeros
                    const int at = (g >> 1) * per + e;
                    const int token = at < n_list ? (s_list[at] & kChunkId) << p.shift : p.c.nk_tokens;
                    for (int sub = 0; sub < S::kSubs; ++sub)
                        tma_load_4d_elect(dst + sub * kSubBytes + e * box * 128, map, &full[s], sub * 64, token,
                                          g & 1 ? vh : kh, g & 1 ? vb : kb);
                }
                ++issued;
            }
            // every issued copy must have landed before the CTA exits
            if (n > 0) {
                const long long t0 = clock64();
                while (!mbar_test(q_ready, 0) && clock64() - t0 < kSpinLimit) {
                }
            }
            for (int g = max(0, issued - S::kStages); g < issued; ++g) {
                const long long t0 = clock64();
                while (!mbar_test(&full[g % S::kStages], (g / S::kStages) & 1) && clock64() - t0 < kSpinLimit) {
                }
            }
        } else if (warp == kSoftWarps) {
            // ---- MMA issuer ----
            constexpr uint32_t kQk = idesc_of<T>(kTileKeys, false), kPv = idesc_of<T>(DH, true);
            const uint32_t base = __shfl_sync(kFull, tmem, 0);
            bool ok = n > 0 && mbar_wait_warp(q_ready, 0, abort_flag);
            auto qk = [&](int t, int s) {
                const uint64_t a = sw128_desc(saddr(q_s) + t * S::kTileBytes), b = sw128_desc(saddr(kv_s) + s * S::kTileBytes);
#pragma unroll
                for (int kk = 0; kk < DH / 16; ++kk) {
                    const uint64_t off = (uint64_t)((kk >> 2) * (kSubBytes >> 4) + (kk & 3) * 2);
                    tc_mma_bf16_elect(base + t * 128, a + off, b + off, kQk, kk > 0 ? 1u : 0u);
                }
                tc_commit_elect(&s_full[t]);
            };
            // half 0 and 1: keys 0-63 and 64-127 of the tile
            auto pv = [&](int t, int s, int half, bool first) {
                const uint64_t b = n_major_desc(saddr(kv_s) + s * S::kTileBytes);
#pragma unroll
                for (int k4 = 0; k4 < kTileKeys / 32; ++k4) {
                    const int kk = half * (kTileKeys / 32) + k4;
                    tc_mma_bf16_ts_elect(base + 256 + t * 128, base + t * 128 + kk * 8, b + (uint64_t)(kk * (2048 >> 4)),
                                         kPv, first && kk == 0 ? 0u : 1u);
                }
                if (half) tc_commit_elect(&o_done[t]);
            };
            if (ok) ok = mbar_wait_warp(&full[0], 0, abort_flag);
            if (ok) {
                tc_fence_after();
                for (int t = 0; t < tiles; ++t) qk(t, 0);
                tc_commit_elect(&empty[0]);
            }
            for (int j = 0; ok && j < n; ++j) {
                const int gv = 2 * j + 1, sv = gv % S::kStages, gk = 2 * j + 2, sk = gk % S::kStages;
                ok = mbar_wait_warp(&full[sv], (gv / S::kStages) & 1, abort_flag);
                if (ok && j + 1 < n) ok = mbar_wait_warp(&full[sk], (gk / S::kStages) & 1, abort_flag);
                for (int t = 0; ok && t < tiles; ++t) {
                    for (int half = 0; ok && half < 2; ++half) {
                        ok = mbar_wait_warp(&p_ready[2 * t + half], j & 1, abort_flag);
                        if (!ok) break;
                        tc_fence_after();
                        pv(t, sv, half, j == 0);
                    }
                    if (!ok) break;
                    if (t == tiles - 1) tc_commit_elect(&empty[sv]);
                    if (j + 1 < n) {
                        qk(t, sk);
                        if (t == tiles - 1) tc_commit_elect(&empty[sk]);
                    }
                }
            }
            tc_commit_elect(mma_done);
            const long long t0 = clock64();
            while (!mbar_test(mma_done, 0) && clock64() - t0 < kSpinLimit) {
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kSoftWarps) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// [batch, heads, tokens, dh] by strides, in boxes of `box` tokens by 64 elements.
// An axis that repeats one row (stride 0) has size 1 in the map; bits 0 and 1 of
// `axes` say whether the head and the batch entry are coordinates.
bool tensor_map(const Masked &p, const void *x, int tokens, int heads, const int64_t (&stride)[3], int box_tokens,
                CUtensorMap *map, int *axes) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const int sizes[2] = {heads, p.c.batch};
    cuuint64_t dims[4] = {(cuuint64_t)p.c.dh, (cuuint64_t)tokens, 1, 1}, bytes[3];
    const cuuint64_t row = (cuuint64_t)p.c.dh * 2;
    bytes[0] = tokens > 1 ? (cuuint64_t)stride[2] * 2 : row;
    *axes = 0;
    for (int i = 0; i < 2; ++i) {
        const int64_t st = stride[1 - i];
        bytes[1 + i] = row;
        if (sizes[i] > 1 && st > 0) {
            dims[2 + i] = sizes[i];
            bytes[1 + i] = (cuuint64_t)st * 2;
            *axes |= 1 << i;
        }
    }
    const cuuint32_t box[4] = {64u, (cuuint32_t)box_tokens, 1u, 1u}, step[4] = {1u, 1u, 1u, 1u};
    return enc(map, p.c.dtype == RR_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
               const_cast<void *>(x), dims, bytes, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Units that fill a tile of 128 rows; operands whose tokens are apart (a map has
// no stride of 0 there) and within the map's strides.
bool tc_takes(const Masked &p) {
    if ((p.group << p.shift) < kTileRows || p.c.nk_tokens < 1 || p.c.width < 1) return false;
    if (p.c.nk_tokens > 1 && (p.c.k_stride[2] == 0 || p.c.v_stride[2] == 0)) return false;
    if (p.c.nq_tokens > 1 && p.c.q_stride[2] == 0) return false;
    for (const int64_t (*s)[3] : {&p.c.q_stride, &p.c.k_stride, &p.c.v_stride, &p.c.out_stride})
        for (int64_t x : *s)
            if (x >= 1ll << 39) return false;
    return true;
}

template <typename T, int DH>
cudaError_t launch_tc_as(const Masked &p, unsigned units, cudaStream_t s) {
    using S = TcShape<DH>;
    static_assert(S::kSmem <= 232448, "shared memory of one CTA");
    Maps maps;
    const rr_masked_attn_config &c = p.c;
    if (!tensor_map(p, p.a.q, c.nq_tokens, c.q_heads, c.q_stride, c.chunk, &maps.q, &maps.axes[0]) ||
        !tensor_map(p, p.a.k, c.nk_tokens, c.kv_heads, c.k_stride, c.chunk, &maps.k, &maps.axes[1]) ||
        !tensor_map(p, p.a.v, c.nk_tokens, c.kv_heads, c.v_stride, c.chunk, &maps.v, &maps.axes[2]) ||
        !tensor_map(p, p.a.out, c.nq_tokens, c.q_heads, c.out_stride, c.chunk < 32 ? c.chunk : 32, &maps.out,
                    &maps.axes[3]))
        return cudaErrorInvalidValue;
    auto kern = masked_attention_tc_kernel<T, DH>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = rr_attn::allow_smem(reinterpret_cast<const void *>(kern), S::kSmem, done);
    if (e != cudaSuccess) return e;
    Masked q = p;
    q.tiles = ((p.group << p.shift) + kTiles * kTileRows - 1) / (kTiles * kTileRows);
    kern<<<units * (unsigned)q.tiles, kTcThreads, S::kSmem, s>>>(q, maps);
    return cudaGetLastError();
}

cudaError_t launch_tc(const Masked &p, unsigned units, cudaStream_t s) {
    if (p.c.dtype == RR_BF16)
        return p.c.dh == 64 ? launch_tc_as<__nv_bfloat16, 64>(p, units, s) : launch_tc_as<__nv_bfloat16, 128>(p, units, s);
    return p.c.dh == 64 ? launch_tc_as<__half, 64>(p, units, s) : launch_tc_as<__half, 128>(p, units, s);
}

}  // namespace rr_masked

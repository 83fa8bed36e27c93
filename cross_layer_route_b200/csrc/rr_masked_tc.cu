// rr_masked_tc.cu -- masked attention over a route on tcgen05 (declared in
// include/rr_attention.h; the masks and the list of key chunks in rr_masked.cuh).
//
// A work item = up to 256 rows of a unit in two tiles of 128 (the query heads that
// share a key head times the chunk's tokens), so that a 128-key tile of K and V
// fetched from L2 serves 256 rows: at 4 dh flops a pair that is what L2 can feed.
// One CTA per SM takes items in turn:
//   warps 0-3, 4-7  softmax of tile 0 and 1, a thread per row (TMEM lane): S is
//                   read from TMEM into registers, scores and masks are applied,
//                   P goes back to TMEM in 16 bits over the first half of S;
//   warp 8          issues tcgen05.mma: S = Q K^T (both operands in shared
//                   memory), O += P V (P from TMEM, V as it lies in memory, an
//                   N-major operand);
//   warp 9          TMA producer: Q, then key chunks gathered by the route into
//                   tiles of 128 keys, K and V in turn through a ring of stages;
//   warps 10, 11    the list of key chunks of the next item.
// (A unit of one row tile has both groups on it, the tiles of keys in turn.)
// While one tile's softmax runs, the tensor cores work for the other, and the next
// item's list, queries and first keys arrive while this one ends.  TMEM: two S
// tiles and two O tiles of 128 columns.  P aliases S: the product that reads it
// is issued before the one that writes the next S, and they execute in order.
//
// The running maximum moves only when it would grow by more than 2^8 (in the
// weights), so O is seldom rescaled: the weights then reach 2^8, times the 2^7
// that keeps small ones away from f16's subnormals, and all sums are fp32.
//
// Measured on a B200: 65536 tokens of 16 query and 4 key heads of 128, chunks of 64,
// 32 routed, 5 documents (1.0 TFLOP) 0.97 ms, 1020 TFLOP/s of 1650, and 1.05 ms in a
// row, where the power limit lowers the clock; the products alone take 0.58 ms and
// with the copies 0.67.  What is left is the softmax: exp (16 a cycle and SM, as
// many as the tensor cores multiply scores for at dh 128) 0.11 ms, the masked last
// tile 0.08 ms, and the wait of a tile for its own two products.  Two prompts' pieces
// of 2048 tokens of 32 heads, 48 routed, scores capped (206 GFLOP): 0.35 ms, bound by
// the cap's polynomial.  Measured and not kept: an eighth of the exps on the FMA
// pipe (2 % faster, a quarter of them slower), code of their own for unmasked tiles
// (no change), one block per item (1.09 ms), results by TMA (6500 cycles an item, by
// 32-byte stores 2000).
//
// Every wait is bounded (kWaitLimit); when one runs out the CTA stops, drains its copies,
// waits for its last MMA, frees TMEM and leaves the rows it has not written NaN.
#include "rr_masked.cuh"
#include "rr_tc.cuh"

namespace rr_masked {

using namespace rr::tc;
using rr_attn::add2;
using rr_attn::fma2;
using rr_attn::pack2;
using rr_attn::unpack2;

constexpr int kSms = 148;
constexpr int kTileRows = 128;
constexpr int kTileKeys = 128;
constexpr int kTiles = 2;
constexpr int kSoftWarps = 4 * kTiles;
constexpr int kTcThreads = 32 * (kSoftWarps + 4);
// Registers: launched with 168 a thread (384 threads: 64512 in all), then the two
// softmax groups take 224 and the third keeps 56: 2 * 128 * 224 + 128 * 56 = 64512.
constexpr int kSoftRegs = 224, kOtherRegs = 56;
constexpr float kSlack = 8.f;     // growth of the maximum that is let pass
constexpr float kLift = 7.f;      // weights are 2^7 at the maximum
constexpr int kSubBytes = kTileRows * 128;    // 128 rows of 64 elements
// Cycles that a wait lasts at most, 8.7 s.  While a softmax warp computes rows on their
// own (row_alone), all other roles wait for it: 32 rows of the widest route's 131072 keys
// at the 610 cycles a key that they take out of L2 are 1.3 s, at 4096 a key the limit.
// (Waits of a second that such rows prolong made capped scores 2 to 5 % slower.)
constexpr long long kWaitLimit = 1ll << 34;


template <int DH>
struct TcShape {
    static constexpr int kSubs = DH / 64;
    static constexpr int kTileBytes = kSubs * kSubBytes;          // a Q, K or V tile
    static constexpr int kStages = DH == 128 ? 4 : 8;
    static constexpr int kLists = 2 * (kMaxWidth + 4) * 4;        // lists and their lengths
    static constexpr int kBars = 2 * kStages + 4 * kTiles + 2 + 5;
    static constexpr int kMisc = 64 + kTileRows * 8;              // flags; the second group's states
    static constexpr int kSmem =
        1024 + kLists + kBars * 8 + kMisc + (kTiles + kStages) * kTileBytes;
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

// 32 bytes, on a 32-byte boundary.
__device__ __forceinline__ void st_global_32(void *x, const uint32_t *w) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(x), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// Tensor maps of the operands; axes: see tensor_map.
struct Maps {
    CUtensorMap q, k, v;
    int axes[3];
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
// The same for 16 columns, waited for at once.
__device__ __forceinline__ void ld16(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
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

// The row of a unit that a softmax thread has.
struct Row {
    int head, token, pos;
    bool valid;
};
__device__ __forceinline__ Row row_of(const Masked &p, const Unit &u, int thread) {
    const int row = u.tile * kTiles * kTileRows + thread, tok = row & (p.c.chunk - 1);
    const bool in_unit = row < p.group << p.shift;
    Row r;
    r.head = u.route_head * p.group + (in_unit ? row >> p.shift : 0);
    r.token = (u.i << p.shift) + tok;
    r.pos = u.p_first + tok;
    r.valid = in_unit && tok < u.tokens;
    return r;
}

// A bounded wait whose outcome the whole warp shares.
__device__ __forceinline__ bool wait_warp(uint64_t *b, uint32_t parity, volatile int *abort_flag) {
    return __all_sync(kFull, mbar_wait(b, parity, abort_flag, kWaitLimit));
}

// The softmax warps' barrier.
__device__ __forceinline__ void soft_sync() {
    asm volatile("bar.sync 2, %0;" ::"n"(32 * kSoftWarps) : "memory");
}

// SINGLE: units of one row tile.  Both softmax groups take it, the key tiles in turn,
// with an S, an O, a maximum and a sum each, joined at the end: the tensor cores work
// for one half of the keys while the other's softmax runs.  8192 tokens, 8 heads of 2
// queries, chunks of 64, 32 routed: 159 -> 118 us at dh 64, 196 -> 146 at dh 128; with
// a cap and a bias, chunks of 32 of 4 queries, 432 -> 317 and 479 -> 372; units of two
// key tiles gain nothing and a unit of one loses 0.5 us.
//
// CAP and BIAS: whether the scores are capped and have a bias.  Each keeps its
// registers and branches out of the others' loop: 1.15 -> 1.01 ms for 65536 tokens
// of 16 heads without either, 0.51 -> 0.35 ms for 2 x 2048 tokens of 32 heads with a
// cap (its polynomial in paired operations).
template <typename T, int DH, bool CAP, bool BIAS, bool SINGLE>
__global__ void __launch_bounds__(kTcThreads, 1)
masked_attention_tc_kernel(const __grid_constant__ Masked p, const __grid_constant__ Maps maps, int items) {
    using S = TcShape<DH>;
    extern __shared__ unsigned char raw[];
    unsigned char *smem = align_smem_1024(raw);
    unsigned char *q_s = smem, *kv_s = smem + kTiles * S::kTileBytes;
    int32_t *s_list = reinterpret_cast<int32_t *>(kv_s + S::kStages * S::kTileBytes);     // two, of kMaxWidth
    int32_t *s_n = s_list + 2 * kMaxWidth;
    uint64_t *full = reinterpret_cast<uint64_t *>(s_n + 8);
    uint64_t *empty = full + S::kStages, *s_full = empty + S::kStages, *p_ready = s_full + kTiles;
    uint64_t *o_done = p_ready + 2 * kTiles, *q_ready = o_done + kTiles, *q_free = q_ready + 1;
    uint64_t *list_ready = q_free + 1, *list_free = list_ready + 2, *mma_done = list_free + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1), *go_on = abort_flag + 1;
    float2 *s_join = reinterpret_cast<float2 *>(tmem_slot + 4);       // maximum and sum of the second group's rows

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = p.group << p.shift;
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
            mbar_init(&list_ready[t], 1);
            mbar_init(&list_free[t], kSoftWarps + 2);
        }
        mbar_init(q_ready, 1);
        mbar_init(q_free, 1);
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
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    auto tiles_of = [&](const Unit &u) {
        return min(kTiles, (rows - u.tile * kTiles * kTileRows + kTileRows - 1) / kTileRows);
    };

    // Item `it` of this CTA uses list it & 1; barriers that complete once per item,
    // stage or tile are waited for by counting them.
    if (warp < kSoftWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        // ---- softmax: one row per thread ----
        const int t = warp >> 2, thread = SINGLE ? threadIdx.x & (kTileRows - 1) : threadIdx.x;
        const bool docs = p.a.doc_q != nullptr;
        constexpr bool bias = BIAS;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;    // TMEM lane 32 (warp mod 4), in bits 16-31
        const uint32_t s_at = tmem + lanes + t * 128, o_at = tmem + lanes + 256 + t * 128;
        // the results' rows start on 32 bytes
        const bool out32 = (reinterpret_cast<uintptr_t>(p.a.out) & 31) == 0 &&
                           ((p.c.out_stride[0] | p.c.out_stride[1] | p.c.out_stride[2]) & 15) == 0;
        int done = 0;                                         // tiles of keys behind this row tile
        bool ok = true;
        for (int it = 0, item = blockIdx.x; item < items; ++it, item += gridDim.x) {
            const int32_t *list = s_list + (it & 1) * kMaxWidth;
            ok = ok && wait_warp(&list_ready[it & 1], (it >> 1) & 1, abort_flag);
            const int n_list = ok ? s_n[4 * (it & 1)] : 0;
            const int n = ((n_list << p.shift) + kTileKeys - 1) / kTileKeys;
            const int tiles = tiles_of(unit_of(p, item));
            const int turns = SINGLE ? (n - t + 1) >> 1 : n;      // tiles of keys of this group
            if (SINGLE || t < tiles) {
                int pos, doc, limit, near;
                const int32_t *doc_k;
                float slope;
                {
                    const Unit u = unit_of(p, item);
                    const Row r0 = row_of(p, u, thread);
                    pos = r0.pos;
                    doc = docs && r0.valid ? p.a.doc_q[(size_t)u.b * p.c.nq_tokens + r0.token] : -1;
                    doc_k = docs ? p.a.doc_k + (size_t)u.b * p.c.nk_tokens : nullptr;
                    // keys below this are in sight; none to a row without a document
                    limit = docs && doc < 0 ? 0 : min(p.c.nk_tokens, p.c.causal ? max(pos + 1, u.prefix) : p.c.nk_tokens);
                    slope = bias ? p.a.slopes[r0.head] * kLog2e : 0.f;
                    near = 0;
                    if (bias && ok) {
                        near = nearest(p, u, list, n_list, pos, doc, 0, 1);
                        if (near == INT_MAX) near = 0;
                    }
                }
                float m = -INFINITY, l = 0.f;
                for (int i = 0; ok && i < turns; ++i) {
                    const int j = SINGLE ? 2 * i + t : i;
                    // what the tile's chunks are to the unit: lane e looks at chunk e; lane i
                    // fetches the documents of keys 4i .. 4i + 3 while S is computed
                    const int per = kTileKeys >> p.shift;
                    const int mine = j * per + lane < n_list ? list[j * per + lane] : -1;
                    const bool plain = __all_sync(kFull, lane >= per || (mine >= 0 && (mine & kChunkFull)));
                    int dk[4];
                    const bool cut = __any_sync(kFull, lane < per && mine >= 0 && (mine & kChunkCut));
                    if (cut) {
                        const int entry = __shfl_sync(kFull, mine, (4 * lane) >> p.shift);
                        const int at = ((entry & kChunkId) << p.shift) + ((4 * lane) & (p.c.chunk - 1));
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            dk[c] = entry >= 0 && at + c < p.c.nk_tokens ? doc_k[at + c] : -1;
                    }
                    ok = wait_warp(&s_full[t], (done + i) & 1, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    float s[kTileKeys];
#pragma unroll
                    for (int c = 0; c < kTileKeys; c += 32) ld32(s_at + c, s + c);
#pragma unroll
                    for (int c = 0; c < kTileKeys; c += 32) wait_ld32(s + c);
                    if constexpr (CAP) {
                        // z = s1 s; the polynomial alone while no score of the warp reaches the cap
                        float tops[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int c = 0; c < kTileKeys; c += 8)
#pragma unroll
                            for (int i = 0; i < 4; ++i) tops[i] = max3(tops[i], fabsf(s[c + 2 * i]), fabsf(s[c + 2 * i + 1]));
                        const float most = max3(max3(tops[0], tops[1], tops[2]), tops[3], tops[3]);
                        if (__all_sync(kFull, most * p.s1 < 1.f)) {
#pragma unroll
                            for (int c = 0; c < kTileKeys; c += 2) rr_attn::tanh_pair(s + c, p.s1);
                        } else {
#pragma unroll
                            for (int c = 0; c < kTileKeys; ++c) s[c] = rr_attn::tanh_f32(s[c] * p.s1);
                        }
                    }
                    const float scale = CAP ? p.s2 : p.s1;     // what remains to multiply
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
                        if (cut) {
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
                        if (i > 0) {
                            const float corr = was == -INFINITY ? 0.f : rr_attn::ex2(was - m);
                            l *= corr;
                            ok = wait_warp(&o_done[t], (done + i - 1) & 1, abort_flag);
                            if (!ok) break;
                            tc_fence_after();
                            // 16 columns at a time: the scores hold 128 registers
#pragma unroll 1
                            for (int c = 0; c < DH; c += 16) {
                                uint32_t o[16];
                                ld16(o_at + c, o);
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
                                st16(o_at + c, o);
                            }
                        }
                    }
                    // an infinite or NaN score makes the row NaN
                    const float ref = !(top < INFINITY) ? NAN : m == -INFINITY ? 0.f : kLift - m;
                    const uint64_t mul2 = pack2(mul, mul), ref2 = pack2(ref, ref);
                    uint64_t sums[2] = {0, 0};
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
#pragma unroll
                        for (int c0 = half * 64; c0 < half * 64 + 64; c0 += 32) {
                            uint32_t w[16];
#pragma unroll
                            for (int c = 0; c < 16; ++c) {
                                float x, y;
                                unpack2(fma2(pack2(s[c0 + 2 * c], s[c0 + 2 * c + 1]), mul2, ref2), x, y);
                                x = rr_attn::ex2(x);
                                y = rr_attn::ex2(y);
                                sums[c & 1] = add2(sums[c & 1], pack2(x, y));
                                w[c] = Half<T>::pack(x, y);
                            }
                            st16(s_at + c0 / 2, w);
                        }
                        wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&p_ready[2 * t + half]);
                    }
                    float sum0, sum1;
                    unpack2(add2(sums[0], sums[1]), sum0, sum1);
                    l += sum0 + sum1;
                }
                if (ok && turns > 0) {
                    ok = wait_warp(&o_done[t], (done + turns - 1) & 1, abort_flag);
                    tc_fence_after();
                }
                done += turns;
                // the groups' halves of a row: O = O0 2^(m0 - m) + O1 2^(m1 - m), without the
                // accumulators of a half that saw nothing
                float from0 = 0.f, from1 = 0.f;
                bool use0 = false, use1 = false;
                if constexpr (SINGLE) {
                    if (t == 1) s_join[thread] = make_float2(m, ok ? l : -1.f);
                    tc_fence_before();
                    soft_sync();
                    tc_fence_after();
                    if (t == 1) {
                        soft_sync();         // the first group has read this one's O
                        tc_fence_after();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&list_free[it & 1]);
                        continue;
                    }
                    const float2 other = s_join[thread];
                    ok = ok && __all_sync(kFull, other.y != -1.f);
                    use0 = l != 0.f;
                    use1 = other.y != 0.f;
                    const float top = !use1 ? m : !use0 ? other.x : fmaxf(m, other.x);
                    if (use0) from0 = rr_attn::ex2(m - top);
                    if (use1) from1 = rr_attn::ex2(other.x - top);
                    l = (use0 ? l * from0 : 0.f) + (use1 ? other.y * from1 : 0.f);
                    m = top;
                }
                // (worked out again: kept over the loop, it costs registers that the scores need)
                int again_item = item;
                asm volatile("" : "+r"(again_item));
                const Unit u = unit_of(p, again_item);
                const Row r0 = row_of(p, u, thread);
                const int row0 = u.tile * kTiles * kTileRows;
                // A thread writes its row in whole sectors.  A row that saw nothing is zero
                // whatever its accumulators hold.
                T *out = static_cast<T *>(p.a.out) + u.b * p.c.out_stride[0] + r0.head * p.c.out_stride[1] +
                         r0.token * p.c.out_stride[2];
                const float inv = l == 0.f ? 0.f : 1.f / l;
                bool bad = false;
#pragma unroll
                for (int c0 = 0; c0 < DH; c0 += 32) {
                    float o[32];
                    if (ok && n > 0) {
                        ld32(o_at + c0, o);
                        wait_ld32(o);
                        if constexpr (SINGLE) {
#pragma unroll
                            for (int c16 = 0; c16 < 32; c16 += 16) {
                                uint32_t second[16];
                                if (n > 1) ld16(o_at + 128 + c0 + c16, second);
#pragma unroll
                                for (int c = 0; c < 16; ++c)
                                    o[c16 + c] = (use0 ? o[c16 + c] * from0 : 0.f) +
                                                 (use1 ? __uint_as_float(second[c]) * from1 : 0.f);
                            }
                        }
                    }
                    uint32_t w[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        if (!ok) o[2 * c] = o[2 * c + 1] = NAN;
                        else if (l == 0.f) o[2 * c] = o[2 * c + 1] = 0.f;
                        bad = bad || !isfinite(o[2 * c]) || !isfinite(o[2 * c + 1]);
                        w[c] = Half<T>::pack_mean(o[2 * c] * inv, o[2 * c + 1] * inv);
                    }
                    if (r0.valid) {
                        if (out32) {
                            st_global_32(out + c0, w);
                            st_global_32(out + c0 + 16, w + 8);
                        } else {
#pragma unroll
                            for (int c = 0; c < 16; c += 4)
                                *reinterpret_cast<uint4 *>(out + c0 + 2 * c) = make_uint4(w[c], w[c + 1], w[c + 2], w[c + 3]);
                        }
                    }
                }
                if (r0.valid && p.a.lse)
                    p.a.lse[((size_t)u.b * p.c.q_heads + r0.head) * p.c.nq_tokens + r0.token] =
                        !ok ? NAN
                            : l == 0.f ? -INFINITY
                                       : (m - kLift + log2f(l)) * kLn2 - (bias ? p.a.slopes[r0.head] * (float)near : 0.f);
                if constexpr (SINGLE) {
                    tc_fence_before();
                    soft_sync();
                }
                // (where the sum is a NaN, a score that the row sees is one, and so is the row)
                unsigned again = __ballot_sync(kFull, ok && bad && r0.valid && l == l);
                while (again) {
                    const int r = __ffs(again) - 1;
                    again &= again - 1;
                    row_alone<T, DH>(p, u, list, n_list, row0 + (warp << 5) + r, __shfl_sync(kFull, near, r));
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&list_free[it & 1]);
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == kSoftWarps + 1) {
            // ---- producer: Q; K_0, V_0, K_1, V_1, ... ----
            const int box = p.c.chunk, per = kTileKeys >> p.shift;
            int g = 0, nq = 0;                       // stages and queries issued
            bool ok = true;
            for (int it = 0, item = blockIdx.x; ok && item < items; ++it, item += gridDim.x) {
                const Unit u = unit_of(p, item);
                const int32_t *list = s_list + (it & 1) * kMaxWidth;
                ok = wait_warp(&list_ready[it & 1], (it >> 1) & 1, abort_flag);
                if (!ok) break;
                const int n_list = s_n[4 * (it & 1)], n = ((n_list << p.shift) + kTileKeys - 1) / kTileKeys;
                const int row0 = u.tile * kTiles * kTileRows, tiles = tiles_of(u);
                if (n > 0) {
                    ok = wait_warp(q_free, (nq & 1) ^ 1, abort_flag);
                    if (!ok) break;
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
                    ++nq;
                }
                const int kh = maps.axes[1] & 1 ? u.kv_head : 0, kb = maps.axes[1] & 2 ? u.b : 0;
                const int vh = maps.axes[2] & 1 ? u.kv_head : 0, vb = maps.axes[2] & 2 ? u.b : 0;
                for (int i = 0; i < 2 * n; ++i) {
                    const int s = g % S::kStages;
                    ok = wait_warp(&empty[s], ((g / S::kStages) & 1) ^ 1, abort_flag);
                    if (!ok) break;
                    mbar_expect_tx_elect(&full[s], S::kTileBytes);
                    const CUtensorMap *map = i & 1 ? &maps.v : &maps.k;
                    const uint32_t dst = saddr(kv_s) + s * S::kTileBytes;
                    for (int e = 0; e < per; ++e) {
                        // past the route: a box past the tokens, which reads as zeros
                        const int at = (i >> 1) * per + e;
                        const int token = at < n_list ? (list[at] & kChunkId) << p.shift : p.c.nk_tokens;
                        for (int sub = 0; sub < S::kSubs; ++sub)
                            tma_load_4d_elect(dst + sub * kSubBytes + e * box * 128, map, &full[s], sub * 64, token,
                                              i & 1 ? vh : kh, i & 1 ? vb : kb);
                    }
                    ++g;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&list_free[it & 1]);
            }
            // every issued copy must have landed before the CTA exits
            for (int s = max(0, g - S::kStages); s < g + (nq > 0); ++s) {
                uint64_t *bar = s < g ? &full[s % S::kStages] : q_ready;
                const int parity = s < g ? (s / S::kStages) & 1 : (nq - 1) & 1;
                const long long t0 = clock64();
                while (!mbar_test(bar, parity) && clock64() - t0 < kSpinLimit) {
                }
            }
        } else if (warp == kSoftWarps) {
            // ---- MMA issuer ----
            constexpr uint32_t kQk = idesc_of<T>(kTileKeys, false), kPv = idesc_of<T>(DH, true);
            const uint32_t base = __shfl_sync(kFull, tmem, 0);
            auto qk = [&](int t, int s) {
                const uint64_t a = sw128_desc(saddr(q_s) + (SINGLE ? 0 : t * S::kTileBytes)), b = sw128_desc(saddr(kv_s) + s * S::kTileBytes);
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
            int g = 0, nq = 0, done[kTiles] = {0, 0};      // stages, queries and tiles of keys used
            bool ok = true;
            for (int it = 0, item = blockIdx.x; ok && item < items; ++it, item += gridDim.x) {
                const Unit u = unit_of(p, item);
                ok = wait_warp(&list_ready[it & 1], (it >> 1) & 1, abort_flag);
                if (!ok) break;
                const int n = ((s_n[4 * (it & 1)] << p.shift) + kTileKeys - 1) / kTileKeys, tiles = tiles_of(u);
                __syncwarp();
                if (lane == 0) mbar_arrive(&list_free[it & 1]);
                if (n == 0) continue;
                ok = wait_warp(q_ready, nq & 1, abort_flag) &&
                     wait_warp(&full[g % S::kStages], (g / S::kStages) & 1, abort_flag);
                if (!ok) break;
                ++nq;
                tc_fence_after();
                if constexpr (SINGLE) {
                    // S of tile j + 2 after O of tile j, whose P it takes the place of
                    const int g0 = g;
                    g += 2 * n;
                    auto scores = [&](int j) {
                        const int at = g0 + 2 * j, s = at % S::kStages;
                        if (j > 0) ok = wait_warp(&full[s], (at / S::kStages) & 1, abort_flag);
                        if (!ok) return;
                        qk(j & 1, s);
                        tc_commit_elect(&empty[s]);
                        if (j + 1 == n) tc_commit_elect(q_free);
                    };
                    scores(0);
                    if (n > 1) scores(1);
                    for (int j = 0; ok && j < n; ++j) {
                        const int t = j & 1, at = g0 + 2 * j + 1, s = at % S::kStages;
                        ok = wait_warp(&full[s], (at / S::kStages) & 1, abort_flag);
                        for (int half = 0; ok && half < 2; ++half) {
                            ok = wait_warp(&p_ready[2 * t + half], ((t ? done[1] : done[0]) + (j >> 1)) & 1, abort_flag);
                            if (!ok) break;
                            tc_fence_after();
                            pv(t, s, half, j < 2);
                        }
                        if (!ok) break;
                        tc_commit_elect(&empty[s]);
                        if (j + 2 < n) scores(j + 2);
                    }
                    done[0] += (n + 1) >> 1;
                    done[1] += n >> 1;
                } else {
                    for (int t = 0; t < tiles; ++t) qk(t, g % S::kStages);
                    tc_commit_elect(&empty[g % S::kStages]);
                    if (n == 1) tc_commit_elect(q_free);
                    for (int j = 0; ok && j < n; ++j, g += 2) {
                        const int gv = g + 1, sv = gv % S::kStages, gk = g + 2, sk = gk % S::kStages;
                        ok = wait_warp(&full[sv], (gv / S::kStages) & 1, abort_flag);
                        if (ok && j + 1 < n) ok = wait_warp(&full[sk], (gk / S::kStages) & 1, abort_flag);
                        for (int t = 0; ok && t < tiles; ++t) {
                            for (int half = 0; ok && half < 2; ++half) {
                                ok = wait_warp(&p_ready[2 * t + half], (done[t] + j) & 1, abort_flag);
                                if (!ok) break;
                                tc_fence_after();
                                pv(t, sv, half, j == 0);
                            }
                            if (!ok) break;
                            if (t == tiles - 1) tc_commit_elect(&empty[sv]);
                            if (j + 1 < n) {
                                qk(t, sk);
                                if (t == tiles - 1) {
                                    tc_commit_elect(&empty[sk]);
                                    if (j + 2 == n) tc_commit_elect(q_free);
                                }
                            }
                        }
                    }
                    for (int t = 0; t < tiles; ++t) done[t] += n;
                }
            }
            tc_commit_elect(mma_done);
            const long long t0 = clock64();
            while (!mbar_test(mma_done, 0) && clock64() - t0 < kSpinLimit) {
            }
        } else {
            // ---- the lists, one item ahead ----
            // (the first warp decides for both whether to go on: they share a barrier)
            const PartTeam<32 * (kSoftWarps + 2), 64, 1> team;
            for (int it = 0, item = blockIdx.x; item < items; ++it, item += gridDim.x) {
                if (warp == kSoftWarps + 2) {
                    const bool ok = wait_warp(&list_free[it & 1], ((it >> 1) & 1) ^ 1, abort_flag);
                    if (lane == 0) *go_on = ok;
                }
                team.sync();
                if (!*go_on) break;
                build_list(team, p, unit_of(p, item), s_list + (it & 1) * kMaxWidth, s_n + 4 * (it & 1));
                if (team.rank() == 0) mbar_arrive(&list_ready[it & 1]);
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

// An axis that repeats one row (stride 0) has size 1 in the map; bits 0 and 1 of
// `axes` say whether the head and the batch entry are coordinates.  Tokens have to
// be apart, and strides below the map's 2^40 bytes.
bool tensor_map(const Masked &p, const void *base, int tokens, int heads, const int64_t (&stride)[3], int box_tokens,
                CUtensorMap *map, int *axes) {
    EncodeTiledFn enc = encode_fn();
    if (!enc || tokens < 1 || (tokens > 1 && stride[2] == 0)) return false;
    for (int64_t x : stride)
        if (x >= 1ll << 39) return false;
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
               const_cast<void *>(base), dims, bytes, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int DH, bool CAP, bool BIAS, bool SINGLE>
cudaError_t launch_tc_as(const Masked &p, unsigned units, cudaStream_t s) {
    using S = TcShape<DH>;
    static_assert(S::kSmem <= 232448, "shared memory of one CTA");
    Maps maps;
    const rr_masked_attn_config &c = p.c;
    if (!tensor_map(p, p.a.q, c.nq_tokens, c.q_heads, c.q_stride, c.chunk, &maps.q, &maps.axes[0]) ||
        !tensor_map(p, p.a.k, c.nk_tokens, c.kv_heads, c.k_stride, c.chunk, &maps.k, &maps.axes[1]) ||
        !tensor_map(p, p.a.v, c.nk_tokens, c.kv_heads, c.v_stride, c.chunk, &maps.v, &maps.axes[2]))
        return cudaErrorNotSupported;
    auto kern = masked_attention_tc_kernel<T, DH, CAP, BIAS, SINGLE>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = rr_attn::allow_smem(reinterpret_cast<const void *>(kern), S::kSmem, done);
    if (e != cudaSuccess) return e;
    Masked q = p;
    q.tiles = ((p.group << p.shift) + kTiles * kTileRows - 1) / (kTiles * kTileRows);
    const int items = (int)(units * (unsigned)q.tiles);       // at most 2^31 - 1: config_ok counts 16 rows
    kern<<<items < kSms ? items : kSms, kTcThreads, S::kSmem, s>>>(q, maps, items);
    return cudaGetLastError();
}

template <typename T, int DH, bool CAP, bool BIAS>
cudaError_t launch_tc_rows(const Masked &p, unsigned units, cudaStream_t s) {
    return (p.group << p.shift) <= kTileRows ? launch_tc_as<T, DH, CAP, BIAS, true>(p, units, s)
                                             : launch_tc_as<T, DH, CAP, BIAS, false>(p, units, s);
}

template <typename T, int DH>
cudaError_t launch_tc_type(const Masked &p, unsigned units, cudaStream_t s) {
    const bool cap = p.c.soft_cap > 0.f, bias = p.a.slopes != nullptr;
    if (cap) return bias ? launch_tc_rows<T, DH, true, true>(p, units, s) : launch_tc_rows<T, DH, true, false>(p, units, s);
    return bias ? launch_tc_rows<T, DH, false, true>(p, units, s) : launch_tc_rows<T, DH, false, false>(p, units, s);
}

// A tile of 128 rows costs the same whatever part of it a unit fills, and mma.sync, at
// a quarter of the rate, pays by the row.  Measured with 8192 tokens, 32 chunks each,
// here and there: 2048 units of 96 rows 150 and 261 us at dh 64, 189 and 437 at dh
// 128; of 64 rows 225 and 236 at dh 64 (287 and 266 by chunks of 32), 274 and 398 at
// dh 128, but with a cap and a bias 559 and 517; of 48 rows 408 and 242, 534 and 486.
cudaError_t launch_tc(const Masked &p, unsigned units, cudaStream_t s) {
    const int rows = p.group << p.shift;
    if (rows < 64 || (rows == 64 && (p.c.dh == 64 || p.c.soft_cap > 0.f)) || p.c.width < 1) return cudaErrorNotSupported;
    if (p.c.dtype == RR_BF16)
        return p.c.dh == 64 ? launch_tc_type<__nv_bfloat16, 64>(p, units, s) : launch_tc_type<__nv_bfloat16, 128>(p, units, s);
    return p.c.dh == 64 ? launch_tc_type<__half, 64>(p, units, s) : launch_tc_type<__half, 128>(p, units, s);
}

}  // namespace rr_masked

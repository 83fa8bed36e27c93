// rr_masked.cu -- masked attention over a route (declared in
// include/rr_attention.h): the entry point and the kernel on mma.sync, for units
// of up to 64 rows and operands without a tensor map (rr_masked_tc.cu has the others).
//
// One CTA = up to 64 rows of a unit (rr_masked.cuh), 16 rows per warp, so the
// query heads that share a key head read its chunks once.  Keys are visited in
// tiles of 64 slots of the concatenated route (a tile holds several chunks, or a
// part of one), two tiles deep: by TMA into swizzled rows, a copy for each chunk
// and 64 elements, or by cp.async into rows padded by 16 bytes (kTmaSlots says
// when); slots past the route are filled with zeros and masked.  S = q K^T and
// O += P V on mma.sync with fp32 sums, P straight from the scores' registers, and
//   x = s2 tanh(s1 s) or s1 s           (base-2 scores)
//   x -= slope (|pos - key| - near)      near: the row's nearest visible key
//   x = -inf where the masks say so, looked at per element only in chunks that
//       are not fully visible to the unit.
// The running maximum moves only when a score passes it by 2^8 (weights are 2^7
// at the maximum, which keeps small ones away from f16's subnormals), so most
// tiles cost one vote and no rescaling.
// A masked key has weight exactly zero; only a masked value row that holds an
// infinity or a NaN could reach a result then, as 0 * NaN, and rows with such
// accumulators are computed again on their own (row_alone).
#include <cuda_runtime.h>

#include "rr_masked.cuh"
#include "rr_tc.cuh"

namespace rr_masked {

using namespace rr_attn;

constexpr int kMaxWarps = 4;    // 16 rows each
constexpr float kSlack = 8.f;   // growth of the maximum that is let pass
constexpr float kLift = 7.f;    // weights are 2^7 at the maximum

// Slots that a call's units visit, at least, for the copies to go by TMA: it saves
// the copies' instructions (8 heads of 4 prompts of 2501 tokens at dh 64, chunks
// of 32, 1.9 M slots: 87 us, by cp.async 105 us), but its two tensor maps take the
// caller 2 us, which shows in calls whose 20 us are the caller's anyway.
constexpr long long kTmaSlots = 1 << 19;

template <int DH, bool TMA>
struct Shape {
    static constexpr int kSlots = 64;                           // key slots per tile
    static constexpr int kRow = TMA ? 64 : DH + 8;              // elements from a slot to the next
    static constexpr int kSub = kSlots * 64;                    // TMA: elements of a tile's 64-element part
    static constexpr int kTile = TMA ? kSlots * DH : kSlots * kRow;
    static constexpr int kMeta = 2 * kSlots * 4;                // documents per slot, two stages
    static constexpr int kAlign = TMA ? 1024 : 0;
    static constexpr int kSmem = kAlign + 4 * kTile * 2 + kMeta + 32;     // and the list
    static constexpr int kMinBlocks = 3;                        // CTAs per SM: at most 168 registers
};

// The two ways' tensor maps, or nothing.
struct TileMaps {
    CUtensorMap k, v;
    int axes[2];
};

// One tile of keys and values by TMA, by one warp: a lane for each copy.
template <int DH>
__device__ __forceinline__ void stage_tile_tma(const Masked &p, const Unit &u, const TileMaps &maps, const int32_t *list,
                                               int slots, int tile, uint32_t sk, uint32_t sv, uint64_t *bar) {
    using S = Shape<DH, true>;
    const int lane = threadIdx.x & 31, box = min(p.c.chunk, S::kSlots), per = S::kSlots / box;
    if (lane == 0) rr::tc::mbar_expect_tx(bar, 2 * S::kTile * 2);
    __syncwarp();
    if (lane < 2 * per * (DH / 64)) {
        const int side = lane & 1, sub = (lane >> 1) % (DH / 64), part = (lane >> 1) / (DH / 64);
        const int slot = tile * S::kSlots + part * box;
        // past the route: a box past the tokens, which reads as zeros
        const int token = slot < slots ? ((list[slot >> p.shift] & kChunkId) << p.shift) + (slot & (p.c.chunk - 1))
                                       : p.c.nk_tokens;
        const int axes = maps.axes[side];
        rr::tc::tma_load_4d((side ? sv : sk) + (sub * S::kSub + part * box * 64) * 2, side ? &maps.v : &maps.k, bar, sub * 64,
                            token, axes & 1 ? u.kv_head : 0, axes & 2 ? u.b : 0);
    }
}

// One tile of keys and values by cp.async.  A thread copies the same 16-byte column of every
// (blockDim / (DH / 8))-th slot.
template <typename T, int DH>
__device__ __forceinline__ void stage_tile(const Masked &p, const Unit &u, const int32_t *list, int slots, int tile,
                                           const T *k, const T *v, uint32_t sk, uint32_t sv) {
    using S = Shape<DH, false>;
    const int c = (threadIdx.x % (DH / 8)) * 8, step = blockDim.x / (DH / 8);
    for (int r = threadIdx.x / (DH / 8); r < S::kSlots; r += step) {
        const int slot = tile * S::kSlots + r;
        int s = slot < slots ? ((list[slot >> p.shift] & kChunkId) << p.shift) + (slot & (p.c.chunk - 1)) : -1;
        if (s >= p.c.nk_tokens) s = -1;
        const int64_t at = max(s, 0);
        const int bytes = s < 0 ? 0 : 16;
        const uint32_t to = (uint32_t)(r * S::kRow + c) * 2;
        cp_async16_zfill(sk + to, k + at * p.c.k_stride[2] + c, bytes);
        cp_async16_zfill(sv + to, v + at * p.c.v_stride[2] + c, bytes);
    }
}

// The documents of a tile's slots.
__device__ __forceinline__ void stage_documents(const Masked &p, const Unit &u, const int32_t *list, int slots, int tile,
                                                int32_t *meta) {
    for (int r = threadIdx.x; r < 64; r += blockDim.x) {
        const int slot = tile * 64 + r;
        const int s = slot < slots ? ((list[slot >> p.shift] & kChunkId) << p.shift) + (slot & (p.c.chunk - 1)) : INT_MAX;
        meta[r] = s < p.c.nk_tokens ? p.a.doc_k[(size_t)u.b * p.c.nk_tokens + s] : -1;
    }
}

template <typename T, int DH, bool TMA>
__global__ void __launch_bounds__(32 * kMaxWarps, Shape<DH, TMA>::kMinBlocks)
masked_attention_kernel(const __grid_constant__ Masked p, const __grid_constant__ TileMaps maps) {
    using S = Shape<DH, TMA>;
    constexpr int kSlots = S::kSlots;
    extern __shared__ __align__(16) unsigned char raw[];
    unsigned char *smem = TMA ? rr::tc::align_smem_1024(raw) : raw;
    T *s_k = reinterpret_cast<T *>(smem);                                  // [2][kSlots][kRow]
    T *s_v = s_k + 2 * S::kTile;                                           // [2][kSlots][kRow]
    int32_t *s_meta = reinterpret_cast<int32_t *>(s_v + 2 * S::kTile);     // [2][kSlots]
    uint64_t *full = reinterpret_cast<uint64_t *>(s_meta + 2 * kSlots);    // [2]
    volatile int *abort_flag = reinterpret_cast<volatile int *>(full + 2);
    int32_t *s_n = s_meta + 2 * kSlots + 5, *s_list = s_n + 3;             // [width]
    if (TMA && threadIdx.x == 0) {
        rr::tc::mbar_init(&full[0], 1);
        rr::tc::mbar_init(&full[1], 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }

    const Unit u = unit_of(p, blockIdx.x);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int n_list = build_list(BlockTeam(), p, u, s_list, s_n);
    const int slots = n_list << p.shift;
    const int n_tiles = (slots + kSlots - 1) / kSlots;

    const T *k = static_cast<const T *>(p.a.k) + u.b * p.c.k_stride[0] + u.kv_head * p.c.k_stride[1];
    const T *v = static_cast<const T *>(p.a.v) + u.b * p.c.v_stride[0] + u.kv_head * p.c.v_stride[1];
    const uint32_t sk0 = smem_u32(s_k), sv0 = smem_u32(s_v);
    const bool docs = p.a.doc_q != nullptr, bias = p.a.slopes != nullptr, cap = p.c.soft_cap > 0.f;
    auto stage = [&](int e) {
        const uint32_t at = (uint32_t)((e & 1) * S::kTile) * 2;
        if constexpr (TMA) {
            if (warp == 0) stage_tile_tma<DH>(p, u, maps, s_list, slots, e, sk0 + at, sv0 + at, &full[e & 1]);
        } else {
            stage_tile<T, DH>(p, u, s_list, slots, e, k, v, sk0 + at, sv0 + at);
        }
        if (docs) stage_documents(p, u, s_list, slots, e, s_meta + (e & 1) * kSlots);
    };
    if (n_tiles > 0) stage(0);
    if constexpr (!TMA) cp_async_commit();

    // This lane's two rows.  The 16 rows of a warp belong to one head (chunks
    // are multiples of 16); rows past the unit or past its tokens are computed
    // on zeros and not stored.
    const int row0 = (u.tile * kMaxWarps + warp) * 16;
    const int head = u.route_head * p.group + min(row0 >> p.shift, p.group - 1);
    const int tok0 = (row0 & (p.c.chunk - 1)) + g;                 // within the chunk; and tok0 + 8
    const bool in_unit = (row0 >> p.shift) < p.group;
    const bool ok0 = in_unit && tok0 < u.tokens, ok1 = in_unit && tok0 + 8 < u.tokens;
    const int pos0 = u.p_first + tok0, pos1 = pos0 + 8;
    const int64_t token = ((int64_t)u.i << p.shift) + tok0;
    uint32_t qf[DH / 16][4];
    {
        const T *q = static_cast<const T *>(p.a.q) + u.b * p.c.q_stride[0] + head * p.c.q_stride[1];
        const uint32_t *q0 = reinterpret_cast<const uint32_t *>(q + token * p.c.q_stride[2]);
        const uint32_t *q1 = reinterpret_cast<const uint32_t *>(q + (token + 8) * p.c.q_stride[2]);
#pragma unroll
        for (int kk = 0; kk < DH / 16; ++kk) {
            qf[kk][0] = ok0 ? q0[kk * 8 + t] : 0u;
            qf[kk][1] = ok1 ? q1[kk * 8 + t] : 0u;
            qf[kk][2] = ok0 ? q0[kk * 8 + 4 + t] : 0u;
            qf[kk][3] = ok1 ? q1[kk * 8 + 4 + t] : 0u;
        }
    }
    int doc0 = -1, doc1 = -1;
    if (docs) {
        const int32_t *dq = p.a.doc_q + (size_t)u.b * p.c.nq_tokens + token;
        if (ok0) doc0 = dq[0];
        if (ok1) doc1 = dq[8];
    }
    // keys below these are in sight; none to a row without a document
    const int end = p.c.nk_tokens, causal = p.c.causal;
    const int limit0 = docs && doc0 < 0 ? 0 : min(end, causal ? max(pos0 + 1, u.prefix) : end);
    const int limit1 = docs && doc1 < 0 ? 0 : min(end, causal ? max(pos1 + 1, u.prefix) : end);
    float slope = 0.f;
    int near0 = 0, near1 = 0;
    if (bias) {
        slope = p.a.slopes[head] * kLog2e;
        near0 = nearest(p, u, s_list, n_list, pos0, doc0, t, 4);
        near1 = nearest(p, u, s_list, n_list, pos1, doc1, t, 4);
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
            near0 = min(near0, __shfl_xor_sync(kFull, near0, d));
            near1 = min(near1, __shfl_xor_sync(kFull, near1, d));
        }
        if (near0 == INT_MAX) near0 = 0;
        if (near1 == INT_MAX) near1 = 0;
    }

    float o[DH / 8][4];
#pragma unroll
    for (int nd = 0; nd < DH / 8; ++nd) o[nd][0] = o[nd][1] = o[nd][2] = o[nd][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;   // l: this lane's part
    const int lm_row = lane & 7, lm_mat = lane >> 3;
    // ldmatrix lanes: row (lane & 7) of matrix (lane >> 3); the keys' matrices are
    // keys 16 np + {0, 0, 8, 8}, dims 16 kk + {0, 8, 0, 8}, the values' the other way
    // round.  Swizzled rows: 16-byte piece c of row r lies at c ^ (r & 7).
    const int k_row = lm_row + ((lm_mat >> 1) << 3), k_col = lm_mat & 1;
    const int v_row = lm_row + ((lm_mat & 1) << 3), v_col = lm_mat >> 1;
    auto at_k = [&](int np, int kk) {
        if constexpr (TMA)
            return (uint32_t)((kk >> 2) * S::kSub * 2 + np * 16 * 128 + k_row * 128 + ((((kk & 3) * 2 + k_col) ^ lm_row) << 4));
        else
            return (uint32_t)((np * 16 + k_row) * S::kRow + kk * 16 + k_col * 8) * 2;
    };
    auto at_v = [&](int kk, int dp) {
        if constexpr (TMA)
            return (uint32_t)((dp >> 2) * S::kSub * 2 + kk * 16 * 128 + v_row * 128 + ((((dp & 3) * 2 + v_col) ^ lm_row) << 4));
        else
            return (uint32_t)((kk * 16 + v_row) * S::kRow + dp * 16 + v_col * 8) * 2;
    };
    bool ok = true;       // (TMA) no wait has run out

    for (int e = 0; e < n_tiles; ++e) {
        const int st = e & 1;
        if (e + 1 < n_tiles) stage(e + 1);
        if constexpr (TMA) {
            ok = rr::tc::mbar_wait_warp(&full[st], (e >> 1) & 1, abort_flag) && ok;
            if (docs) __syncthreads();        // the documents
        } else {
            cp_async_commit();
            cp_async_wait_one();
            __syncthreads();
        }
        const uint32_t sk = sk0 + st * S::kTile * 2, sv = sv0 + st * S::kTile * 2;

        float s[kSlots / 8][4];
#pragma unroll
        for (int n = 0; n < kSlots / 8; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
        for (int kk = 0; kk < DH / 16; ++kk) {
#pragma unroll
            for (int np = 0; np < kSlots / 16; ++np) {
                uint32_t b0, b1, b2, b3;
                ldmatrix_x4(sk + at_k(np, kk), b0, b1, b2, b3);
                Half<T>::mma(s[2 * np], qf[kk], b0, b1);
                Half<T>::mma(s[2 * np + 1], qf[kk], b2, b3);
            }
        }

        // Scores in base 2.  Column of s[n][c]: 8n + 2t + (c & 1); row: c >> 1.
        float mul = p.s1;
        if (cap) {
            // tanh by its polynomial alone while no score of the warp reaches the cap
            mul = p.s2;
            float most = 0.f;
#pragma unroll
            for (int n = 0; n < kSlots / 8; ++n)
                most = fmaxf(most, fmaxf(fmaxf(fabsf(s[n][0]), fabsf(s[n][1])), fmaxf(fabsf(s[n][2]), fabsf(s[n][3]))));
            if (__all_sync(kFull, most * p.s1 < 1.f)) {
#pragma unroll
                for (int n = 0; n < kSlots / 8; ++n) {
                    tanh_pair(s[n], p.s1);
                    tanh_pair(s[n] + 2, p.s1);
                }
            } else {
#pragma unroll
                for (int n = 0; n < kSlots / 8; ++n)
#pragma unroll
                    for (int c = 0; c < 4; ++c) s[n][c] = tanh_f32(s[n][c] * p.s1);
            }
        }
        // 16 columns at a time: they are of one chunk
#pragma unroll
        for (int n2 = 0; n2 < kSlots / 8; n2 += 2) {
            const int at = (e * kSlots + 8 * n2) >> p.shift;
            const int entry = at < n_list ? s_list[at] : -1;
            const bool full = entry >= 0 && (entry & kChunkFull);
            if (!bias && full) continue;
            const int base = entry < 0 ? 0 : ((entry & kChunkId) << p.shift) + ((8 * n2) & (p.c.chunk - 1)) + 2 * t;
            if (bias) {
                const float from0 = (float)(pos0 - base), from1 = from0 + 8.f, n0 = (float)near0, n1 = (float)near1;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float col = (float)(8 * (c >> 1) + (c & 1));
                    float *x = s[n2 + (c >> 1)];
                    x[c & 1] = fmaf(-slope, fabsf(from0 - col) - n0, x[c & 1] * mul);
                    x[2 + (c & 1)] = fmaf(-slope, fabsf(from1 - col) - n1, x[2 + (c & 1)] * mul);
                }
            }
            if (!full) {
                const int left0 = entry < 0 ? 0 : limit0 - base, left1 = entry < 0 ? 0 : limit1 - base;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int col = 8 * (c >> 1) + (c & 1);
                    float *x = s[n2 + (c >> 1)];
                    bool see0 = col < left0, see1 = col < left1;
                    if (entry >= 0 && (entry & kChunkCut)) {
                        const int dk = s_meta[st * kSlots + 8 * n2 + 2 * t + col];
                        see0 = see0 && dk == doc0;
                        see1 = see1 && dk == doc1;
                    }
                    if (!see0) x[c & 1] = -INFINITY;
                    if (!see1) x[2 + (c & 1)] = -INFINITY;
                }
            }
        }
        if (bias) mul = 1.f;

        float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
        for (int n = 0; n < kSlots / 8; ++n) {
            mx0 = fmaxf(mx0, fmaxf(s[n][0], s[n][1]));
            mx1 = fmaxf(mx1, fmaxf(s[n][2], s[n][3]));
        }
        mx0 *= mul;
        mx1 *= mul;
        if (__any_sync(kFull, mx0 > m0 + kSlack || mx1 > m1 + kSlack)) {
#pragma unroll
            for (int d = 1; d < 4; d <<= 1) {
                mx0 = fmaxf(mx0, __shfl_xor_sync(kFull, mx0, d));
                mx1 = fmaxf(mx1, __shfl_xor_sync(kFull, mx1, d));
            }
            const float was0 = m0, was1 = m1;
            m0 = fmaxf(m0, mx0);
            m1 = fmaxf(m1, mx1);
            // a row with no visible key so far keeps m = -inf
            const float corr0 = was0 == -INFINITY ? 0.f : ex2(was0 - m0), corr1 = was1 == -INFINITY ? 0.f : ex2(was1 - m1);
            l0 *= corr0;
            l1 *= corr1;
#pragma unroll
            for (int nd = 0; nd < DH / 8; ++nd) {
                o[nd][0] *= corr0;
                o[nd][1] *= corr0;
                o[nd][2] *= corr1;
                o[nd][3] *= corr1;
            }
        }
        const float ref0 = m0 == -INFINITY ? 0.f : kLift - m0, ref1 = m1 == -INFINITY ? 0.f : kLift - m1;
        float la0 = 0.f, lb0 = 0.f, la1 = 0.f, lb1 = 0.f;
#pragma unroll
        for (int n = 0; n < kSlots / 8; ++n) {
            s[n][0] = ex2(fmaf(s[n][0], mul, ref0));
            s[n][1] = ex2(fmaf(s[n][1], mul, ref0));
            s[n][2] = ex2(fmaf(s[n][2], mul, ref1));
            s[n][3] = ex2(fmaf(s[n][3], mul, ref1));
            la0 += s[n][0];
            lb0 += s[n][1];
            la1 += s[n][2];
            lb1 += s[n][3];
        }
        l0 += la0 + lb0;
        l1 += la1 + lb1;
#pragma unroll
        for (int kk = 0; kk < kSlots / 16; ++kk) {
            const uint32_t pa[4] = {Half<T>::pack(s[2 * kk][0], s[2 * kk][1]), Half<T>::pack(s[2 * kk][2], s[2 * kk][3]),
                                    Half<T>::pack(s[2 * kk + 1][0], s[2 * kk + 1][1]),
                                    Half<T>::pack(s[2 * kk + 1][2], s[2 * kk + 1][3])};
#pragma unroll
            for (int dp = 0; dp < DH / 16; ++dp) {
                uint32_t b0, b1, b2, b3;
                ldmatrix_x4_trans(sv + at_v(kk, dp), b0, b1, b2, b3);
                Half<T>::mma(o[2 * dp], pa, b0, b1);
                Half<T>::mma(o[2 * dp + 1], pa, b2, b3);
            }
        }
        __syncthreads();   // every warp is done with this stage before it is refilled
    }

    if (TMA && !ok) {
        // the copies in flight land before the block leaves
        for (int e = max(0, n_tiles - 2); e < n_tiles; ++e) {
            const long long t0 = clock64();
            while (!rr::tc::mbar_test(&full[e & 1], (e >> 1) & 1) && clock64() - t0 < rr::tc::kSpinLimit) {
            }
        }
    }
    l0 += __shfl_xor_sync(kFull, l0, 1);
    l0 += __shfl_xor_sync(kFull, l0, 2);
    l1 += __shfl_xor_sync(kFull, l1, 1);
    l1 += __shfl_xor_sync(kFull, l1, 2);
    if (!ok) l0 = l1 = NAN;
    const float inv0 = l0 == 0.f ? 0.f : 1.f / l0, inv1 = l1 == 0.f ? 0.f : 1.f / l1;
    bool bad0 = false, bad1 = false;
#pragma unroll
    for (int nd = 0; nd < DH / 8; ++nd) {
        bad0 = bad0 || !isfinite(o[nd][0]) || !isfinite(o[nd][1]);
        bad1 = bad1 || !isfinite(o[nd][2]) || !isfinite(o[nd][3]);
    }
    // a row that saw nothing is zero whatever its accumulators hold
    T *out = static_cast<T *>(p.a.out) + u.b * p.c.out_stride[0] + head * p.c.out_stride[1];
    uint32_t *o0 = reinterpret_cast<uint32_t *>(out + token * p.c.out_stride[2]);
    uint32_t *o1 = reinterpret_cast<uint32_t *>(out + (token + 8) * p.c.out_stride[2]);
#pragma unroll
    for (int nd = 0; nd < DH / 8; ++nd) {
        if (ok0) o0[nd * 4 + t] = l0 == 0.f ? 0u : Half<T>::pack_mean(o[nd][0] * inv0, o[nd][1] * inv0);
        if (ok1) o1[nd * 4 + t] = l1 == 0.f ? 0u : Half<T>::pack_mean(o[nd][2] * inv1, o[nd][3] * inv1);
    }
    if (p.a.lse && t == 0) {
        float *lse = p.a.lse + ((size_t)u.b * p.c.q_heads + head) * p.c.nq_tokens + token;
        const float unit = bias ? p.a.slopes[head] : 0.f;
        if (ok0) lse[0] = l0 == 0.f ? -INFINITY : (m0 - kLift + log2f(l0)) * kLn2 - unit * (float)near0;
        if (ok1) lse[8] = l1 == 0.f ? -INFINITY : (m1 - kLift + log2f(l1)) * kLn2 - unit * (float)near1;
    }
    // rows to compute on their own, one bit for each of the warp's 16
    // (where the sum is a NaN, a score that the row sees is one, and so is the row)
    const unsigned b0 = __ballot_sync(kFull, bad0 && ok0 && l0 != 0.f && l0 == l0);
    const unsigned b1 = __ballot_sync(kFull, bad1 && ok1 && l1 != 0.f && l1 == l1);
    for (int r = 0; r < 16 && (b0 | b1); ++r) {
        if (!(((r < 8 ? b0 : b1) >> (4 * (r & 7))) & 15u)) continue;
        const int near = __shfl_sync(kFull, r < 8 ? near0 : near1, 4 * (r & 7));
        row_alone<T, DH>(p, u, s_list, n_list, row0 + r, near);
    }
}

template <typename T, int DH, bool TMA>
cudaError_t launch(const Masked &p, const TileMaps &maps, unsigned units, cudaStream_t s) {
    using S = Shape<DH, TMA>;
    auto kern = masked_attention_kernel<T, DH, TMA>;
    const int list = 4 * p.c.width;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = rr_attn::allow_smem(reinterpret_cast<const void *>(kern), S::kSmem + 4 * kMaxWidth, done);
    if (e != cudaSuccess) return e;
    const int warps = min(kMaxWarps, (p.group << p.shift) / 16);
    kern<<<units * (unsigned)p.tiles, 32 * warps, S::kSmem + list, s>>>(p, maps);
    return cudaGetLastError();
}

template <typename T, int DH>
cudaError_t launch_small(const Masked &p, unsigned units, cudaStream_t s) {
    const rr_masked_attn_config &c = p.c;
    TileMaps maps;
    const int box = c.chunk < 64 ? c.chunk : 64;
    if ((long long)units * c.width * c.chunk >= kTmaSlots &&
        tensor_map(p, p.a.k, c.nk_tokens, c.kv_heads, c.k_stride, box, &maps.k, &maps.axes[0]) &&
        tensor_map(p, p.a.v, c.nk_tokens, c.kv_heads, c.v_stride, box, &maps.v, &maps.axes[1]))
        return launch<T, DH, true>(p, maps, units, s);
    return launch<T, DH, false>(p, maps, units, s);
}

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

bool soft_cap_ok(float x) { return x == 0.f || (x >= 1e-3f && x <= 1e30f); }

// Strides of [batch, heads, tokens]; those of a size of one count nothing.
bool strides_ok(const int64_t (&s)[3], int batch, int heads, int tokens) {
    const int sizes[3] = {batch, heads, tokens};
    for (int i = 0; i < 3; ++i)
        if (sizes[i] > 1 && (s[i] < 0 || s[i] % 8 != 0 || s[i] > (1ll << 40))) return false;
    return true;
}
void drop_strides(int64_t (&s)[3], int batch, int heads, int tokens) {
    if (batch <= 1) s[0] = 0;
    if (heads <= 1) s[1] = 0;
    if (tokens <= 1) s[2] = 0;
}

bool config_ok(const rr_masked_attn_config *c) {
    if (!c) return false;
    if (c->batch < 0 || c->nq_tokens < 0 || c->nk_tokens < 0 || c->q_offset < 0) return false;
    if (c->kv_heads < 1 || c->route_heads < 1 || c->q_heads < 1) return false;
    if (c->route_heads % c->kv_heads != 0 || c->q_heads % c->route_heads != 0) return false;
    if (c->dh != 64 && c->dh != 128) return false;
    if (c->chunk != 16 && c->chunk != 32 && c->chunk != 64 && c->chunk != 128) return false;
    if (c->width < 0 || c->width > kMaxWidth || c->route_stride < (c->width > 1 ? c->width : 1)) return false;
    if (c->dtype != RR_BF16 && c->dtype != RR_F16) return false;
    if ((long long)c->q_offset + c->nq_tokens > 1 << 24 || c->nk_tokens > 1 << 24) return false;
    if (!(c->scale >= 0.f) || !isfinite(c->scale)) return false;
    if (!(c->scale <= 1e30f) || !soft_cap_ok(c->soft_cap)) return false;
    if (!strides_ok(c->q_stride, c->batch, c->q_heads, c->nq_tokens) ||
        !strides_ok(c->k_stride, c->batch, c->kv_heads, c->nk_tokens) ||
        !strides_ok(c->v_stride, c->batch, c->kv_heads, c->nk_tokens) ||
        !strides_ok(c->out_stride, c->batch, c->q_heads, c->nq_tokens))
        return false;
    const int32_t out_sizes[3] = {c->batch, c->q_heads, c->nq_tokens};
    if (!rr_attn::rows_apart(out_sizes, c->out_stride, 3, c->dh)) return false;
    const long long group = c->q_heads / c->route_heads, chunks = (c->nq_tokens + c->chunk - 1) / c->chunk;
    const long long heads = (long long)c->batch * c->route_heads, rows16 = group * c->chunk / 16;
    if (group * c->chunk > 1 << 24) return false;
    if (chunks > 0 && heads > 0x7fffffffLL / chunks) return false;
    if (heads * chunks > 0 && rows16 > 0x7fffffffLL / (heads * chunks)) return false;
    return true;
}

}  // namespace rr_masked

extern "C" rr_status rr_masked_attention(const rr_masked_attn_config *cfg, const rr_masked_attn_args *args,
                                         void *stream) {
    using namespace rr_masked;
    if (!config_ok(cfg) || !args) return RR_EINVAL;
    if (cfg->batch == 0 || cfg->nq_tokens == 0) return RR_OK;
    const rr_masked_attn_args &a = *args;
    if (!a.q || !a.out || !aligned(a.q, 16) || !aligned(a.out, 16)) return RR_EINVAL;
    if (cfg->width > 0 && (!a.route || !aligned(a.route, 4))) return RR_EINVAL;
    if (cfg->nk_tokens > 0 && (!a.k || !a.v || !aligned(a.k, 16) || !aligned(a.v, 16))) return RR_EINVAL;
    if (cfg->nk_tokens > 0 ? !a.doc_q != !a.doc_k : a.doc_k && !a.doc_q) return RR_EINVAL;
    if (!aligned(a.slopes, 4) || !aligned(a.doc_q, 4) || !aligned(a.doc_k, 4) || !aligned(a.prefix, 4) ||
        !aligned(a.lse, 4))
        return RR_EINVAL;
    Masked p;
    p.c = *cfg;
    drop_strides(p.c.q_stride, cfg->batch, cfg->q_heads, cfg->nq_tokens);
    drop_strides(p.c.k_stride, cfg->batch, cfg->kv_heads, cfg->nk_tokens);
    drop_strides(p.c.v_stride, cfg->batch, cfg->kv_heads, cfg->nk_tokens);
    drop_strides(p.c.out_stride, cfg->batch, cfg->q_heads, cfg->nq_tokens);
    p.a = a;
    p.group = cfg->q_heads / cfg->route_heads;
    p.shift = cfg->chunk == 16 ? 4 : cfg->chunk == 32 ? 5 : cfg->chunk == 64 ? 6 : 7;
    p.nqc = (cfg->nq_tokens + cfg->chunk - 1) >> p.shift;
    p.nkc = (cfg->nk_tokens + cfg->chunk - 1) >> p.shift;
    const float scale = cfg->scale > 0.f ? cfg->scale : 1.0f / sqrtf((float)cfg->dh);
    p.s1 = cfg->soft_cap > 0.f ? scale / cfg->soft_cap : scale * kLog2e;
    p.s2 = cfg->soft_cap * kLog2e;
    p.tiles = ((p.group << p.shift) + 16 * kMaxWarps - 1) / (16 * kMaxWarps);
    const unsigned units = (unsigned)((long long)cfg->batch * cfg->route_heads * p.nqc);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = launch_tc(p, units, s);
    if (e != cudaErrorNotSupported) return e == cudaSuccess ? RR_OK : RR_ECUDA;
    if (cfg->dtype == RR_BF16)
        e = cfg->dh == 64 ? launch_small<__nv_bfloat16, 64>(p, units, s) : launch_small<__nv_bfloat16, 128>(p, units, s);
    else
        e = cfg->dh == 64 ? launch_small<__half, 64>(p, units, s) : launch_small<__half, 128>(p, units, s);
    return e == cudaSuccess ? RR_OK : RR_ECUDA;
}

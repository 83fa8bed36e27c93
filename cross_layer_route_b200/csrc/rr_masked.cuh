// rr_masked.cuh -- what the kernels of the masked attention share (declared in
// include/rr_attention.h): the problem, the list of a unit's key chunks, the
// masks, and the row that is computed on its own.
//
// A unit is one query chunk of one route head: the `group` query heads that
// share the route (and therefore the key head) times the chunk's tokens, rows
// numbered head * chunk + token.  All of its rows read the same key chunks.
#pragma once

#include <cuda.h>
#include <limits.h>
#include <math.h>

#include "../../include/rr_attention.h"
#include "rr_frag.cuh"

namespace rr_masked {

using rr_attn::Half;
using rr_attn::kFull;
using rr_attn::kMaxWidth;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kChunkFull = 1 << 30;   // list flag: every key of the chunk is visible to every row
constexpr int kChunkCut = 1 << 29;    // ... its documents differ from row to row or key to key
constexpr int kChunkId = kChunkCut - 1;

struct Masked {
    rr_masked_attn_config c;
    rr_masked_attn_args a;
    int group;        // query heads per route head
    int shift;        // log2(chunk)
    int nqc, nkc;     // query and key chunks
    int tiles;        // row tiles per unit
    // scores in base 2: x log2(e) = s * s1 without a cap, s2 * tanh(s * s1) with one
    float s1, s2;
};

struct Unit {
    int b, route_head, i, tile;   // batch entry, route head, query chunk, row tile
    int kv_head;
    int tokens;                   // valid query tokens of the chunk
    int p_first, p_last;          // positions of its first and last valid token
    int prefix;                   // keys below it are visible under causal
};

__device__ __forceinline__ Unit unit_of(const Masked &p, unsigned block) {
    Unit u;
    u.tile = (int)(block % (unsigned)p.tiles);
    unsigned r = block / (unsigned)p.tiles;
    u.i = (int)(r % (unsigned)p.nqc);
    r /= (unsigned)p.nqc;
    u.route_head = (int)(r % (unsigned)p.c.route_heads);
    u.b = (int)(r / (unsigned)p.c.route_heads);
    u.kv_head = u.route_head / (p.c.route_heads / p.c.kv_heads);
    u.tokens = min(p.c.chunk, p.c.nq_tokens - (u.i << p.shift));
    u.p_first = p.c.q_offset + (u.i << p.shift);
    u.p_last = u.p_first + u.tokens - 1;
    u.prefix = p.a.prefix ? p.a.prefix[u.b] : 0;
    return u;
}

// Smallest and largest of n <= 128 int32 at x: this lane's part.
__device__ __forceinline__ void lane_min_max(const int32_t *x, int n, int &lo, int &hi) {
    lo = INT_MAX;
    hi = INT_MIN;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = (threadIdx.x & 31) + 32 * i;
        if (e < n) {
            const int v = x[e];
            lo = min(lo, v);
            hi = max(hi, v);
        }
    }
}

// The threads that build a list together: all of a block, or two warps of it.
struct BlockTeam {
    __device__ __forceinline__ int rank() const { return threadIdx.x; }
    __device__ __forceinline__ int size() const { return blockDim.x; }
    __device__ __forceinline__ void sync() const { __syncthreads(); }
};
template <int FIRST, int THREADS, int BARRIER>
struct PartTeam {
    __device__ __forceinline__ int rank() const { return threadIdx.x - FIRST; }
    __device__ __forceinline__ int size() const { return THREADS; }
    __device__ __forceinline__ void sync() const { asm volatile("bar.sync %0, %1;" ::"n"(BARRIER), "n"(THREADS) : "memory"); }
};

// The unit's route in shared memory: list[0..n-1] = key chunks that can hold a
// visible key, in route order, kChunkFull set where all of their keys are
// visible to all rows (neither the masks nor the last chunk's end cut them),
// kChunkCut where the documents cut them.
// By a team; ends with its barrier.
template <typename Team>
__device__ __forceinline__ int build_list(const Team team, const Masked &p, const Unit &u, int32_t *list, int32_t *n_out) {
    const int warp = team.rank() >> 5, lane = threadIdx.x & 31, warps = team.size() >> 5;
    const int32_t *route =
        p.a.route + (((size_t)u.b * p.c.route_heads + u.route_head) * p.nqc + u.i) * (size_t)p.c.route_stride;
    const int width = p.c.width;
    const bool causal = p.c.causal != 0, docs = p.a.doc_q != nullptr;
    for (int e = team.rank(); e < width; e += team.size()) {
        int j = route[e];
        if (j < 0 || j >= p.nkc) j = -1;
        if (j >= 0) {
            const int lo = j << p.shift, hi = min(lo + p.c.chunk, p.c.nk_tokens);
            bool full = hi - lo == p.c.chunk;
            if (causal) {
                if (lo > u.p_last && lo >= u.prefix) j = -1;
                full = full && (hi - 1 <= u.p_first || hi <= u.prefix);
            }
            if (j >= 0 && full) j |= kChunkFull;
        }
        list[e] = j;
    }
    int qlo = 0, qhi = 0;
    if (docs) lane_min_max(p.a.doc_q + (size_t)u.b * p.c.nq_tokens + (u.i << p.shift), u.tokens, qlo, qhi);
    team.sync();
    if (docs) {
        // documents are mostly runs of tokens: a chunk of one document is either
        // visible to a query chunk of one document as a whole or not at all
        qlo = __reduce_min_sync(kFull, qlo);
        qhi = __reduce_max_sync(kFull, qhi);
        constexpr int kAtOnce = 4;     // entries whose loads are in flight together
        for (int e0 = warp * kAtOnce; e0 < width; e0 += warps * kAtOnce) {
            int j[kAtOnce], klo[kAtOnce], khi[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                j[i] = e0 + i < width ? list[e0 + i] : -1;
                const int lo = j[i] < 0 ? 0 : (j[i] & kChunkId) << p.shift;
                lane_min_max(p.a.doc_k + (size_t)u.b * p.c.nk_tokens + lo,
                             j[i] < 0 ? 0 : min(p.c.chunk, p.c.nk_tokens - lo), klo[i], khi[i]);
            }
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                klo[i] = __reduce_min_sync(kFull, klo[i]);
                khi[i] = __reduce_max_sync(kFull, khi[i]);
                if (lane == 0 && j[i] >= 0) {
                    if (khi[i] < 0 || qhi < 0 || khi[i] < qlo || klo[i] > qhi) list[e0 + i] = -1;
                    else if (klo[i] != khi[i] || qlo != qhi) list[e0 + i] = (j[i] & ~kChunkFull) | kChunkCut;
                }
            }
        }
        team.sync();
    }
    if (warp == 0) {
        int n = 0;
        for (int e0 = 0; e0 < width; e0 += 32) {
            const int j = e0 + lane < width ? list[e0 + lane] : -1;
            const unsigned m = __ballot_sync(kFull, j >= 0);
            __syncwarp();
            if (j >= 0) list[n + __popc(m & ((1u << lane) - 1u))] = j;
            n += __popc(m);
            __syncwarp();
        }
        if (lane == 0) *n_out = n;
    }
    team.sync();
    return *n_out;
}

// Key s against a query at position pos: the causal rule with its exception.
__device__ __forceinline__ bool in_sight(const Masked &p, int prefix, int pos, int s) {
    return p.c.causal == 0 || s <= pos || s < prefix;
}

// Distance from a row to the nearest key that it sees, among list entries
// first, first + step, ... (INT_MAX: none).  The bias is taken relative to it,
// so that a row whose keys are all far away keeps the bits of its scores: at
// distance 2^20 a product slope * distance in fp32 has a step of 1/16.
__device__ __forceinline__ int nearest(const Masked &p, const Unit &u, const int32_t *list, int n, int pos, int doc,
                                       int first, int step) {
    int best = INT_MAX;
    for (int e = first; e < n; e += step) {
        const int lo = (list[e] & kChunkId) << p.shift;
        int hi = min(lo + p.c.chunk, p.c.nk_tokens);
        if (p.c.causal) hi = min(hi, max(pos + 1, u.prefix));
        if (hi <= lo) continue;
        const int d = pos < lo ? lo - pos : pos >= hi ? pos - (hi - 1) : 0;
        if (d >= best) continue;
        if (!(list[e] & kChunkCut)) {
            best = d;
        } else {
            const int32_t *dk = p.a.doc_k + (size_t)u.b * p.c.nk_tokens;
            for (int s = lo; s < hi; ++s)
                if (dk[s] == doc) best = min(best, abs(pos - s));
        }
    }
    return best;
}

// One row computed by a warp on the CUDA cores, reading only what it sees: the way
// out for a row whose accumulators hold an infinity or a NaN.  There a masked value
// row that holds one has met a weight of zero in the matrix product, or the row's
// own result is not finite; both end here with the right values.  32 keys at a time:
// a lane scores one, then the warp adds their values, a lane DH / 32 dims.  Measured:
// 610 cycles a key at dh 128 and 380 at dh 64, in all 0.2 s for a warp's 32 rows of
// 16384 keys and 1.3 s for 131072, the most that a route holds.
// `row` numbers the unit's rows.
template <typename T, int DH>
__device__ __forceinline__ void row_alone(const Masked &p, const Unit &u, const int32_t *list, int n, int row, int near) {
    constexpr int E = DH / 32;
    const int lane = threadIdx.x & 31;
    __syncwarp();     // other lanes have stored the row that is stored anew below
    const int head = u.route_head * p.group + (row >> p.shift), token = (u.i << p.shift) + (row & (p.c.chunk - 1));
    const int pos = p.c.q_offset + token;
    const T *q = static_cast<const T *>(p.a.q) + u.b * p.c.q_stride[0] + head * p.c.q_stride[1] + token * p.c.q_stride[2];
    const T *k = static_cast<const T *>(p.a.k) + u.b * p.c.k_stride[0] + u.kv_head * p.c.k_stride[1];
    const T *v = static_cast<const T *>(p.a.v) + u.b * p.c.v_stride[0] + u.kv_head * p.c.v_stride[1] + lane * E;
    const int doc = p.a.doc_q ? p.a.doc_q[(size_t)u.b * p.c.nq_tokens + token] : 0;
    const float slope = p.a.slopes ? p.a.slopes[head] * kLog2e : 0.f;
    // weights of at most 2^-18, of at most 2^17 keys: their sums with finite values are finite
    // (the least, 2^-126 before, does not become zero: it may be an infinity's)
    constexpr float kSmall = 1.f / (1 << 18);
    static_assert(kMaxWidth * 128 <= 1 << 17, "keys of a route");
    float o[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 1
    for (int slot0 = 0; slot0 < n << p.shift; slot0 += 32) {
        const int slot = slot0 + lane;
        const int s = slot < n << p.shift ? ((list[slot >> p.shift] & kChunkId) << p.shift) + (slot & (p.c.chunk - 1))
                                          : INT_MAX;
        bool see = s < p.c.nk_tokens && in_sight(p, u.prefix, pos, s);
        if (see && p.a.doc_q) see = doc >= 0 && p.a.doc_k[(size_t)u.b * p.c.nk_tokens + s] == doc;
        float x = -INFINITY;
        if (see) {
            x = 0.f;
#pragma unroll 1
            for (int c = 0; c < DH; c += 8) {
                const uint4 kw = *reinterpret_cast<const uint4 *>(k + s * p.c.k_stride[2] + c);
                const uint4 qw = *reinterpret_cast<const uint4 *>(q + c);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x += Half<T>::up(reinterpret_cast<const T *>(&qw)[e]) * Half<T>::up(reinterpret_cast<const T *>(&kw)[e]);
            }
            x *= p.s1;
            if (p.c.soft_cap > 0.f) x = p.s2 * rr_attn::tanh_f32(x);
            if (p.a.slopes) x -= slope * (float)(abs(pos - s) - near);
        }
        float top = x;
#pragma unroll
        for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
        const float mn = fmaxf(m, top), base = mn == -INFINITY ? 0.f : mn;
        const float corr = rr_attn::ex2(m - base), w = rr_attn::ex2(x - base) * kSmall;
        m = mn;
        float sum = w;
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
        l = l * corr + sum;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= corr;
        unsigned seen = __ballot_sync(kFull, see);
#pragma unroll 1
        while (seen) {
            const int from = __ffs(seen) - 1;
            seen &= seen - 1;
            const float wk = __shfl_sync(kFull, w, from);
            const T *vk = v + __shfl_sync(kFull, s, from) * p.c.v_stride[2];
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] += wk * Half<T>::up(vk[e]);
        }
    }
    T *out = static_cast<T *>(p.a.out) + u.b * p.c.out_stride[0] + head * p.c.out_stride[1] +
             token * p.c.out_stride[2] + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) out[e] = Half<T>::down(l == 0.f ? 0.f : o[e] / l);
}

// Tensor map of [batch, heads, tokens, dh] by strides, in boxes of tokens by 64
// elements (rr_masked_tc.cu); false where these strides have none.
bool tensor_map(const Masked &p, const void *x, int tokens, int heads, const int64_t (&stride)[3], int box_tokens,
                CUtensorMap *map, int *axes);

// The kernel on tcgen05 (rr_masked_tc.cu); cudaErrorNotSupported, and nothing
// launched, for problems that are not for it.
cudaError_t launch_tc(const Masked &p, unsigned units, cudaStream_t s);

}  // namespace rr_masked

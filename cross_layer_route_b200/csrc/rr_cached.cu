// rr_cached.cu -- attention of a sequence's newest tokens over the paged cache
// (declared in include/rr_cache.h).
//
// A CTA takes some of one sequence's tokens (cut_of says how many) for one key head
// and up to 8 NT rows (query token, query head) that read it; its warps take pairs
// of 16 tokens in turn, each with its own running softmax, so nothing in the loop
// waits for another warp.  Both products put the cache on the 16-row side of
// mma.sync m16n8k16, where none of it is wasted on padding:
//   S^T = K Q^T   A = 16 tokens x 16 dims.  A lane's 16-byte read of a token's row
//                 holds dims that need not be the ones of the standard fragment:
//                 the query fragments use the same order.
//   O^T = V^T P^T A = 16 dims x 16 tokens.  A lane holds 4 tokens' bytes of the
//                 same dims; bytes of two tokens are paired with prmt.
// Codes become f16 exactly.  The scales are powers of two: a row's goes to its
// score (keys) or its weight (values).  With one for every 32 elements, a key's
// groups are summed one by one in fp32, and a value's codes are multiplied by
// their group's scale over the row's largest, exact down to 2^-35.
// Weights are f16 and relative to the largest weight * scale seen so far, which
// stands at 2^7 (and at 2^15 before it is noticed), so neither a wide spread of
// scales nor a long tail of small weights is lost; the sum of the weights is
// fp32 and not rounded.  That reference is kept relative to the running maximum
// of the scores: a score of 2^24 or more would swallow a scale added to it.
// The references move only when a score passes them by 2^8: most steps then
// cost one vote and no shuffles.
// A warp copies its steps (cp.async) into a ring of its own, one or two pairs ahead.
//
// Measured on a B200: 64 sequences of up to 12001 tokens (8 heads of 128, 4 queries
// each, e4m3, 1.06 GB of cache) 217 us, 4.9 TB/s of the 6.5 a copy reaches.  The
// memory alone would take 164 us, the loop without its copies 150: the 64
// conversions and 50 shifts and permutations that a step of 16 tokens needs share
// one half-rate pipe, which is busy half of the time.  In 4 bits a step has half
// the bytes and more of those (scales of 32 elements), so there the pipe is the
// bound: 16 sequences of 128 routed chunks of 64 tokens, 142 MB, 72 us.  Measured
// and not kept: 16 warps with single steps (237 us), shifts as products' upper
// halves on the other pipe (223 us, in 4 bits 12 % slower), two sums per score.
#include <cooperative_groups.h>
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
constexpr int kAttnWarps = 6;
constexpr int kJoinWarps = 4;
constexpr int kMaxCluster = 8;   // blocks of a cluster
constexpr float kLift = 7.f;     // weights are 2^7 at the maximum
constexpr float kSlack = 8.f;    // ... and 2^15 at most
constexpr int kGroupLift = 12;   // codes of 4 bits carry 2^12
constexpr int kState = 4;        // floats beside a partial row: max, sum, value reference, nearest

// CTAs per SM: what 128 O values a thread and the other fragments leave room for.
constexpr int ctas_per_sm(int dh, int nt) { return nt * dh <= 128 ? 2 : 1; }

// How the work is cut.  A job is a sequence's tokens for a key head and a row block.
// kOne: a CTA takes a job.  kCluster: a cluster of CTAs takes a job, kSplits: so do
// CTAs that leave their parts in the workspace.  kShares: all jobs' steps, laid end
// to end, are cut into equal shares, one per CTA; a share ends in the middle of a
// job and may hold several.  The caller counts the CTAs from the page table's width;
// sequences that are far shorter can leave fewer steps than CTAs, which then take one
// each (shares_of), so that no share is empty and a job's shares are neighbours.
enum { kOne, kCluster, kSplits, kShares };
constexpr int kMaxShared = 512;  // sequences of a call cut into shares

struct Cached {
    rr_cache_config c;
    rr_cache_pool pool;
    rr_cached_attn_config n;
    rr_cached_attn_args a;
    float *part;       // [parts, 8 NT rows, dh + kState], with splits or shares
    int shift;         // log2(chunk)
    int group, rows;   // query heads per key head, rows per key head
    int mode;
    int blocks;        // CTAs that share a job (cluster, splits), or all jobs (shares)
    int zs;            // row blocks of 8 NT rows per key head
    float s1, s2;      // as in the masked attention
};

template <int FMT, int DH>
struct Words {
    static constexpr int kK = FMT == RR_E4M3 ? DH / 16 : DH / 32;   // 32-bit words of one key row a lane holds
    static constexpr int kV = FMT == RR_E4M3 ? DH / 32 : DH / 64;
    static constexpr int kRowBytes = FMT == RR_E4M3 ? DH : DH / 2;
    static constexpr int kGroups = FMT == RR_E4M3 ? 1 : DH / 32;
    // A step (16 tokens of a page) in shared memory: keys, values, their scales.
    static constexpr int kSide = 16 * kRowBytes;
    static constexpr int kScales = 16 * kGroups;
    static constexpr int kStage = 2 * kSide + 2 * kScales;
    // pairs of steps that a warp's ring holds, one of them in use: twelve warps on
    // an SM then have 100 KB of copies in flight
    static constexpr int kPairs = kRowBytes == 128 ? 2 : 3;
    static constexpr int kRing = kPairs * 2 * kStage;
};

// Byte offset of 16-byte piece `c` of row `r` in a step's keys or values.  Rows
// lie in lines of 128 bytes, whose eight pieces are permuted so that the lanes
// that read together meet eight different pieces: a key row's pieces by the
// lanes of a token or (one piece of each group of 32 elements) by all tokens, a
// value row's by the lanes of a dim range for tokens 2t.
template <int ROW, bool VALUES>
__device__ __forceinline__ int piece_at(int r, int c) {
    constexpr int kPer = 128 / ROW;                  // rows per line
    const int line = r / kPer, at = (r % kPer) * (ROW / 16) + c;
    const int turn = VALUES ? 2 * ((ROW == 128 ? line >> 1 : line) & 3) : ROW == 128 ? 4 * (line & 1) : line & 3;
    return line * 128 + ((at ^ turn) << 4);
}

// Starts the copy of one step: 16 tokens from row `krow` of the pool on.  Values
// behind the sequence's end are whatever the page held, and a NaN code there
// would meet a weight of zero in the product: zeros in their place.  pos < 0:
// all zeros.  `kat`, `vat`: this lane's first pieces.
template <int FMT, int DH>
__device__ __forceinline__ void copy_step(uint32_t stage, uint32_t kat, uint32_t vat, const Cached &p, size_t krow,
                                          int pos, int len) {
    using W = Words<FMT, DH>;
    constexpr int kPieces = W::kSide / 16, kCopies = (kPieces + 31) / 32;
    const int lane = threadIdx.x & 31;
    const unsigned char *codes = static_cast<const unsigned char *>(p.pool.codes) + krow * W::kRowBytes + 16 * lane;
    const unsigned char *values = codes + p.c.chunk * W::kRowBytes;
    const int side = lane / W::kGroups, c = lane % W::kGroups;
    const unsigned char *scales =
        static_cast<const unsigned char *>(p.pool.scales) + (krow + side * p.c.chunk) * W::kGroups + 16 * c;
    const uint32_t sat = stage + 2 * W::kSide + side * W::kScales + 16 * c;
    // piece lane + 32 i lies 512 i behind the lane's first; the values' pieces of
    // rows of 128 bytes change places every four rows
    const uint32_t vodd = W::kRowBytes == 128 ? vat ^ 64 : vat;
    if (pos >= 0 && pos + 16 <= len) {
        if (kPieces >= 32 || lane < kPieces) {
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                cp_async16(stage + kat + 512 * i, codes + 512 * i);
                cp_async16(stage + W::kSide + (i & 1 ? vodd : vat) + 512 * i, values + 512 * i);
            }
        }
        if (lane < 2 * W::kGroups) cp_async16(sat, scales);
    } else {
        const int left = pos < 0 ? 0 : len - pos;
        if (kPieces >= 32 || lane < kPieces) {
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                const int r = (lane + 32 * i) / (W::kRowBytes / 16);
                cp_async16_zfill(stage + kat + 512 * i, codes + 512 * i, left ? 16 : 0);
                cp_async16_zfill(stage + W::kSide + (i & 1 ? vodd : vat) + 512 * i, values + 512 * i, r < left ? 16 : 0);
            }
        }
        if (lane < 2 * W::kGroups) cp_async16_zfill(sat, scales, left ? 16 : 0);
    }
}

template <int N>
__device__ __forceinline__ void read_words(uint32_t (&w)[N], const unsigned char *x) {
    if constexpr (N == 4) {
        const uint4 a = *reinterpret_cast<const uint4 *>(x);
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    } else if constexpr (N == 2) {
        const uint2 a = *reinterpret_cast<const uint2 *>(x);
        w[0] = a.x, w[1] = a.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t *>(x);
    }
}

// Key words of token r, lane quarter t: of the 16-byte pieces t and t + 4, or of
// piece t; with a scale for every 32 elements word t of each group's piece, so
// that one k-step stays within one group.
template <int FMT, int DH>
__device__ __forceinline__ void read_key(uint32_t (&w)[Words<FMT, DH>::kK], const unsigned char *stage, int r, int t) {
    using W = Words<FMT, DH>;
    if constexpr (FMT == RR_E2M1) {
#pragma unroll
        for (int j = 0; j < W::kGroups; ++j)
            w[j] = *reinterpret_cast<const uint32_t *>(stage + piece_at<W::kRowBytes, false>(r, j) + 4 * t);
    } else {
        uint32_t a[4];
#pragma unroll
        for (int h = 0; h < W::kK / 4; ++h) {
            read_words(a, stage + piece_at<W::kRowBytes, false>(r, t + 4 * h));
#pragma unroll
            for (int j = 0; j < 4; ++j) w[4 * h + j] = a[j];
        }
    }
}

template <int FMT, int DH>
__device__ __forceinline__ void read_value(uint32_t (&w)[Words<FMT, DH>::kV], const unsigned char *stage, int r, int g) {
    using W = Words<FMT, DH>;
    const int at = 4 * W::kV * g;
    read_words(w, stage + W::kSide + piece_at<W::kRowBytes, true>(r, at / 16) + at % 16);
}

template <int FMT, int DH>
__device__ __forceinline__ uint32_t read_scales(const unsigned char *stage, int side, int r) {
    using W = Words<FMT, DH>;
    const unsigned char *x = stage + 2 * W::kSide + side * W::kScales + r * W::kGroups;
    if constexpr (W::kGroups == 1) return *x;
    else if constexpr (W::kGroups == 2) return *reinterpret_cast<const uint16_t *>(x);
    else return *reinterpret_cast<const uint32_t *>(x);
}

// Two codes (the low 16 or 8 bits) as f16.
__device__ __forceinline__ uint32_t f16x2_of_e4m3(uint32_t two) {
    uint32_t d;
    asm("{.reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.rn.f16x2.e4m3x2 %0, lo;}" : "=r"(d) : "r"(two));
    return d;
}
__device__ __forceinline__ uint32_t f16x2_of_e2m1(uint32_t two) {
    uint32_t d;
    asm("{.reg .b8 x, y, z, w; mov.b32 {x, y, z, w}, %1; cvt.rn.f16x2.e2m1x2 %0, x;}" : "=r"(d) : "r"(two));
    return d;
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

// Largest of a row's scale bytes, NaN (255) among them.
template <int G>
__device__ __forceinline__ unsigned top_scale(uint32_t w) {
    if constexpr (G == 1) return w;
    const unsigned m = __vmaxu2(w & 0x00ff00ffu, (w >> 8) & 0x00ff00ffu);
    return G == 2 ? m & 0xffffu : max(m & 0xffffu, m >> 16);
}
// The same without the NaN bytes (0 if all are).
template <int G>
__device__ __forceinline__ unsigned top_number(uint32_t w) {
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < G; ++i) {
        const unsigned b = (w >> (8 * i)) & 255;
        m = max(m, b == 255 ? 0u : b);
    }
    return m;
}
// 2^(byte - top + kGroupLift) in f16; zero below 2^-24 and for NaN bytes.
__device__ __forceinline__ uint32_t group_factor(unsigned byte, unsigned top) {
    const int e = (int)byte - (int)top + kGroupLift;
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

// Steps of 16 tokens of a sequence.
__device__ __forceinline__ int steps_of(const Cached &p, int b) {
    const int len = p.a.seq_lens[b];
    const int entries = len <= 0 ? 0 : p.a.route ? p.n.width : min(p.n.table_width, ((len - 1) >> p.shift) + 1);
    return entries << (p.shift - 4);
}

// prefix[i] = steps of the sequences before i, for i in [0, batch], by the block.
__device__ __forceinline__ void sum_steps(const Cached &p, int *prefix) {
    for (int i = threadIdx.x; i < p.n.batch; i += blockDim.x) prefix[1 + i] = steps_of(p, i);
    __syncthreads();
    if (threadIdx.x < 32) {
        int sum = 0;
        for (int i = threadIdx.x; i - (int)threadIdx.x < p.n.batch; i += 32) {
            int x = i < p.n.batch ? prefix[1 + i] : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int y = __shfl_up_sync(kFull, x, d);
                if ((int)threadIdx.x >= d) x += y;
            }
            if (i < p.n.batch) prefix[1 + i] = sum + x;
            sum += __shfl_sync(kFull, x, 31);
        }
        if (threadIdx.x == 0) prefix[0] = 0;
    }
    __syncthreads();
}

// The shares that a call of `total` steps is cut into.
__device__ __forceinline__ int shares_of(const Cached &p, long long total) { return (int)min((long long)p.blocks, total); }

// Two dims of one row's result from its sums: o relative to 2^(n2 - kLift) of the
// weights', their sum to 2^n1; dim 0's caller writes lse.
template <int DH>
__device__ __forceinline__ void write_out(const Cached &p, int b, int head, int row, int dim, float x, float y, float n1,
                                          float sum, float n2, float near) {
    const bool none = sum == 0.f;
    // (the power in two factors: values' scales reach down to 2^-127, in 4 bits another
    // kGroupLift below, and ex2 has no results below 2^-126)
    const float half = ex2(0.5f * (n2 - kLift)), f = half / sum;
    x = none ? 0.f : x * f * half;
    y = none ? 0.f : y * f * half;
    const size_t orow = ((size_t)b * p.n.q_tokens + row / p.group) * p.n.q_heads + head * p.group + row % p.group;
    static_cast<uint32_t *>(p.a.out)[(orow * DH + dim) / 2] = p.n.dtype == RR_BF16 ? pack_bf16(x, y) : pack_f16(x, y);
    if (p.a.lse && dim == 0)
        p.a.lse[orow] = none ? -INFINITY
                             : (n1 + log2f(sum)) * kLn2 -
                                   (p.a.slopes ? p.a.slopes[head * p.group + row % p.group] * near : 0.f);
}

// The ring's memory, which also takes the warps' states when they are joined.
template <int FMT, int DH, int NT>
__host__ __device__ constexpr int joined_bytes() {
    const int ring = kAttnWarps * Words<FMT, DH>::kRing, states = kAttnWarps * 32 * (DH / 16 * 4 * NT + 6 * NT) * 4;
    return ring > states ? ring : states;
}

template <int FMT, int DH, int NT>
__global__ void __launch_bounds__(32 * kAttnWarps, ctas_per_sm(DH, NT))
cached_attention_kernel(const __grid_constant__ Cached p) {
    using W = Words<FMT, DH>;
    constexpr int kRows = 8 * NT, kQRow = DH + 4;      // padded query rows: lanes 8 banks apart
    constexpr int kMT = DH / 16;                       // 16-dim tiles of the values
    constexpr int kKeep = kMT * 4 * NT + 6 * NT;       // floats of a warp's state per lane
    constexpr int kGap = 16;
    extern __shared__ __align__(16) unsigned char smem[];
    __half *s_q = reinterpret_cast<__half *>(smem);                                   // [kRows][kQRow]
    float *s_row = reinterpret_cast<float *>(smem + kRows * kQRow * 2);               // [kRows] score factor
    int *s_near = reinterpret_cast<int *>(s_row + kRows);
    unsigned char *s_ring = smem + kRows * kQRow * 2 + kRows * 4 + kGap;    // [warps][stages][stage]
    float *s_merge = reinterpret_cast<float *>(s_ring);                               // after the loop
    float *s_part = reinterpret_cast<float *>(s_ring + joined_bytes<FMT, DH, NT>());  // [kRows][DH + kState]

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    int *s_prefix = reinterpret_cast<int *>(s_part + kRows * (DH + kState));          // [batch + 1], with shares
    long long cur = 0, stop = 0;                       // this share, in steps of all jobs
    if (p.mode == kShares) {
        sum_steps(p, s_prefix);
        const long long total = (long long)s_prefix[p.n.batch] * p.c.heads * p.zs;
        const int shares = shares_of(p, total);
        if ((int)blockIdx.x >= shares) return;
        cur = total * blockIdx.x / shares;
        stop = total * (blockIdx.x + 1) / shares;
    }
    const int sub_shift = p.shift - 4;                 // steps per chunk
    for (;;) {
        int head, b, row0, begin, end, job = 0;
        if (p.mode == kShares) {
            // the job that step `cur` is in: heads and row blocks of sequence b one after another
            const int hz = p.c.heads * p.zs;
            int lo = 0, hi = p.n.batch - 1;                // the last b whose first step is not behind cur
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if ((long long)s_prefix[mid] * hz <= cur) lo = mid;
                else hi = mid - 1;
            }
            b = lo;
            const int steps = s_prefix[b + 1] - s_prefix[b];
            const long long off = cur - (long long)s_prefix[b] * hz;
            const int in_b = (int)(off / steps);
            begin = (int)(off % steps);
            end = (int)min((long long)steps, begin + (stop - cur));
            head = in_b / p.zs;
            row0 = in_b % p.zs * kRows;
            job = b * hz + in_b;
        } else {
            head = blockIdx.y % p.c.heads;
            b = blockIdx.y / p.c.heads;
            row0 = blockIdx.z * kRows;
            // (the grid: blocks of a job, sequences and heads, row blocks)
            job = (blockIdx.y * p.zs + blockIdx.z) * p.blocks;
            const long long all = steps_of(p, b);
            begin = (int)(all * blockIdx.x / gridDim.x);
            end = (int)(all * (blockIdx.x + 1) / gridDim.x);
        }
        const int len = p.a.seq_lens[b];
        const int32_t *table = p.a.page_table + (size_t)b * p.n.table_stride;
        const int32_t *route = p.a.route ? p.a.route + ((size_t)b * p.c.heads + head) * p.n.route_stride : nullptr;
        const int entries = len <= 0 ? 0 : route ? p.n.width : min(p.n.table_width, ((len - 1) >> p.shift) + 1);

        // A warp takes pairs of steps, begin + 2 warp on and every 2 kAttnWarps after
        // that; lane i looks up the page of the i-th of 32 steps.
        const int mine = begin + 2 * warp < end ? (end - begin - 2 * warp + 2 * kAttnWarps - 1) / (2 * kAttnWarps) : 0;
        int pos_l = -1;
        size_t row_l = 0;
        const uint32_t ring = smem_u32(s_ring) + warp * W::kRing;
        uint32_t fill = ring;                              // the pair filled next
        const int first_row = lane / (W::kRowBytes / 16), first_piece = lane % (W::kRowBytes / 16);
        const uint32_t kat = piece_at<W::kRowBytes, false>(first_row, first_piece);
        const uint32_t vat = piece_at<W::kRowBytes, true>(first_row, first_piece);
        int queue[W::kPairs][2];                           // positions of the steps in flight, oldest first
        auto fetch = [&](int i) {
            if (i < mine) {
                if ((i & 15) == 0) {
                    pos_l = -1;
                    row_l = 0;
                    const int step = begin + 2 * (warp + (i + (lane >> 1)) * kAttnWarps) + (lane & 1);
                    if (step < end) {
                        const int entry = step >> sub_shift;
                        const int id = route ? route[entry] : entry;
                        if (id >= 0 && id < p.n.table_width) {
                            const int at = (id << p.shift) + ((step & ((1 << sub_shift) - 1)) << 4);
                            const int page = at < len ? table[id] : -1;
                            if (page >= 0 && page < p.c.pages) {
                                pos_l = at;
                                row_l = ((size_t)page * p.c.heads + head) * 2 * p.c.chunk + (at & (p.c.chunk - 1));
                            }
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int from = 2 * (i & 15) + u;
                    const int pos = __shfl_sync(kFull, pos_l, from);
                    const size_t row = __shfl_sync(kFull, row_l, from);
                    queue[W::kPairs - 1][u] = pos;
                    copy_step<FMT, DH>(fill + u * W::kStage, kat, vat, p, row, pos, len);
                }
                fill = fill == ring + W::kRing - 2 * W::kStage ? ring : fill + 2 * W::kStage;
            }
            cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < W::kPairs - 1; ++i) {
            fetch(i);
            queue[i][0] = queue[W::kPairs - 1][0];
            queue[i][1] = queue[W::kPairs - 1][1];
        }

        // queries: eight lanes a row, DH / 8 elements each
        for (int r = warp * 4 + lane / 8; r < kRows; r += kAttnWarps * 4) {
            const int row = row0 + r, at8 = (lane & 7) * (DH / 8);
            float x[DH / 8];
            unsigned amax = 0;
#pragma unroll
            for (int i = 0; i < DH / 8; i += 8) {
                uint4 w = make_uint4(0u, 0u, 0u, 0u);
                if (row < p.rows) {
                    const int64_t at = b * p.n.q_stride[0] + (row / p.group) * p.n.q_stride[1] +
                                       (head * p.group + row % p.group) * p.n.q_stride[2] + at8 + i;
                    w = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.a.q) + at));
                }
                const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = p.n.dtype == RR_BF16 ? __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&h[e]))
                                                          : __half22float2(*reinterpret_cast<const __half2 *>(&h[e]));
                    x[i + 2 * e] = f.x;
                    x[i + 2 * e + 1] = f.y;
                    amax = max(amax, max(__float_as_uint(f.x) & 0x7fffffffu, __float_as_uint(f.y) & 0x7fffffffu));
                }
            }
            const unsigned group_mask = 0xffu << (lane & 24);
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) amax = max(amax, __shfl_xor_sync(group_mask, amax, d));
            const int shift = query_shift(amax);
            // 2^shift in two factors: a shift can be as large as 162
            const float half0 = __uint_as_float((unsigned)(127 + shift / 2) << 23);
            const float half1 = __uint_as_float((unsigned)(127 + shift - shift / 2) << 23);
#pragma unroll
            for (int i = 0; i < DH / 8; i += 2)
                *reinterpret_cast<uint32_t *>(s_q + r * kQRow + at8 + i) = pack_f16(x[i] * half0 * half1, x[i + 1] * half0 * half1);
            if ((lane & 7) == 0) s_row[r] = ldexpf(p.s1, -shift);
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
            const int dim = FMT == RR_E2M1 ? 32 * (j / 2) + 8 * t + 4 * (j % 2) : 64 * (j / 4) + 16 * t + 4 * (j % 4);
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

        const unsigned char *stage = s_ring + warp * W::kRing, *last_pair = stage + W::kRing - 2 * W::kStage;
        const int all_see = len - p.n.q_tokens;            // positions up to here are visible to every row
        for (int i = 0; i < mine; ++i, stage = stage == last_pair ? stage - (W::kRing - 2 * W::kStage) : stage + 2 * W::kStage) {
            __syncwarp();     // every lane is done with the pair that is filled now
            fetch(i + W::kPairs - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(W::kPairs - 1) : "memory");
            __syncwarp();
            const int pos[2] = {queue[0][0], queue[0][1]};
#pragma unroll
            for (int j = 0; j + 1 < W::kPairs; ++j) queue[j][0] = queue[j + 1][0], queue[j][1] = queue[j + 1][1];
            if (pos[0] < 0 && pos[1] < 0) continue;

            // S^T: tokens g, g + 8 of each step by rows 2t, 2t + 1
            float s[2][NT][4];
            uint32_t vs[2][2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const unsigned char *st = stage + u * W::kStage;
                uint32_t ks[2], k0[W::kK], k1[W::kK];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    ks[h] = read_scales<FMT, DH>(st, 0, g + 8 * h);
                    vs[u][h] = read_scales<FMT, DH>(st, 1, g + 8 * h);
                }
                read_key<FMT, DH>(k0, st, g, t);
                read_key<FMT, DH>(k1, st, g + 8, t);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) s[u][nt][0] = s[u][nt][1] = s[u][nt][2] = s[u][nt][3] = 0.f;
                if constexpr (FMT == RR_E4M3) {
#pragma unroll
                    for (int j = 0; j < DH / 16; ++j) {
                        const uint32_t a[4] = {f16x2_of_e4m3(k0[j]), f16x2_of_e4m3(k1[j]), f16x2_of_e4m3(k0[j] >> 16),
                                               f16x2_of_e4m3(k1[j] >> 16)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            uint32_t b0, b1;
                            if constexpr (NT <= 2) b0 = qf[nt][j][0], b1 = qf[nt][j][1];
                            else query(nt, j, b0, b1);
                            mma_f16(s[u][nt], a, b0, b1);
                        }
                    }
                    const float kf[2] = {power_of_two(ks[0]), power_of_two(ks[1])};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 4; ++c) s[u][nt][c] = s[u][nt][c] * rowf[nt][c & 1] * kf[c >> 1];
                } else {
                    // each group's part of the score by the group's scale
#pragma unroll
                    for (int grp = 0; grp < W::kGroups; ++grp) {
                        float part[NT][4];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) part[nt][0] = part[nt][1] = part[nt][2] = part[nt][3] = 0.f;
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t w0 = k0[grp] >> (16 * j), w1 = k1[grp] >> (16 * j);
                            const uint32_t a[4] = {f16x2_of_e2m1(w0), f16x2_of_e2m1(w1), f16x2_of_e2m1(w0 >> 8),
                                                   f16x2_of_e2m1(w1 >> 8)};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                uint32_t b0, b1;
                                if constexpr (NT <= 2) b0 = qf[nt][2 * grp + j][0], b1 = qf[nt][2 * grp + j][1];
                                else query(nt, 2 * grp + j, b0, b1);
                                mma_f16(part[nt], a, b0, b1);
                            }
                        }
                        const float kf[2] = {power_of_two((ks[0] >> (8 * grp)) & 255), power_of_two((ks[1] >> (8 * grp)) & 255)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int c = 0; c < 4; ++c) s[u][nt][c] = fmaf(part[nt][c], kf[c >> 1], s[u][nt][c]);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 4; ++c) s[u][nt][c] *= rowf[nt][c & 1];
                }
            }

            // The values' scales: the exponent ev that goes to a token's weight, and with
            // groups the f16 factors of this lane's dims.  NaN scales and groups 2^26 below
            // their row's largest are rare, and looked at once per step.
            float ev[2][2];
            uint32_t vf[2][2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if constexpr (FMT == RR_E4M3) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) ev[u][h] = vs[u][h] == 255 ? NAN : (float)((int)vs[u][h] - 127);
                } else {
                    const int grp8 = (DH == 128 ? g / 2 : g / 4) * 8;
                    unsigned top[2] = {top_scale<W::kGroups>(vs[u][0]), top_scale<W::kGroups>(vs[u][1])};
                    const uint32_t both = top[0] | top[1] << 16;
                    const int from = 8 * t;                // the lane of token 2t; of 2t + 1: from + 4
                    const uint32_t w0 = __shfl_sync(kFull, vs[u][0], from), w1 = __shfl_sync(kFull, vs[u][0], from + 4);
                    const uint32_t w2 = __shfl_sync(kFull, vs[u][1], from), w3 = __shfl_sync(kFull, vs[u][1], from + 4);
                    const uint32_t ta = __shfl_sync(kFull, both, from), tb = __shfl_sync(kFull, both, from + 4);
                    const int f0 = (int)((w0 >> grp8) & 255) - (int)(ta & 0xffffu) + kGroupLift + 15;
                    const int f1 = (int)((w1 >> grp8) & 255) - (int)(tb & 0xffffu) + kGroupLift + 15;
                    const int f2 = (int)((w2 >> grp8) & 255) - (int)(ta >> 16) + kGroupLift + 15;
                    const int f3 = (int)((w3 >> grp8) & 255) - (int)(tb >> 16) + kGroupLift + 15;
                    vf[u][0] = (uint32_t)f0 << 10 | (uint32_t)f1 << 26;
                    vf[u][1] = (uint32_t)f2 << 10 | (uint32_t)f3 << 26;
                    if (__any_sync(kFull, min(min(f0, f1), min(f2, f3)) < 1 || max(top[0], top[1]) == 255)) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
#pragma unroll
                            for (int grp = 0; grp < W::kGroups; ++grp)
                                if (pos[u] >= 0 && ((vs[u][h] >> (8 * grp)) & 255) == 255)
#pragma unroll
                                    for (int r = 0; r < 2 * NT; ++r)
                                        if (pos[u] + g + 8 * h <= pos_r[r >> 1][r & 1]) broken |= 1u << (r * W::kGroups + grp);
                            top[h] = top_number<W::kGroups>(vs[u][h]);
                        }
                        vf[u][0] = group_factor((w0 >> grp8) & 255, top_number<W::kGroups>(w0)) |
                                   group_factor((w1 >> grp8) & 255, top_number<W::kGroups>(w1)) << 16;
                        vf[u][1] = group_factor((w2 >> grp8) & 255, top_number<W::kGroups>(w2)) |
                                   group_factor((w3 >> grp8) & 255, top_number<W::kGroups>(w3)) << 16;
                    }
                    ev[u][0] = (float)((int)top[0] - 127 - kGroupLift);
                    ev[u][1] = (float)((int)top[1] - 127 - kGroupLift);
                }
            }

            // scores in base 2 and their masks; c: token g + 8 (c >> 1), row c & 1
            if (cap) {
                // tanh by its polynomial alone while no score of the warp reaches the cap
                float most = 0.f;
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 4; ++c) most = fmaxf(most, fabsf(s[u][nt][c]));
                const bool within = __all_sync(kFull, most < 1.f);
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        if (within) {
                            tanh_pair(s[u][nt], 1.f);
                            tanh_pair(s[u][nt] + 2, 1.f);
                        } else {
#pragma unroll
                            for (int c = 0; c < 4; ++c) s[u][nt][c] = tanh_f32(s[u][nt][c]);
                        }
#pragma unroll
                        for (int c = 0; c < 4; ++c) s[u][nt][c] *= p.s2;
                    }
            }
            if (bias) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            s[u][nt][c] -= slope[nt][c & 1] *
                                           (float)(pos_r[nt][c & 1] - near_r[nt][c & 1] - pos[u] - g - 8 * (c >> 1));
            }
            if (max(pos[0], pos[1]) + 15 > all_see || min(pos[0], pos[1]) < 0) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            if (pos[u] < 0 || pos[u] + g + 8 * (c >> 1) > pos_r[nt][c & 1]) s[u][nt][c] = -INFINITY;
            }
            // A masked score is -inf: its weights are zero and it moves no reference
            // whatever its value's scale, a NaN too.
            const float top_ev = fmaxf(fmaxf(ev[0][0], ev[0][1]), fmaxf(ev[1][0], ev[1][1]));
            bool grow = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    // (an upper bound of the tokens' sums: at worst a move that was not needed)
                    const float a = fmaxf(fmaxf(s[0][nt][r], s[0][nt][2 + r]), fmaxf(s[1][nt][r], s[1][nt][2 + r]));
                    grow = grow || a - m1[nt][r] > fminf(kSlack, m2[nt][r] + kSlack - top_ev);
                }
            if (__any_sync(kFull, grow)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float a = fmaxf(m1[nt][r], fmaxf(fmaxf(s[0][nt][r], s[0][nt][2 + r]), fmaxf(s[1][nt][r], s[1][nt][2 + r])));
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) a = fmaxf(a, __shfl_xor_sync(kFull, a, d));
                        const float base = a == -INFINITY ? 0.f : a, down = m1[nt][r] - base;
                        float c = fmaxf(fmaxf(s[0][nt][r] - base + ev[0][0], s[0][nt][2 + r] - base + ev[0][1]),
                                        fmaxf(s[1][nt][r] - base + ev[1][0], s[1][nt][2 + r] - base + ev[1][1]));
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) c = fmaxf(c, __shfl_xor_sync(kFull, c, d));
                        const float was = m2[nt][r] + down;
                        c = fmaxf(c, was);
                        l[nt][r] *= ex2(down);
                        const float corr = c == -INFINITY ? 1.f : ex2(was - c);
                        m1[nt][r] = a;
                        m2[nt][r] = c;
#pragma unroll
                        for (int i2 = 0; i2 < kMT; ++i2) {
                            o[i2][nt][r] *= corr;
                            o[i2][nt][2 + r] *= corr;
                        }
                    }
            }

#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const unsigned char *st = stage + u * W::kStage;
                // weights: P^T fragments by transposing 8x8 blocks
                uint32_t pb[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float w[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int r = c & 1;
                        // -inf - -inf: a row that has seen nothing yet
                        const bool none = s[u][nt][c] == -INFINITY;
                        const float x = s[u][nt][c] - m1[nt][r];
                        l[nt][r] += none ? 0.f : ex2(x);
                        w[c] = none ? 0.f : ex2(x + (ev[u][c >> 1] - m2[nt][r] + kLift));
                    }
                    pb[nt][0] = transpose_8x8(pack_f16(w[0], w[1]));
                    pb[nt][1] = transpose_8x8(pack_f16(w[2], w[3]));
                }

                // O^T: dims (DH / 8) g + 2 i (rows g) and + 1 (rows g + 8) of tile i
                uint32_t v[4][W::kV];
#pragma unroll
                for (int q = 0; q < 4; ++q) read_value<FMT, DH>(v[q], st, 2 * t + (q & 1) + 8 * (q >> 1), g);
#pragma unroll
                for (int j = 0; j < W::kV; ++j) {
                    if constexpr (FMT == RR_E4M3) {
                        const uint32_t x0 = __byte_perm(v[0][j], v[1][j], 0x5140), x1 = __byte_perm(v[2][j], v[3][j], 0x5140);
                        const uint32_t y0 = __byte_perm(v[0][j], v[1][j], 0x7362), y1 = __byte_perm(v[2][j], v[3][j], 0x7362);
                        const uint32_t a[4] = {f16x2_of_e4m3(x0), f16x2_of_e4m3(x0 >> 16), f16x2_of_e4m3(x1),
                                               f16x2_of_e4m3(x1 >> 16)};
                        const uint32_t c[4] = {f16x2_of_e4m3(y0), f16x2_of_e4m3(y0 >> 16), f16x2_of_e4m3(y1),
                                               f16x2_of_e4m3(y1 >> 16)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_f16(o[2 * j][nt], a, pb[nt][0], pb[nt][1]);
                            mma_f16(o[2 * j + 1][nt], c, pb[nt][0], pb[nt][1]);
                        }
                    } else {
                        // byte i of a row holds dims 2i (low half) and 2i + 1
                        const uint32_t lo0 = (v[0][j] & 0x0f0f0f0fu) | (v[1][j] & 0x0f0f0f0fu) << 4;
                        const uint32_t hi0 = ((v[0][j] >> 4) & 0x0f0f0f0fu) | (v[1][j] & 0xf0f0f0f0u);
                        const uint32_t lo1 = (v[2][j] & 0x0f0f0f0fu) | (v[3][j] & 0x0f0f0f0fu) << 4;
                        const uint32_t hi1 = ((v[2][j] >> 4) & 0x0f0f0f0fu) | (v[3][j] & 0xf0f0f0f0u);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint32_t a[4] = {mul_f16x2(f16x2_of_e2m1(lo0 >> (8 * q)), vf[u][0]),
                                                   mul_f16x2(f16x2_of_e2m1(hi0 >> (8 * q)), vf[u][0]),
                                                   mul_f16x2(f16x2_of_e2m1(lo1 >> (8 * q)), vf[u][1]),
                                                   mul_f16x2(f16x2_of_e2m1(hi1 >> (8 * q)), vf[u][1])};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma_f16(o[4 * j + q][nt], a, pb[nt][0], pb[nt][1]);
                        }
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

        // The warps' results, joined through the ring's memory: every warp leaves
        // its state, and takes (tile of dims, tile of rows) pairs to join.
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
#if __CUDA_ARCH__ >= 900
        cudaTriggerProgrammaticLaunchCompletion();
#endif
        {
            float *at = s_merge + warp * 32 * kKeep + lane;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int i = 0; i < kMT; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) at[32 * ((nt * kMT + i) * 4 + c)] = o[i][nt][c];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float *st = at + 32 * (NT * kMT * 4 + nt * 6 + 3 * r);
                    st[0] = m1[nt][r];
                    st[32] = m2[nt][r];
                    st[64] = l[nt][r];
                }
            }
        }
        __syncthreads();
        for (int pair = warp; pair < kMT * NT; pair += kAttnWarps) {
            const int nt = pair / kMT, i = pair % kMT;
            const float *at = s_merge + lane;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = row0 + nt * 8 + 2 * t + r;
                if (row >= p.rows) continue;
                const float *st = at + 32 * (NT * kMT * 4 + nt * 6 + 3 * r), *os = at + 32 * (pair * 4 + r);
                float a[kAttnWarps], c[kAttnWarps], n1 = -INFINITY, n2 = -INFINITY;
#pragma unroll
                for (int w = 0; w < kAttnWarps; ++w) {
                    a[w] = st[w * 32 * kKeep];
                    n1 = fmaxf(n1, a[w]);
                }
                const float b1 = n1 == -INFINITY ? 0.f : n1;
#pragma unroll
                for (int w = 0; w < kAttnWarps; ++w) {
                    a[w] -= b1;
                    c[w] = st[w * 32 * kKeep + 32] + a[w];
                    n2 = fmaxf(n2, c[w]);
                }
                const float b2 = n2 == -INFINITY ? 0.f : n2;
                float sum = 0.f, x = 0.f, y = 0.f;
#pragma unroll
                for (int w = 0; w < kAttnWarps; ++w) {
                    const float f = ex2(c[w] - b2);
                    sum += st[w * 32 * kKeep + 64] * ex2(a[w]);
                    x += os[w * 32 * kKeep] * f;
                    y += os[w * 32 * kKeep + 64] * f;
                }
                const int dim = (DH / 8) * g + 2 * i;
                const int back = p.n.q_tokens - 1 - row / p.group, near = max(0, *s_near - back);
                if (p.mode != kOne) {
                    // a part's number is share + job: both grow, one at a time; with splits
                    // job * blocks + split
                    float *part = (p.mode == kCluster ? s_part : p.part + (size_t)(blockIdx.x + job) * kRows * (DH + kState)) +
                                  (row - row0) * (DH + kState);
                    *reinterpret_cast<float2 *>(part + dim) = make_float2(x, y);
                    if (g == 0 && i == 0) *reinterpret_cast<float4 *>(part + DH) = make_float4(n1, sum, n2, (float)near);
                } else {
                    write_out<DH>(p, b, head, row, dim, x, y, n1, sum, n2, (float)near);
                }
            }
        }
        if (p.mode == kShares) {
            cur += end - begin;
            if (cur >= stop) return;
            __syncthreads();      // the block is done with this job's queries and sums
            continue;
        }
        if (p.mode != kCluster) return;
        // The blocks that share these tokens are a cluster: each joins a part of the
        // results out of all blocks' shared memory.
        cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
        cluster.sync();
        const int valid = min(kRows, p.rows - row0);
        for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < valid * (DH / 2); i += gridDim.x * blockDim.x) {
            const int r = i / (DH / 2), dim = i % (DH / 2) * 2;
            float n1 = -INFINITY, n2 = -INFINITY, near = 0.f;
            float4 st[kMaxCluster];
            float2 xy[kMaxCluster];
#pragma unroll
            for (int s = 0; s < kMaxCluster; ++s) {
                if (s < p.blocks) {
                    const float *at = cluster.map_shared_rank(s_part, s) + r * (DH + kState);
                    st[s] = *reinterpret_cast<const float4 *>(at + DH);
                    xy[s] = *reinterpret_cast<const float2 *>(at + dim);
                    n1 = fmaxf(n1, st[s].x);
                    near = st[s].w;
                }
            }
            const float b1 = n1 == -INFINITY ? 0.f : n1;
#pragma unroll
            for (int s = 0; s < kMaxCluster; ++s) {
                if (s < p.blocks) {
                    st[s].x -= b1;
                    st[s].z += st[s].x;
                    n2 = fmaxf(n2, st[s].z);
                }
            }
            const float b2 = n2 == -INFINITY ? 0.f : n2;
            float sum = 0.f, x = 0.f, y = 0.f;
#pragma unroll
            for (int s = 0; s < kMaxCluster; ++s) {
                if (s < p.blocks) {
                    const float f = ex2(st[s].z - b2);
                    sum += st[s].y * ex2(st[s].x);
                    x += xy[s].x * f;
                    y += xy[s].y * f;
                }
            }
            write_out<DH>(p, b, head, row0 + r, dim, x, y, n1, sum, n2, near);
        }
        cluster.sync();      // no block leaves while its memory is read
        return;
    }
}

// Joins the parts of one row: a block per row, its warps take parts in turn, a lane
// DH / 32 dims.  Launched while the attention's last blocks still run (its results
// are waited for below), which hides the launch.
template <int DH, int NT>
__global__ void __launch_bounds__(32 * kJoinWarps) cached_join_kernel(const __grid_constant__ Cached p) {
    constexpr int E = DH / 32, kRows = 8 * NT;
    __shared__ float s_o[kJoinWarps][DH], s_l[kJoinWarps];
    __shared__ int s_prefix[kMaxShared + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int bh = blockIdx.x / p.rows, row = blockIdx.x % p.rows, head = bh % p.c.heads, b = bh / p.c.heads;
    const int hz = p.c.heads * p.zs, in_b = head * p.zs + row / kRows;
    int parts = p.blocks;
    size_t part = (size_t)(b * hz + in_b) * p.blocks;      // its first
    if (p.mode == kShares) {
        sum_steps(p, s_prefix);
        const int steps = s_prefix[b + 1] - s_prefix[b];
        const long long total = (long long)s_prefix[p.n.batch] * hz, first = (long long)s_prefix[b] * hz + (long long)in_b * steps;
        // the shares that the job's first and last step are in
        const int shares = shares_of(p, total);
        const int c0 = steps ? (int)(((first + 1) * shares - 1) / total) : 0;
        parts = steps ? (int)(((first + steps) * shares - 1) / total) - c0 + 1 : 0;
        part = (size_t)c0 + b * hz + in_b;
    }
    const float *at = p.part + (part * kRows + row % kRows) * (DH + kState);
    const size_t stride = (size_t)kRows * (DH + kState);
#if __CUDA_ARCH__ >= 900
    cudaGridDependencySynchronize();
#endif
    float n1 = -INFINITY, n2 = -INFINITY;
    for (int s = lane; s < parts; s += 32) n1 = fmaxf(n1, at[s * stride + DH]);
#pragma unroll
    for (int d = 16; d; d >>= 1) n1 = fmaxf(n1, __shfl_xor_sync(kFull, n1, d));
    const float b1 = n1 == -INFINITY ? 0.f : n1;
    for (int s = lane; s < parts; s += 32) n2 = fmaxf(n2, at[s * stride + DH + 2] + (at[s * stride + DH] - b1));
#pragma unroll
    for (int d = 16; d; d >>= 1) n2 = fmaxf(n2, __shfl_xor_sync(kFull, n2, d));
    const float b2 = n2 == -INFINITY ? 0.f : n2;
    float l = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 4
    for (int s = warp; s < parts; s += kJoinWarps) {
        const float *x = at + s * stride;
        const float4 st = *reinterpret_cast<const float4 *>(x + DH);
        float v[E];
        if constexpr (E == 4) *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(x + lane * 4);
        else *reinterpret_cast<float2 *>(v) = *reinterpret_cast<const float2 *>(x + lane * 2);
        l += st.y * ex2(st.x - b1);
        const float f = ex2(st.z + (st.x - b1) - b2);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += v[e] * f;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
    if (lane == 0) s_l[warp] = l;
    __syncthreads();
    if (threadIdx.x >= DH / 2) return;
    const int d = 2 * threadIdx.x;
    float x = 0.f, y = 0.f;
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
        l += s_l[w];
        x += s_o[w][d];
        y += s_o[w][d + 1];
    }
    write_out<DH>(p, b, head, row, d, x, y, n1, l, n2, parts ? at[DH + 3] : 0.f);
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
    const int sizes[3] = {n->batch, n->q_tokens, n->q_heads};
    for (int i = 0; i < 3; ++i) {
        const int64_t x = n->q_stride[i];
        if (sizes[i] > 1 && (x < 0 || x % 8 != 0 || x > (1ll << 40))) return false;
    }
    return true;
}

// Tiles of 8 rows that a CTA takes at once, sharing the codes' conversion.  At dh 128
// four of them fill the registers (one CTA per SM either way), so two are better
// where four would stand half empty or few CTAs leave the SMs to latency: 16
// sequences of up to 8000 tokens, 8 heads: 32 rows 148 us by fours and 165 by twos,
// 40 rows 261 and 211; one such sequence, 32 rows: 39 and 30.  At dh 64 two CTAs of
// twos fit an SM and one of fours, and the warps that hide latency are worth more than
// the conversions: the same three by twos 73, 99 and 18.5 us, by fours 80, 137 and 21
// (by ones 99, 120 and 20.5; three CTAs of twos spill: 109, 149 and 27).
int tiles_of(const rr_cache_config *c, const rr_cached_attn_config *n) {
    const int rows = n->q_heads / c->heads * n->q_tokens, twos = (rows + 15) / 16;
    if (rows <= 8) return 1;
    return c->dh == 128 && twos % 2 == 0 && (long long)n->batch * c->heads * twos > 148 ? 4 : 2;
}

// The cut of a call (above) with the least cost, in steps.  A job costs its steps and
// a start and an end worth about 24; CTAs come in waves of 148 SMs.  Sequences are
// taken to have three quarters of the table's length on average, and all of a
// route's.  Parts in the workspace take a second launch, for caller and GPU together
// about 36 steps, and shares, which are even whatever the lengths, 12 more for every
// CTA to find its own.  A cluster needs no second launch, but clusters do not pack,
// so they are for at most half the SMs.  Measured, with 8 heads and up to 751 steps:
// 24 sequences by splits 105 us, by shares 91; 64 sequences 217 and 222; with 2 heads
// and 188 steps, 24 sequences in clusters of 3 26.6 us, by 3 splits 22.5, by shares 27;
// with 8 heads and 256 steps, one sequence in a cluster 11.3 us and 15 with the
// caller's share, by splits 12.7 and 20.
struct Cut {
    int mode, blocks, zs;
};
Cut cut_of(const rr_cache_config *c, const rr_cached_attn_config *n, bool route) {
    const long long rows = (long long)(n->q_heads / c->heads) * n->q_tokens;
    const int nt = tiles_of(c, n), slots = 148 * ctas_per_sm(c->dh, nt);
    const int zs = (int)((rows + 8 * nt - 1) / (8 * nt));
    const long long jobs = (long long)n->batch * c->heads * zs;
    const double steps = (double)(route ? n->width : n->table_width) * (c->chunk / 16), fill = route ? 1.0 : 0.75;
    Cut best = {kOne, 1, zs};
    if (jobs == 0) return best;
    double least = 1e300;
    const long long tried = 4 * slots / jobs + 1;
    for (int s = 1; s == 1 || (s <= tried && steps / s >= 2 * kAttnWarps); ++s) {
        const double one = steps / s + 24.0, waves = (double)jobs * s / slots;
        double cost = waves <= 1.0 ? one : ((fill * waves > 1.0 ? fill * waves : 1.0) + 0.4) * one;
        int mode = s == 1 ? kOne : kCluster;
        if (s > kMaxCluster || (s > 1 && jobs * s > 74)) mode = kSplits, cost += 36.0;
        if (cost < least) least = cost, best = {mode, s, zs};
    }
    // (sums of steps are int)
    const double work = fill * jobs * steps;
    const int shares = work / (2 * kAttnWarps) < slots ? (int)(work / (2 * kAttnWarps)) : slots;
    if (n->batch <= kMaxShared && n->batch * steps < 1e9 && shares > 1 &&
        work / shares + 24.0 * (1.0 + (double)jobs / shares) + 48.0 < least)
        best = {kShares, shares, zs};
    return best;
}

size_t part_bytes(const rr_cache_config *c, const rr_cached_attn_config *n, const Cut &cut) {
    const size_t jobs = (size_t)n->batch * c->heads * cut.zs;
    const size_t parts = cut.mode == kSplits ? jobs * cut.blocks : cut.mode == kShares ? jobs + cut.blocks : 0;
    return parts * 8 * tiles_of(c, n) * (c->dh + kState) * sizeof(float);
}

template <int FMT, int DH, int NT>
cudaError_t launch(const Cached &p, cudaStream_t s) {
    const int most = 8 * NT * (DH + 4) * 2 + 8 * NT * 4 + 16 + joined_bytes<FMT, DH, NT>() + 8 * NT * (DH + kState) * 4 +
                     4 * (kMaxShared + 1);
    const int smem = most - (p.mode == kShares ? 4 * (kMaxShared - p.n.batch) : 4 * (kMaxShared + 1));
    auto kern = cached_attention_kernel<FMT, DH, NT>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = rr_attn::allow_smem(reinterpret_cast<const void *>(kern), most, done);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    cudaLaunchConfig_t config = {};
    config.blockDim = dim3(32 * kAttnWarps);
    config.dynamicSmemBytes = smem;
    config.stream = s;
    config.attrs = &attr;
    config.gridDim = p.mode == kShares ? dim3(p.blocks) : dim3(p.blocks, p.n.batch * p.c.heads, p.zs);
    if (p.mode == kCluster) {
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = p.blocks;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        config.numAttrs = 1;
    }
    e = cudaLaunchKernelEx(&config, kern, p);
    if (e != cudaSuccess || p.mode < kSplits) return e;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    config.numAttrs = 1;
    config.gridDim = dim3((unsigned)p.n.batch * p.c.heads * p.rows);
    config.blockDim = dim3(32 * kJoinWarps);
    config.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&config, cached_join_kernel<DH, NT>, p);
}

template <int FMT, int DH>
cudaError_t launch_rows(const Cached &p, cudaStream_t s) {
    switch (tiles_of(&p.c, &p.n)) {
        case 1: return launch<FMT, DH, 1>(p, s);
        case 4:
            if constexpr (DH == 128) return launch<FMT, DH, 4>(p, s);
    }
    return launch<FMT, DH, 2>(p, s);
}

}  // namespace rr_cache

extern "C" size_t rr_cached_attention_workspace_bytes(const rr_cache_config *cfg, const rr_cached_attn_config *attn,
                                                      int32_t routed) {
    using namespace rr_cache;
    if (!config_ok(cfg, attn)) return 0;
    return part_bytes(cfg, attn, cut_of(cfg, attn, routed != 0));
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
    const Cut cut = cut_of(cfg, attn, a.route != nullptr);
    const size_t need = part_bytes(cfg, attn, cut);
    if (need > 0 && (!workspace || !aligned(workspace, 256))) return RR_EINVAL;
    if (workspace_bytes < need) return RR_ENOMEM;
    Cached p;
    p.c = *cfg;
    p.pool = *pool;
    p.n = *attn;
    if (attn->batch == 1) p.n.q_stride[0] = 0;
    if (attn->q_tokens == 1) p.n.q_stride[1] = 0;
    if (attn->q_heads == 1) p.n.q_stride[2] = 0;
    p.a = a;
    p.part = static_cast<float *>(workspace);
    p.shift = chunk_shift(cfg->chunk);
    p.group = attn->q_heads / cfg->heads;
    p.rows = p.group * attn->q_tokens;
    p.mode = cut.mode;
    p.blocks = cut.blocks;
    p.zs = cut.zs;
    const float scale = attn->scale > 0.f ? attn->scale : 1.0f / sqrtf((float)cfg->dh);
    p.s1 = attn->soft_cap > 0.f ? scale / attn->soft_cap : scale * kLog2e;
    p.s2 = attn->soft_cap * kLog2e;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (cfg->format == RR_E4M3) e = cfg->dh == 64 ? launch_rows<RR_E4M3, 64>(p, s) : launch_rows<RR_E4M3, 128>(p, s);
    else e = cfg->dh == 64 ? launch_rows<RR_E2M1, 64>(p, s) : launch_rows<RR_E2M1, 128>(p, s);
    return e == cudaSuccess ? RR_OK : RR_ECUDA;
}

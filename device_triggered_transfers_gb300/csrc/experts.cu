// Tokens' rows sorted by the experts that a rank holds, and back with weights, and their gradients (dtt_ops.h has
// the definitions).
//
// The sort is a counting sort, stable and without atomics whose order could show: each warp counts a run of its
// own, and places it once the sums before it are known.  The row kernels go by tokens, so that a token's row is
// read once for all of its choices (dispatch, combine_backward) or written once (combine), and gradients of a
// token's several rows are added without atomics.
#include <algorithm>
#include <cstdint>

#include "dtt_ops.h"
#include "internal.h"
#include "rowio.cuh"

namespace dtt {
namespace {

// Whether a thread gives an item of the ring up: a build of its own shows that the results stay the same.
#ifndef DTT_EXPERTS_LATE
#define DTT_EXPERTS_LATE false
#endif
// And whether the fetching warp gives up its wait for the oldest item.
#ifndef DTT_EXPERTS_FETCH_LATE
#define DTT_EXPERTS_FETCH_LATE false
#endif
constexpr uint32_t kMostExperts = 1024, kMostChoices = 32;
constexpr uint32_t kRouteThreads = 512, kRouteWarps = kRouteThreads / 32;
// 131072 pairs: 198 us with their rows' dispatch, with half as many parts 201, a quarter 206.
constexpr uint32_t kMostParts = 128;           // CTAs of the sort, at most
constexpr uint32_t kPartPairs = 1024;          // pairs of a CTA, at least, while there are fewer
// A row's threads, at most.  131072 rows of 4096 (bf16) combined: 209 us with 256 (four CTAs an SM), 224 with 512 (two),
// 211 with 128 (eight); backward 402, 450, 411.
constexpr uint32_t kCopyThreads = 256, kRowThreads = 256;
constexpr uint32_t kFillRows = 8;              // rows of one CTA where an expert's rows are filled up

struct RouteParams {
    const void* ids;
    int32_t* position;
    int32_t* offsets;
    int32_t* counts;
    uint32_t* parts;            // [gridDim.x][experts]: each CTA's pairs of each expert
    uint64_t pairs, each;       // each: of a CTA, a multiple of kRouteThreads
    uint32_t experts, first, align, max_rows;
    uint32_t wide;              // ids of 64 bits
};

// The expert of pair i as the rank counts them, `experts` where it is another rank's, or none.
__device__ __forceinline__ uint32_t expert_of(const RouteParams& p, uint64_t i) {
    const int64_t id = p.wide ? reinterpret_cast<const int64_t*>(p.ids)[i] : reinterpret_cast<const int32_t*>(p.ids)[i];
    const uint64_t e = (uint64_t)id - p.first;                 // below: wraps to a large number
    return id >= 0 && e < p.experts ? (uint32_t)e : p.experts;
}

// The warp's run of pairs, 32 neighbours at a time in their order: each(i, e, same), e the expert of the lane's pair i
// (`experts` from `to` on), same the lanes that share it.  Experts of kAhead times 32 pairs are loaded together.
constexpr uint32_t kAhead = 4;
template <class F>
__device__ __forceinline__ void walk_run(const RouteParams& p, uint64_t from, uint64_t to, F each) {
    const uint32_t lane = threadIdx.x % 32;
    for (uint64_t i0 = from; i0 < to; i0 += 32 * kAhead) {
        uint32_t e[kAhead];
#pragma unroll
        for (uint32_t k = 0; k < kAhead; ++k) {
            const uint64_t i = i0 + 32 * k + lane;
            e[k] = i < to ? expert_of(p, i) : p.experts;
        }
#pragma unroll
        for (uint32_t k = 0; k < kAhead; ++k) each(i0 + 32 * k + lane, e[k], __match_any_sync(0xFFFFFFFFu, e[k]));
    }
}

// How many of the run each expert has: mine[e], zero before.  Pairs of 32 neighbours that share an expert are counted by
// the first of them.
__device__ __forceinline__ void count_run(const RouteParams& p, uint64_t from, uint64_t to, uint32_t* mine) {
    walk_run(p, from, to, [&](uint64_t, uint32_t e, uint32_t same) {
        if (e < p.experts && threadIdx.x % 32 == __ffs(same) - 1) mine[e] += __popc(same);
        __syncwarp();
    });
}

__global__ void __launch_bounds__(kRouteThreads) route_count_kernel(const __grid_constant__ RouteParams p) {
    launch_next();
    wait_previous();
    extern __shared__ uint32_t counts[];           // [kRouteWarps][experts]
    const uint32_t t = threadIdx.x, warp = t / 32;
    for (uint32_t i = t; i < kRouteWarps * p.experts; i += kRouteThreads) counts[i] = 0;
    __syncthreads();
    const uint64_t run = p.each / kRouteWarps, from = blockIdx.x * p.each + warp * run;
    count_run(p, min(from, p.pairs), min(from + run, p.pairs), counts + warp * p.experts);
    __syncthreads();
    for (uint32_t e = t; e < p.experts; e += kRouteThreads) {
        uint32_t sum = 0;
        for (uint32_t w = 0; w < kRouteWarps; ++w) sum += counts[w * p.experts + e];
        p.parts[(uint64_t)blockIdx.x * p.experts + e] = sum;
    }
}

// Exclusive sums over the experts' rows: n = experts values at `v`, in place; `carry`: 32 words.
__device__ __forceinline__ void scan_experts(uint32_t* v, uint32_t n, uint32_t* carry) {
    const uint32_t t = threadIdx.x, lane = t % 32, warp = t / 32;
    constexpr uint32_t per = kMostExperts / kRouteThreads;
    uint32_t x[per], sum = 0;
#pragma unroll
    for (uint32_t k = 0; k < per; ++k) {
        x[k] = per * t + k < n ? v[per * t + k] : 0;
        sum += x[k];
    }
    uint32_t upto = sum;
#pragma unroll
    for (uint32_t d = 1; d < 32; d *= 2) {
        const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, upto, d);
        if (lane >= d) upto += o;
    }
    if (lane == 31) carry[warp] = upto;
    __syncthreads();
    uint32_t before = upto - sum;
    for (uint32_t w = 0; w < warp; ++w) before += carry[w];
#pragma unroll
    for (uint32_t k = 0; k < per; ++k) {
        if (per * t + k < n) v[per * t + k] = before;
        before += x[k];
    }
}

// parts null: the one CTA counts its pairs itself.
__global__ void __launch_bounds__(kRouteThreads) route_place_kernel(const __grid_constant__ RouteParams p) {
    launch_next();
    wait_previous();
    extern __shared__ uint32_t counts[];           // [kRouteWarps][experts], then [experts] twice
    __shared__ uint32_t carry[32];
    uint32_t* total = counts + kRouteWarps * p.experts;
    uint32_t* offset = total + p.experts;
    const uint32_t t = threadIdx.x, warp = t / 32, lane = t % 32;
    for (uint32_t i = t; i < kRouteWarps * p.experts; i += kRouteThreads) counts[i] = 0;
    __syncthreads();
    const uint64_t run = p.each / kRouteWarps;
    const uint64_t from = min(blockIdx.x * p.each + warp * run, p.pairs), to = min(blockIdx.x * p.each + warp * run + run, p.pairs);
    count_run(p, from, to, counts + warp * p.experts);
    __syncthreads();
    // of each expert, the pairs of the CTAs before this one and of all: kRouteThreads / experts threads (or one) add up the
    // parts of as many ranges of CTAs
    if (p.parts) {
        const uint32_t groups = p.experts < kRouteThreads ? kRouteThreads / p.experts : 1, g = t / p.experts;
        const uint32_t each = (gridDim.x + groups - 1) / groups;
        for (uint32_t e = t; e < p.experts; e += kRouteThreads) total[e] = offset[e] = 0;
        __syncthreads();
        if (g < groups || groups == 1)
            for (uint32_t e = groups == 1 ? t : t % p.experts; e < p.experts; e += kRouteThreads) {
                uint32_t sum = 0, before = 0;
                const uint32_t b0 = groups == 1 ? 0 : g * each, b1 = min(b0 + each, gridDim.x);
#pragma unroll 16
                for (uint32_t b = b0; b < b1; ++b) {
                    const uint32_t n = p.parts[(uint64_t)b * p.experts + e];
                    sum += n;
                    before += b < blockIdx.x ? n : 0;
                }
                atomicAdd(total + e, sum);             // whole numbers: in any order
                atomicAdd(offset + e, before);
            }
        __syncthreads();
    }
    // each warp's first place among its expert's rows
    for (uint32_t e = t; e < p.experts; e += kRouteThreads) {
        uint32_t before = p.parts ? offset[e] : 0;
        for (uint32_t w = 0; w < kRouteWarps; ++w) {
            const uint32_t n = counts[w * p.experts + e];
            counts[w * p.experts + e] = before;
            before += n;
        }
        if (!p.parts) total[e] = before;
        offset[e] = (total[e] + p.align - 1) / p.align * p.align;
    }
    __syncthreads();
    scan_experts(offset, p.experts, carry);
    __syncthreads();
    if (blockIdx.x == 0)
        for (uint32_t e = t; e < p.experts; e += kRouteThreads) {
            const uint32_t at = min(offset[e], p.max_rows);
            p.offsets[e] = (int32_t)at;
            p.counts[e] = (int32_t)min(total[e], p.max_rows - at);
            if (e + 1 == p.experts)
                p.offsets[e + 1] = (int32_t)min(offset[e] + (total[e] + p.align - 1) / p.align * p.align, p.max_rows);
        }
    uint32_t* mine = counts + warp * p.experts;
    walk_run(p, from, to, [&](uint64_t i, uint32_t e, uint32_t same) {
        uint32_t at = p.max_rows;
        if (e < p.experts) at = offset[e] + mine[e] + __popc(same & ((1u << lane) - 1));
        __syncwarp();
        if (e < p.experts && lane == __ffs(same) - 1) mine[e] += __popc(same);
        __syncwarp();
        if (i < to) p.position[i] = at < p.max_rows ? (int32_t)at : -1;
    });
}

// ---- rows --------------------------------------------------------------------------------------
struct Rows {
    char* at;
    uint64_t pitch;
    uint32_t bytes;             // of a row
};

// What the row kernels know of a sort.
struct Sorted {
    const int32_t* position;    // [tokens][k]
    const int32_t* offsets;
    const int32_t* counts;
    uint64_t tokens;
    uint32_t k, experts, max_rows;
    uint32_t fills, fill_ctas;  // CTAs of one expert's filled rows, and all of them: the grid's first
};

__device__ __forceinline__ uint32_t row_of(const Sorted& s, uint64_t pair) { return (uint32_t)s.position[pair]; }   // -1: no row

// Rows from an expert's last to where the next one's begin, zeros: part `cta` of fill_ctas, by `threads` threads.
template <class W>
__device__ __forceinline__ void zero_words(char* row, uint32_t bytes, uint32_t t, uint32_t threads) {
    for (uint32_t i = t; i < bytes / sizeof(W); i += threads) reinterpret_cast<W*>(row)[i] = W{};
}
template <class W>
__device__ __forceinline__ void fill_rows(const Sorted& s, const Rows& rows, uint32_t cta, uint32_t t, uint32_t threads) {
    const uint32_t e = cta / s.fills;
    const uint32_t from = (uint32_t)s.offsets[e] + (uint32_t)s.counts[e] + cta % s.fills * kFillRows;
    const uint32_t to = min(min((uint32_t)s.offsets[e + 1], s.max_rows), from + kFillRows);
    for (uint32_t r = from; r < to; ++r) zero_words<W>(rows.at + r * rows.pitch, rows.bytes, t, threads);
}
template <class W>
__device__ __forceinline__ void fill_rows(const Sorted& s, const Rows& rows, uint32_t cta) {
    fill_rows<W>(s, rows, cta, threadIdx.y * blockDim.x + threadIdx.x, blockDim.x * blockDim.y);
}

template <class W>
__device__ __forceinline__ void copy_row(const Sorted& s, const char* from, const Rows& rows, uint64_t token) {
    for (uint32_t i = threadIdx.x; i < rows.bytes / sizeof(W); i += blockDim.x) {
        const W v = reinterpret_cast<const W*>(from)[i];
        for (uint32_t j = 0; j < s.k; ++j) {
            const uint32_t r = row_of(s, token * s.k + j);
            if (r < s.max_rows) reinterpret_cast<W*>(rows.at + r * rows.pitch)[i] = v;
        }
    }
}

struct DispatchParams {
    Sorted s;
    const char* x;
    const char* scales;         // of no tokens: null
    uint64_t x_pitch, scales_pitch;
    Rows rows, row_scales;      // row_scales' may be null: no scales
};

// W: the word that rows are moved by, SW: their scales.
template <class W, class SW>
__global__ void __launch_bounds__(kCopyThreads) dispatch_kernel(const __grid_constant__ DispatchParams p) {
    launch_next();
    wait_previous();
    if (blockIdx.x < p.s.fill_ctas) {
        fill_rows<W>(p.s, p.rows, blockIdx.x);
        if (p.row_scales.at) fill_rows<SW>(p.s, p.row_scales, blockIdx.x);
        return;
    }
    const uint64_t token = blockIdx.x - p.s.fill_ctas;
    copy_row<W>(p.s, p.x + token * p.x_pitch, p.rows, token);
    if (p.row_scales.at) copy_row<SW>(p.s, p.scales + token * p.scales_pitch, p.row_scales, token);
}

struct CombineParams {
    Sorted s;
    const char* rows;
    const float* weights;       // or null
    char* out;
    uint64_t rows_pitch, out_pitch;
    uint32_t cols;
};

// Eight columns of a row from c, which VEC has in one piece, as they are loaded: those from `cols` on are zeros.
template <uint32_t DT>
struct Columns {
    static constexpr uint32_t size = DT == DTT_BF16 ? 2 : 4;
    uint32_t raw[2 * size];
    template <bool VEC>
    __device__ __forceinline__ void load(const char* row, uint32_t c, uint32_t cols) {
        if constexpr (VEC) {
            const Raw8 q = raw8(row + (uint64_t)c * size, DT);
            raw[0] = q.a.x, raw[1] = q.a.y, raw[2] = q.a.z, raw[3] = q.a.w;
            if constexpr (DT != DTT_BF16) raw[4] = q.b.x, raw[5] = q.b.y, raw[6] = q.b.z, raw[7] = q.b.w;
        } else {
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i) {
                if constexpr (DT == DTT_BF16) {
                    const uint32_t v = c + i < cols ? reinterpret_cast<const uint16_t*>(row)[c + i] : 0;
                    raw[i / 2] = i % 2 ? raw[i / 2] | v << 16 : v;
                } else {
                    raw[i] = c + i < cols ? reinterpret_cast<const uint32_t*>(row)[c + i] : 0;
                }
            }
        }
    }
    __device__ __forceinline__ void none() {
#pragma unroll
        for (uint32_t i = 0; i < 2 * size; ++i) raw[i] = 0;
    }
    __device__ __forceinline__ void expand(float (&v)[8]) const {
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) {
            if constexpr (DT == DTT_BF16) v[i] = i % 2 ? bf16_hi(raw[i / 2]) : bf16_lo(raw[i / 2]);
            else v[i] = __uint_as_float(raw[i]);
        }
    }
};

// How many of a token's rows are on their way to a thread at once: what 64 registers hold.  (Backward with eight of bf16 it
// takes more, and so fewer CTAs: 534 us and not 402.)
template <uint32_t DT> constexpr uint32_t kAtOnce = DT == DTT_BF16 ? 8 : 4;

// A token by blockDim.x threads, eight columns each at a time, blockDim.y tokens a CTA.  A token's rows lie anywhere, so
// that what counts is how many loads are out: all of a batch's go before the first is looked at.
template <bool VEC, uint32_t RDT, uint32_t ODT>
__global__ void __launch_bounds__(kRowThreads, 4) combine_kernel(const __grid_constant__ CombineParams p) {
    launch_next();
    wait_previous();
    constexpr uint32_t J = kAtOnce<RDT>;
    const uint64_t token = (uint64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (token >= p.s.tokens) return;
    const uint64_t pairs = token * p.s.k;
    for (uint32_t c = 8 * threadIdx.x; c < p.cols; c += 8 * blockDim.x) {
        float sum[8] = {};
        for (uint32_t j0 = 0; j0 < p.s.k; j0 += J) {
            Columns<RDT> v[J];
            float w[J];
#pragma unroll
            for (uint32_t j = 0; j < J; ++j) {
                const uint32_t r = j0 + j < p.s.k ? row_of(p.s, pairs + j0 + j) : ~0u;
                w[j] = 0.0f;                    // without a row: zeros, with a weight of 0
                v[j].none();
                if (r < p.s.max_rows) {
                    w[j] = p.weights ? p.weights[pairs + j0 + j] : 1.0f;
                    v[j].template load<VEC>(p.rows + r * p.rows_pitch, c, p.cols);
                }
            }
#pragma unroll
            for (uint32_t j = 0; j < J; ++j) {
                float f[8];
                v[j].expand(f);
#pragma unroll
                for (uint32_t i = 0; i < 8; ++i) sum[i] = fmaf(w[j], f[i], sum[i]);
            }
        }
        store8<VEC>(p.out + token * p.out_pitch, ODT, c, p.cols, sum);
    }
}

struct BackwardParams {
    Sorted s;
    const char* dout;
    const char* rows;
    const float* weights;
    Rows drows;
    float* dweights;            // or null: rows are not read
    uint64_t dout_pitch, rows_pitch;
    uint32_t cols;
};

// Sums over a warp of N values a lane, N a power of two up to 32: lane l gets value l % N's.  Each exchange halves the
// values that a lane goes on with.
template <uint32_t N>
__device__ __forceinline__ float sum_of_mine(float (&v)[N]) {
#pragma unroll
    for (uint32_t h = N / 2; h > 0; h /= 2) {
        const bool up = threadIdx.x & h;
#pragma unroll
        for (uint32_t i = 0; i < h; ++i) {
            const float keep = up ? v[i + h] : v[i], give = up ? v[i] : v[i + h];
            v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, h);
        }
    }
#pragma unroll
    for (uint32_t d = N; d < 32; d *= 2) v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], d);
    return v[0];
}

// Tokens as above; a token's own row is read once for a batch of its rows, whose dot products with it are summed up over
// the token's threads at the end.
template <bool VEC, uint32_t RDT, uint32_t GDT, class W>
__global__ void __launch_bounds__(kRowThreads, 4) combine_backward_kernel(const __grid_constant__ BackwardParams p) {
    launch_next();
    wait_previous();
    constexpr uint32_t J = 4;
    __shared__ float sums[2][kRowThreads / 32][J];
    if (blockIdx.x < p.s.fill_ctas) return fill_rows<W>(p.s, p.drows, blockIdx.x);
    const uint64_t token = (uint64_t)(blockIdx.x - p.s.fill_ctas) * blockDim.y + threadIdx.y;
    if (token >= p.s.tokens) return;            // a whole warp: tokens share no barrier
    const uint64_t pairs = token * p.s.k;
    const char* dout = p.dout + token * p.dout_pitch;
    uint32_t turn = 0;
    for (uint32_t j0 = 0; j0 < p.s.k; j0 += J, turn ^= 1) {
        uint32_t r[J];
        float w[J], dot[J];
#pragma unroll
        for (uint32_t j = 0; j < J; ++j) {
            r[j] = j0 + j < p.s.k ? row_of(p.s, pairs + j0 + j) : ~0u;
            w[j] = r[j] < p.s.max_rows ? p.weights[pairs + j0 + j] : 0.0f;
            dot[j] = 0.0f;
        }
        for (uint32_t c = 8 * threadIdx.x; c < p.cols; c += 8 * blockDim.x) {
            Columns<GDT> gs;
            Columns<RDT> v[J];
            gs.template load<VEC>(dout, c, p.cols);
            if (p.dweights) {
#pragma unroll
                for (uint32_t j = 0; j < J; ++j) {
                    v[j].none();
                    if (r[j] < p.s.max_rows) v[j].template load<VEC>(p.rows + r[j] * p.rows_pitch, c, p.cols);
                }
            }
            float g[8];
            gs.expand(g);
#pragma unroll
            for (uint32_t j = 0; j < J; ++j) {
                if (r[j] >= p.s.max_rows) continue;
                float f[8];
                if (p.dweights) {
                    v[j].expand(f);
#pragma unroll
                    for (uint32_t i = 0; i < 8; ++i) dot[j] = fmaf(g[i], f[i], dot[j]);
                }
#pragma unroll
                for (uint32_t i = 0; i < 8; ++i) f[i] = g[i] * w[j];
                store8<VEC>(p.drows.at + r[j] * p.drows.pitch, RDT, c, p.cols, f);
            }
        }
        if (!p.dweights) continue;
        const uint32_t lane = threadIdx.x % 32;
        float sum = sum_of_mine(dot);
        if (blockDim.x > 32) {
            if (lane < J) sums[turn][threadIdx.x / 32][lane] = sum;
            __syncthreads();
            sum = 0.0f;
            if (threadIdx.x < J)
                for (uint32_t i = 0; i < blockDim.x / 32; ++i) sum += sums[turn][i][threadIdx.x];
        }
        if (threadIdx.x < J && j0 + threadIdx.x < p.s.k) p.dweights[pairs + j0 + threadIdx.x] = sum;
    }
}

// ---- rows through shared memory -----------------------------------------------------------------
// For many tokens of long rows: persistent CTAs, three an SM, of eight warps that add up and one that fetches.  An item is a
// batch of a token's rows in 2048 columns (and for the gradients the token's own row), each row's piece in a slot of its own,
// so that items of few rows, as where most experts are other ranks', are many under way.  The ninth warp has bulk copies of the
// next items going, so that reading positions, rows and adding up overlap.  A thread whose wait for an item runs out
// takes it, and all after it, straight from global memory: the results are the same.  A warp of which nobody waits any more is
// not counted among those that are done with an item: it may be items ahead, and would be counted again in a slower one's place,
// whose slots were then filled while it reads them.  The fetching warp's wait runs out instead, and then the others'.
constexpr uint32_t kAdders = 256, kTile = 8 * kAdders, kBatch = 8, kItems = 12, kRingCtas = 3;
#ifndef DTT_EXPERTS_WAIT_LIMIT
#define DTT_EXPERTS_WAIT_LIMIT (1u << 18)      // looks at an mbarrier; one that fails takes 4 us: a second
#endif
constexpr uint32_t kWaitLimit = DTT_EXPERTS_WAIT_LIMIT;
constexpr uint32_t kRingSmem = 72 * 1024;      // of a CTA's slots, at most

__device__ __forceinline__ bool arrived(uint32_t bar, uint32_t parity) {      // false: the wait ran out
    for (uint32_t i = 0; i < kWaitLimit; ++i) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done) : "r"(bar), "r"(parity) : "memory");
        if (done) return true;
    }
    return false;
}
__device__ __forceinline__ void arrive(uint32_t bar) { asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory"); }
__device__ __forceinline__ void bulk(uint32_t dst, const char* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}
__device__ __forceinline__ void adders_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kAdders) : "memory"); }

template <uint32_t RDT, uint32_t GDT, bool BACK>
struct Slots {
    static constexpr uint32_t re = RDT == DTT_BF16 ? 2 : 4, ge = GDT == DTT_BF16 ? 2 : 4;
    static constexpr uint32_t bytes = kTile * (BACK && ge > re ? ge : re), count = kRingSmem / bytes;
    static_assert(count > kBatch, "an item with all its rows fits");
};
// What the adders know of an item.
struct __align__(16) Known {
    uint4 rows[kBatch];         // of those there are, in order: number, weight, its piece's place in the slots
    uint32_t own_at, mask, none[2];
};

struct RingParams {
    Sorted s;
    const char* rows;
    const char* own;            // backward: dout
    const float* weights;       // or null: 1
    char* out;                  // forward
    Rows drows;                 // backward
    float* dweights;            // backward, or null: rows are not read
    uint64_t rows_pitch, own_pitch, out_pitch;
    uint32_t cols;
};

// Items in turn, and the parity of their barriers.
struct Turn {
    uint32_t at = 0, phase = 0;
    __device__ __forceinline__ void next() {
        if (++at == kItems) {
            at = 0;
            phase ^= 1;
        }
    }
};

// The pairs j0 .. j0 + kBatch - 1 of a token as lane j of a warp has them: their rows, as they are, and weights.
struct Pairs {
    uint32_t row = ~0u;
    float weight = 1.0f;
};
__device__ __forceinline__ Pairs lane_pairs(const RingParams& p, uint64_t token, uint32_t j0) {
    const uint32_t lane = threadIdx.x % 32;
    Pairs r;
    if (token < p.s.tokens && lane < kBatch && j0 + lane < p.s.k) {
        const uint64_t pair = token * p.s.k + j0 + lane;
        r.row = row_of(p.s, pair);
        if (p.weights) r.weight = p.weights[pair];
    }
    return r;
}

// What of an item does not depend on its columns, for the lane that fetches a piece: lane j row j's, lane kBatch the token's.
struct Pieces {
    const char* from;           // null: none
    uint32_t row, weight;       // row: of the token's lane the mask of the rows there are
    uint32_t rank;              // which of the rows there are
    uint32_t place, size;       // slots before this piece's, and bytes of an element
    bool known;                 // the adders are told
    uint32_t slots, bytes;      // of the item, and of its columns: bytes each
};
template <uint32_t RDT, uint32_t GDT, bool BACK>
__device__ __forceinline__ Pieces pieces_of(const RingParams& p, uint64_t token, const Pairs& mine) {
    using S = Slots<RDT, GDT, BACK>;
    const uint32_t lane = threadIdx.x % 32;
    const bool reads = !BACK || p.dweights, has = mine.row < p.s.max_rows;
    const uint32_t mask = __ballot_sync(0xFFFFFFFFu, has), rows = reads ? __popc(mask) : 0;
    const bool own = BACK && mask, mine_is_own = lane == kBatch;
    Pieces r;
    r.slots = rows + own;
    r.bytes = rows * S::re + (own ? S::ge : 0);
    r.from = mine_is_own ? (own ? p.own + token * p.own_pitch : nullptr) : reads && has ? p.rows + mine.row * p.rows_pitch : nullptr;
    r.row = mine_is_own ? mask : mine.row;
    r.weight = __float_as_uint(mine.weight);
    r.rank = mine_is_own ? kBatch : __popc(mask & ((1u << lane) - 1));
    r.place = mine_is_own ? rows : reads ? r.rank : 0;
    r.size = mine_is_own ? S::ge : S::re;
    r.known = has || mine_is_own;
    return r;
}

// The ninth warp.  Items in the adders' order: forward a token's columns, and its batches within them; backward its
// batches, and the columns within (the first alone where a batch has no rows).  It is one warp's instructions one after the
// other, so that what does not depend on the columns is worked out once a batch, and lanes do the rows' and the token's
// piece at once: 2000 tokens without a row here 4.6 us, with all of it for each item 5.8.
template <uint32_t RDT, uint32_t GDT, bool BACK>
__device__ __forceinline__ void fetch(const RingParams& p, uint32_t slots, uint32_t full, uint32_t empty, Known* known) {
    using S = Slots<RDT, GDT, BACK>;
    const uint32_t lane = threadIdx.x % 32, tiles = (p.cols + kTile - 1) / kTile, batches = (p.s.k + kBatch - 1) / kBatch;
    Turn turn, oldest;                          // the next item's, and of those under way the first
    uint32_t under_way = 0, free = S::count, head = 0;
    uint32_t held = 0;                          // slots of the item whose turn is the lane's number
    static_assert(kItems <= 32, "a lane each");
    bool late = false;
    // the first item under way is done with: its copies have landed, which adders that have given up do not tell (even
    // lanes look), and the adders have taken them (odd ones); all lanes give up if one does
    const uint32_t done = lane % 2 ? empty : full;
    const auto retire = [&] {
        late = late || __any_sync(0xFFFFFFFFu, DTT_EXPERTS_FETCH_LATE || !arrived(done + 8 * oldest.at, oldest.phase));
        if (late) return;                       // it is still under way: its copies may be
        free += __shfl_sync(0xFFFFFFFFu, held, oldest.at);
        --under_way;
        oldest.next();
    };
    const auto item = [&](const Pieces& x, uint32_t tile) {
        while (!late && (under_way == kItems || free < x.slots)) retire();
        if (late) return;
        const uint32_t c = tile * kTile, columns = min(kTile, p.cols - c), bar = full + 8 * turn.at, at = head + x.place;
        const uint32_t to = (at < S::count ? at : at - S::count) * S::bytes;
        if (x.known)
            reinterpret_cast<uint4*>(known + turn.at)[x.rank] = lane < kBatch ? make_uint4(x.row, x.weight, to, 0) : make_uint4(to, x.row, 0, 0);
        __syncwarp();
        if (lane == 0) bar_expect_tx(bar, columns * x.bytes);
        __syncwarp();
        if (x.from) bulk(slots + to, x.from + (uint64_t)c * x.size, columns * x.size, bar);
        if (lane == turn.at) held = x.slots;
        head += x.slots;
        if (head >= S::count) head -= S::count;
        free -= x.slots;
        ++under_way;
        turn.next();
    };
    uint64_t token = blockIdx.x;
    // the first batches of the next two tokens: their latency is not to be an item's
    Pairs ahead = lane_pairs(p, token, 0), further = lane_pairs(p, token + gridDim.x, 0);
    for (; token < p.s.tokens && !late; token += gridDim.x) {
        const Pairs first = ahead;
        ahead = further;
        further = lane_pairs(p, token + 2 * (uint64_t)gridDim.x, 0);
        const Pieces of_first = pieces_of<RDT, GDT, BACK>(p, token, first);
        const auto batch_of = [&](uint32_t batch) { return batch == 0 ? of_first : pieces_of<RDT, GDT, BACK>(p, token, lane_pairs(p, token, batch * kBatch)); };
        if constexpr (BACK) {
            for (uint32_t batch = 0; batch < batches && !late; ++batch) {
                const Pieces x = batch_of(batch);
                for (uint32_t tile = 0; tile < (x.slots ? tiles : 1) && !late; ++tile) item(x, tile);
            }
        } else {
            for (uint32_t tile = 0; tile < tiles && !late; ++tile)
                for (uint32_t batch = 0; batch < batches && !late; ++batch) item(batch_of(batch), tile);
        }
    }
    // no copy is under way when the CTA leaves
    for (; under_way; --under_way, oldest.next()) (void)arrived(full + 8 * oldest.at, oldest.phase);
}

// Eight columns of a row's piece, or from global memory.
template <uint32_t DT>
__device__ __forceinline__ void piece8(bool late, const char* item, const char* global, float (&v)[8]) {
    if (late) expand8(raw8(global, DT), DT, v);
    else expand8(raw8(item, DT), DT, v);
}

// 131072 rows of 4096 in bf16: combined in 174 us, the copy rate (reads outnumber writes); their gradients in 361 us, 0.93.
// 2000 tokens of 8064 with a row each: 18 to 23 us for the gradients, by how evenly the router's choices fall.  Items of few rows are bound by the adders' instructions one
// after the other, so that three CTAs an SM with 72 KiB of slots each are ahead of two with 108 (177, 368 and 22 us
// where these take 174, 361 and 18), and the rows that there are come one behind the other (18.2 where each of eight places is looked at).
template <uint32_t RDT, uint32_t GDT, bool BACK>
__global__ void __launch_bounds__(kAdders + 32, kRingCtas) rows_ring_kernel(const __grid_constant__ RingParams p) {
    using S = Slots<RDT, GDT, BACK>;
    launch_next();
    extern __shared__ __align__(128) uint8_t slots[];
    __shared__ uint64_t full[kItems], empty[kItems];
    __shared__ Known known[kItems];
    __shared__ float sums[2][kAdders / 32][kBatch];
    const uint32_t t = threadIdx.x;
    if (t == 0) {
        for (uint32_t i = 0; i < kItems; ++i) {
            bar_init(saddr(full + i), 1);
            bar_init(saddr(empty + i), kAdders / 32);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncthreads();
    wait_previous();
    if (t >= kAdders) return fetch<RDT, GDT, BACK>(p, saddr(slots), saddr(full), saddr(empty), known);

    const uint32_t tiles = (p.cols + kTile - 1) / kTile, lane = t % 32;
    Turn ring;
    bool late = false;
    // the next item, and what it knows of its rows
    const auto wait = [&] { late = late || DTT_EXPERTS_LATE || !arrived(saddr(full + ring.at), ring.phase); };
    const auto mask_of = [&](uint64_t token, uint32_t j0) {
        if (!late) return known[ring.at].mask;
        uint32_t mask = 0;
        for (uint32_t j = 0; j < kBatch && j0 + j < p.s.k; ++j) mask |= (row_of(p.s, token * p.s.k + j0 + j) < p.s.max_rows ? 1u : 0u) << j;
        return mask;
    };
    const auto row_at = [&](uint64_t pairs, uint32_t mask, uint32_t i) {          // the i-th of the rows there are
        if (!late) return known[ring.at].rows[i];
        const uint64_t pair = pairs + __fns(mask, 0, i + 1);
        return make_uint4(row_of(p.s, pair), __float_as_uint(p.weights ? p.weights[pair] : 1.0f), 0, 0);
    };
    const char* base = reinterpret_cast<const char*>(slots);
    const auto done = [&] {
        if (__any_sync(0xFFFFFFFFu, !late) && lane == 0) arrive(saddr(empty + ring.at));
        ring.next();
    };
    if constexpr (BACK)
        for (uint32_t f = blockIdx.x; f < p.s.fill_ctas; f += gridDim.x) fill_rows<uint4>(p.s, p.drows, f, t, kAdders);
    uint32_t turn = 0;
    for (uint64_t token = blockIdx.x; token < p.s.tokens; token += gridDim.x) {
        if constexpr (!BACK) {
            for (uint32_t tile = 0; tile < tiles; ++tile) {
                const uint32_t c = tile * kTile + 8 * t;
                float sum[8] = {};
                for (uint32_t j0 = 0; j0 < p.s.k; j0 += kBatch) {
                    wait();
                    const uint32_t mask = c < p.cols ? mask_of(token, j0) : 0, n = __popc(mask);
#pragma unroll
                    for (uint32_t j = 0; j < kBatch; ++j) {
                        if (j >= n) break;
                        const uint4 row = row_at(token * p.s.k + j0, mask, j);
                        const float w = __uint_as_float(row.y);
                        float v[8];
                        piece8<RDT>(late, base + row.z + 8 * t * S::re, p.rows + row.x * p.rows_pitch + (uint64_t)c * S::re, v);
#pragma unroll
                        for (uint32_t i = 0; i < 8; ++i) sum[i] = fmaf(w, v[i], sum[i]);
                    }
                    done();
                }
                if (c < p.cols) store8<true>(p.out + token * p.out_pitch, GDT, c, p.cols, sum);
            }
        } else {
            for (uint32_t j0 = 0; j0 < p.s.k; j0 += kBatch) {
                float dot[kBatch] = {};
                uint32_t mask = 0;
                for (uint32_t tile = 0; tile < tiles; ++tile) {
                    const uint32_t c = tile * kTile + 8 * t;
                    wait();
                    mask = mask_of(token, j0);
                    if (mask && c < p.cols) {
                        const uint32_t n = __popc(mask);
                        float g[8];
                        piece8<GDT>(late, base + known[ring.at].own_at + 8 * t * S::ge, p.own + token * p.own_pitch + (uint64_t)c * S::ge, g);
#pragma unroll
                        for (uint32_t j = 0; j < kBatch; ++j) {
                            if (j >= n) break;
                            const uint4 row = row_at(token * p.s.k + j0, mask, j);
                            const float w = __uint_as_float(row.y);
                            float v[8];
                            if (p.dweights) {
                                piece8<RDT>(late, base + row.z + 8 * t * S::re, p.rows + row.x * p.rows_pitch + (uint64_t)c * S::re, v);
#pragma unroll
                                for (uint32_t i = 0; i < 8; ++i) dot[j] = fmaf(g[i], v[i], dot[j]);
                            }
#pragma unroll
                            for (uint32_t i = 0; i < 8; ++i) v[i] = g[i] * w;
                            store8_first_out(p.drows.at + row.x * p.drows.pitch, RDT, c, v);
                        }
                    }
                    done();
                    if (!mask) break;            // one item, without copies
                }
                if (!p.dweights) continue;
                float sum = 0.0f;
                if (mask) {                     // for all adders, or for none
                    const float mine = sum_of_mine(dot);
                    if (lane < kBatch) sums[turn][t / 32][lane] = mine;
                    adders_sync();
                    if (t < kBatch && mask >> t & 1) {
                        const uint32_t rank = __popc(mask & ((1u << t) - 1));
#pragma unroll
                        for (uint32_t i = 0; i < kAdders / 32; ++i) sum += sums[turn][i][rank];
                    }
                    turn ^= 1;
                }
                if (t < kBatch && j0 + t < p.s.k) p.dweights[token * p.s.k + j0 + t] = sum;
            }
        }
    }
}

// ---- host --------------------------------------------------------------------------------------
int check_desc(const char* who, const dtt_experts_desc* d) {
    if (!d) return fail(DTT_EINVAL, "%s: null desc", who);
    if (d->experts < 1 || d->experts > kMostExperts) return fail(DTT_EINVAL, "%s: experts must be 1 .. %u", who, kMostExperts);
    if (d->top_k < 1 || d->top_k > kMostChoices) return fail(DTT_EINVAL, "%s: top_k must be 1 .. %u", who, kMostChoices);
    if (d->align < 1 || d->align > 65536) return fail(DTT_EINVAL, "%s: align must be 1 .. 65536", who);
    if (d->first >= 1u << 31) return fail(DTT_EINVAL, "%s: first must be below 2^31", who);
    return DTT_OK;
}

int check_sizes(const char* who, const dtt_experts_desc* d, uint64_t tokens, uint64_t max_rows) {
    const int rc = check_desc(who, d);
    if (rc) return rc;
    if (tokens >= (1ull << 31) / d->top_k || tokens * d->top_k + (uint64_t)d->experts * d->align >= 1ull << 31 || max_rows >= 1ull << 31)
        return fail(DTT_EINVAL, "%s: 2^31 rows or more", who);
    return DTT_OK;
}

int check_ptr(const char* who, const char* name, const void* p, uint32_t to, bool optional = false) {
    if (!p) return optional ? DTT_OK : fail(DTT_EINVAL, "%s: %s is missing", who, name);
    if (reinterpret_cast<uintptr_t>(p) % to) return fail(DTT_EINVAL, "%s: %s must be aligned to its %u-byte elements", who, name, to);
    return DTT_OK;
}

int check_rows(const char* who, const char* name, const void* p, uint64_t pitch, uint64_t rows, uint64_t bytes, uint32_t element, bool optional = false) {
    const int rc = check_ptr(who, name, p, element, optional);
    if (rc || !p) return rc;
    if (pitch % element) return fail(DTT_EINVAL, "%s: %s: the pitch is no multiple of its %u-byte elements", who, name, element);
    if (rows > 1 && pitch < bytes) return fail(DTT_EINVAL, "%s: %s: the pitch is less than a row", who, name);
    return DTT_OK;
}

Sorted sorted_of(const dtt_experts_desc* d, uint64_t tokens, uint64_t max_rows, const int32_t* position, const int32_t* offsets, const int32_t* counts) {
    Sorted s{position, offsets, counts, tokens, d->top_k, d->experts, (uint32_t)max_rows, 0, 0};
    if (offsets && d->align > 1) {
        s.fills = (d->align - 1 + kFillRows - 1) / kFillRows;
        s.fill_ctas = s.fills * d->experts;
    }
    return s;
}

// The widest word, of 16, 4, 2 and 1 bytes, that every address and length is a multiple of.
uint32_t word_of(std::initializer_list<uint64_t> all) {
    uint64_t bits = 0;
    for (uint64_t a : all) bits |= a;
    return bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : bits % 2 == 0 ? 2 : 1;
}
uint64_t bits_of(const void* p) { return reinterpret_cast<uintptr_t>(p); }

template <class SW>
cudaError_t launch_dispatch(uint32_t word, uint32_t grid, cudaStream_t stream, const DispatchParams& p) {
    auto kernel = word == 16 ? dispatch_kernel<uint4, SW> : word == 4 ? dispatch_kernel<uint32_t, SW> : word == 2 ? dispatch_kernel<uint16_t, SW> : dispatch_kernel<uint8_t, SW>;
    return launch(kernel, grid, kCopyThreads, 0, 0, true, stream, p);
}

// A token's threads, as many as it has eights of columns, and the tokens of a CTA: several where a token is one warp.
dim3 token_block(uint64_t cols) {
    const uint32_t t = (uint32_t)std::min<uint64_t>((cols + 255) / 256 * 32, kRowThreads);
    return dim3(t, t == 32 ? 8 : 1);
}
uint64_t ctas_of(uint64_t tokens, dim3 block) { return (tokens + block.y - 1) / block.y; }

using CombineKernel = void (*)(CombineParams);
template <bool VEC>
CombineKernel combine_of(uint32_t rows, uint32_t out) {
    if (rows == DTT_BF16) return out == DTT_BF16 ? combine_kernel<VEC, DTT_BF16, DTT_BF16> : combine_kernel<VEC, DTT_BF16, DTT_F32>;
    return out == DTT_BF16 ? combine_kernel<VEC, DTT_F32, DTT_BF16> : combine_kernel<VEC, DTT_F32, DTT_F32>;
}
CombineKernel combine_of(bool vec, uint32_t rows, uint32_t out) { return vec ? combine_of<true>(rows, out) : combine_of<false>(rows, out); }

using BackwardKernel = void (*)(BackwardParams);
template <bool VEC, class W>
BackwardKernel backward_of(uint32_t rows, uint32_t dout) {
    if (rows == DTT_BF16) return dout == DTT_BF16 ? combine_backward_kernel<VEC, DTT_BF16, DTT_BF16, W> : combine_backward_kernel<VEC, DTT_BF16, DTT_F32, W>;
    return dout == DTT_BF16 ? combine_backward_kernel<VEC, DTT_F32, DTT_BF16, W> : combine_backward_kernel<VEC, DTT_F32, DTT_F32, W>;
}
BackwardKernel backward_of(bool vec, uint32_t rows, uint32_t dout) { return vec ? backward_of<true, uint4>(rows, dout) : backward_of<false, uint16_t>(rows, dout); }

// The rows through shared memory: for the grid and what it takes.
struct RingLaunch {
    void (*kernel)(RingParams);
    uint32_t smem;
};
template <bool BACK, uint32_t RDT, uint32_t GDT>
RingLaunch ring_of() { return {rows_ring_kernel<RDT, GDT, BACK>, Slots<RDT, GDT, BACK>::bytes * Slots<RDT, GDT, BACK>::count}; }
template <bool BACK>
RingLaunch ring_of(uint32_t rows, uint32_t other) {
    if (rows == DTT_BF16) return other == DTT_BF16 ? ring_of<BACK, DTT_BF16, DTT_BF16>() : ring_of<BACK, DTT_BF16, DTT_F32>();
    return other == DTT_BF16 ? ring_of<BACK, DTT_F32, DTT_BF16>() : ring_of<BACK, DTT_F32, DTT_F32>();
}
// Measured over 80 to 20000 tokens, with 8 choices of 64 experts all here, 8 of 64 with a quarter here, and 2 of 16 all
// here (bf16, us straight from global memory and by the ring).  Forward, 2600 tokens of 1024 columns: 11.2 and 11.4, 6.2 and
// 6.8, 6.0 and 6.3; of 2048: 20.1 and 17.6, 11.2 and 8.4, 10.8 and 8.1; of 8064: 71 and 58, 34 and 25, 32 and 24.  300 tokens
// of 2048: 3.9 and 4.2, 2.4 and 2.6, 2.3 and 2.4; of 4096: 7.4 and 7.0, 3.9 and 3.4, 3.6 and 3.1; 80 of 4096: 3.3 and 3.8, 2.8
// and 2.9, 2.6 and 2.5.  Backward, 2600 tokens of 1024: 21.0 and 17.6, 11.7 and 10.1, 8.9 and 9.6; of 2048: 38 and 33, 21 and 12, 16
// and 12; 300 of 2048: 7.5 and 6.4, 3.8 and 3.4, 2.6 and 3.1; of 4096: 13.1 and 10.6, 6.6 and 4.6, 4.5 and 4.1.
bool through_ring(bool vec, uint64_t tokens, uint32_t k, uint64_t cols, bool back) {
    const uint64_t least = back ? (k >= 8 ? 1024 : 2048) : tokens >= 8 * kSms ? 2048 : 4096;
    return vec && cols >= least && tokens >= kSms;
}
cudaError_t launch_ring(const RingLaunch& r, const RingParams& p, cudaStream_t stream) {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) sms = 1;
    return launch(r.kernel, (uint32_t)std::min<uint64_t>(p.s.tokens, kRingCtas * (uint64_t)sms), kAdders + 32, r.smem, 0, true, stream, p);
}

uint32_t elem_bytes(uint32_t dt) { return dt == DTT_BF16 ? 2 : 4; }
bool aligned(const void* p, uint64_t pitch) { return bits_of(p) % 16 == 0 && pitch % 16 == 0; }

}  // namespace

cudaError_t preload_experts_kernels() {
    cudaError_t e = cudaSuccess;
    auto add = [&](auto... kernels) { ((e = e == cudaSuccess ? prepare_kernel(kernels) : e), ...); };
    add(route_count_kernel, route_place_kernel, dispatch_kernel<uint4, uint4>, dispatch_kernel<uint4, uint32_t>, dispatch_kernel<uint32_t, uint4>,
        dispatch_kernel<uint32_t, uint32_t>, dispatch_kernel<uint16_t, uint4>, dispatch_kernel<uint16_t, uint32_t>, dispatch_kernel<uint8_t, uint4>,
        dispatch_kernel<uint8_t, uint32_t>);
    for (uint32_t i = 0; i < 8; ++i) {
        const uint32_t a = i & 1 ? DTT_F32 : DTT_BF16, b = i & 2 ? DTT_F32 : DTT_BF16;
        add(combine_of(i & 4, a, b), backward_of(i & 4, a, b));
        const RingLaunch r = i & 4 ? ring_of<true>(a, b) : ring_of<false>(a, b);
        add(r.kernel);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(r.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)r.smem);
    }
    constexpr int most = (kRouteWarps + 2) * kMostExperts * 4;
    for (auto k : {route_count_kernel, route_place_kernel})
        if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    return e;
}

}  // namespace dtt

using namespace dtt;

extern "C" int dtt_experts_workspace(const dtt_experts_desc* d, uint64_t* bytes) {
    const char* who = "dtt_experts_workspace";
    const int rc = check_desc(who, d);
    if (rc) return rc;
    if (!bytes) return fail(DTT_EINVAL, "%s: null bytes", who);
    *bytes = (uint64_t)kMostParts * d->experts * 4;
    return DTT_OK;
}

extern "C" int dtt_experts_route(const dtt_experts_desc* d, uint64_t tokens, const void* ids, uint32_t id_bytes, uint64_t max_rows,
                                 int32_t* position, int32_t* offsets, int32_t* counts, void* workspace, uint64_t workspace_bytes,
                                 cudaStream_t stream) {
    const char* who = "dtt_experts_route";
    int rc = check_sizes(who, d, tokens, max_rows);
    if (rc) return rc;
    if (id_bytes != 4 && id_bytes != 8) return fail(DTT_EINVAL, "%s: ids are of 4 or 8 bytes", who);
    if ((rc = check_ptr(who, "ids", ids, id_bytes, tokens == 0)) || (rc = check_ptr(who, "position", position, 4, tokens == 0)) ||
        (rc = check_ptr(who, "offsets", offsets, 4)) || (rc = check_ptr(who, "counts", counts, 4)) ||
        (rc = check_ptr(who, "the workspace", workspace, 16)))
        return rc;
    if (workspace_bytes < (uint64_t)kMostParts * d->experts * 4) return fail(DTT_EINVAL, "%s: the workspace is short", who);
    if ((rc = preload_once())) return rc;
    RouteParams p{};
    p.ids = ids;
    p.position = position;
    p.offsets = offsets;
    p.counts = counts;
    p.pairs = tokens * d->top_k;
    p.experts = d->experts;
    p.first = d->first;
    p.align = d->align;
    p.max_rows = (uint32_t)max_rows;
    p.wide = id_bytes == 8;
    const uint32_t parts = (uint32_t)std::clamp<uint64_t>((p.pairs + kPartPairs - 1) / kPartPairs, 1, kMostParts);
    p.each = ((p.pairs + parts - 1) / parts + kRouteThreads - 1) / kRouteThreads * kRouteThreads;
    p.parts = parts > 1 ? static_cast<uint32_t*>(workspace) : nullptr;
    const uint32_t smem = kRouteWarps * d->experts * 4;
    cudaError_t e = cudaSuccess;
    if (parts > 1) e = launch(route_count_kernel, parts, kRouteThreads, smem, 0, true, stream, p);
    if (e == cudaSuccess) e = launch(route_place_kernel, parts, kRouteThreads, smem + 2 * d->experts * 4, 0, true, stream, p);
    if (e != cudaSuccess) return fail(DTT_ECUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    return DTT_OK;
}

extern "C" int dtt_experts_dispatch(const dtt_experts_desc* d, uint64_t tokens, const int32_t* position, const int32_t* offsets,
                                    const int32_t* counts, const void* x, uint64_t x_pitch, uint64_t row_bytes, void* rows,
                                    uint64_t rows_pitch, uint64_t max_rows, const float* scales, uint64_t scales_pitch,
                                    uint64_t scale_count, float* row_scales, uint64_t row_scales_pitch, cudaStream_t stream) {
    const char* who = "dtt_experts_dispatch";
    int rc = check_sizes(who, d, tokens, max_rows);
    if (rc) return rc;
    if (row_bytes < 1 || row_bytes > 1ull << 26 || scale_count > 1ull << 24) return fail(DTT_EINVAL, "%s: a row has 1 .. 2^26 bytes and up to 2^24 scales", who);
    const bool missing = scales ? !row_scales && max_rows : row_scales && tokens;          // scales of no tokens, or of no rows, may be null
    if (missing || ((scales || row_scales) && !scale_count))
        return fail(DTT_EINVAL, "%s: scales and row_scales go together, with one scale a row at least", who);
    if ((rc = check_ptr(who, "position", position, 4, tokens == 0)) || (rc = check_ptr(who, "offsets", offsets, 4)) || (rc = check_ptr(who, "counts", counts, 4)) ||
        (rc = check_rows(who, "x", x, x_pitch, tokens, row_bytes, 1, tokens == 0)) || (rc = check_rows(who, "rows", rows, rows_pitch, max_rows, row_bytes, 1, max_rows == 0)) ||
        (rc = check_rows(who, "scales", scales, scales_pitch, tokens, scale_count * 4, 4, true)) ||
        (rc = check_rows(who, "row_scales", row_scales, row_scales_pitch, max_rows, scale_count * 4, 4, true)))
        return rc;
    DispatchParams p{};
    p.s = sorted_of(d, tokens, max_rows, position, offsets, counts);
    const uint64_t grid = tokens + p.s.fill_ctas;
    if (grid == 0 || max_rows == 0) return DTT_OK;
    if ((rc = preload_once())) return rc;
    p.x = static_cast<const char*>(x);
    p.x_pitch = x_pitch;
    p.rows = Rows{static_cast<char*>(rows), rows_pitch, (uint32_t)row_bytes};
    p.scales = reinterpret_cast<const char*>(scales);
    p.scales_pitch = scales_pitch;
    p.row_scales = Rows{reinterpret_cast<char*>(row_scales), row_scales_pitch, (uint32_t)scale_count * 4};
    const uint32_t word = word_of({bits_of(x), x_pitch, row_bytes, bits_of(rows), rows_pitch});
    const bool wide = !row_scales || word_of({bits_of(scales), scales_pitch, scale_count * 4, bits_of(row_scales), row_scales_pitch}) == 16;
    const cudaError_t e = wide ? launch_dispatch<uint4>(word, (uint32_t)grid, stream, p) : launch_dispatch<uint32_t>(word, (uint32_t)grid, stream, p);
    if (e != cudaSuccess) return fail(DTT_ECUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    return DTT_OK;
}

extern "C" int dtt_experts_combine(const dtt_experts_desc* d, uint64_t tokens, uint64_t cols, const int32_t* position, const void* rows,
                                   uint32_t rows_dtype, uint64_t rows_pitch, uint64_t max_rows, const float* weights, void* out,
                                   uint32_t out_dtype, uint64_t out_pitch, cudaStream_t stream) {
    const char* who = "dtt_experts_combine";
    int rc = check_sizes(who, d, tokens, max_rows);
    if (rc) return rc;
    for (uint32_t t : {rows_dtype, out_dtype})
        if (t != DTT_BF16 && t != DTT_F32) return fail(DTT_EINVAL, "%s: rows and out are bf16 or f32", who);
    if (cols < 1 || cols > 1ull << 24) return fail(DTT_EINVAL, "%s: cols must be 1 .. 2^24", who);
    if (tokens == 0) return DTT_OK;
    const uint32_t re = elem_bytes(rows_dtype), oe = elem_bytes(out_dtype);
    if ((rc = check_ptr(who, "position", position, 4)) || (rc = check_rows(who, "rows", rows, rows_pitch, max_rows, cols * re, re, max_rows == 0)) ||
        (rc = check_ptr(who, "weights", weights, 4, true)) || (rc = check_rows(who, "out", out, out_pitch, tokens, cols * oe, oe)))
        return rc;
    if ((rc = preload_once())) return rc;
    CombineParams p{};
    p.s = sorted_of(d, tokens, max_rows, position, nullptr, nullptr);
    p.rows = static_cast<const char*>(rows);
    p.weights = weights;
    p.out = static_cast<char*>(out);
    p.rows_pitch = rows_pitch;
    p.out_pitch = out_pitch;
    p.cols = (uint32_t)cols;
    const bool vec = cols % 8 == 0 && aligned(rows, rows_pitch) && aligned(out, out_pitch);
    const dim3 block = token_block(cols);
    RingParams q{};
    q.s = p.s;
    q.rows = p.rows;
    q.weights = weights;
    q.out = p.out;
    q.rows_pitch = rows_pitch;
    q.out_pitch = out_pitch;
    q.cols = p.cols;
    const cudaError_t e = through_ring(vec, tokens, d->top_k, cols, false) ? launch_ring(ring_of<false>(rows_dtype, out_dtype), q, stream) : launch(combine_of(vec, rows_dtype, out_dtype), (uint32_t)ctas_of(tokens, block), block, 0, 0, true, stream, p);
    if (e != cudaSuccess) return fail(DTT_ECUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    return DTT_OK;
}

extern "C" int dtt_experts_combine_backward(const dtt_experts_desc* d, uint64_t tokens, uint64_t cols, const int32_t* position,
                                            const int32_t* offsets, const int32_t* counts, const void* dout, uint32_t dout_dtype,
                                            uint64_t dout_pitch, const void* rows, uint32_t rows_dtype, uint64_t rows_pitch,
                                            uint64_t max_rows, const float* weights, void* drows, uint64_t drows_pitch,
                                            float* dweights, cudaStream_t stream) {
    const char* who = "dtt_experts_combine_backward";
    int rc = check_sizes(who, d, tokens, max_rows);
    if (rc) return rc;
    for (uint32_t t : {rows_dtype, dout_dtype})
        if (t != DTT_BF16 && t != DTT_F32) return fail(DTT_EINVAL, "%s: rows and dout are bf16 or f32", who);
    if (cols < 1 || cols > 1ull << 24) return fail(DTT_EINVAL, "%s: cols must be 1 .. 2^24", who);
    const uint32_t re = elem_bytes(rows_dtype), ge = elem_bytes(dout_dtype);
    if ((rc = check_ptr(who, "position", position, 4, tokens == 0)) || (rc = check_ptr(who, "offsets", offsets, 4)) || (rc = check_ptr(who, "counts", counts, 4)) ||
        (rc = check_rows(who, "dout", dout, dout_pitch, tokens, cols * ge, ge, tokens == 0)) ||
        (rc = check_rows(who, "rows", rows, rows_pitch, max_rows, cols * re, re, !dweights || max_rows == 0)) ||
        (rc = check_ptr(who, "weights", weights, 4, tokens == 0)) || (rc = check_rows(who, "drows", drows, drows_pitch, max_rows, cols * re, re, max_rows == 0)) ||
        (rc = check_ptr(who, "dweights", dweights, 4, true)))
        return rc;
    BackwardParams p{};
    p.s = sorted_of(d, tokens, max_rows, position, offsets, counts);
    const dim3 block = token_block(cols);
    const uint64_t grid = ctas_of(tokens, block) + p.s.fill_ctas;
    if (grid == 0) return DTT_OK;
    if ((rc = preload_once())) return rc;
    p.dout = static_cast<const char*>(dout);
    p.rows = static_cast<const char*>(rows);
    p.weights = weights;
    p.drows = Rows{static_cast<char*>(drows), drows_pitch, (uint32_t)cols * re};
    p.dweights = dweights;
    p.dout_pitch = dout_pitch;
    p.rows_pitch = rows_pitch;
    p.cols = (uint32_t)cols;
    const bool vec = cols % 8 == 0 && aligned(dout, dout_pitch) && aligned(drows, drows_pitch) && (!dweights || aligned(rows, rows_pitch));
    RingParams q{};
    q.s = p.s;
    q.rows = p.rows;
    q.own = p.dout;
    q.weights = weights;
    q.drows = p.drows;
    q.dweights = dweights;
    q.rows_pitch = rows_pitch;
    q.own_pitch = dout_pitch;
    q.cols = p.cols;
    const cudaError_t e = through_ring(vec, tokens, d->top_k, cols, true) ? launch_ring(ring_of<true>(rows_dtype, dout_dtype), q, stream) : launch(backward_of(vec, rows_dtype, dout_dtype), (uint32_t)grid, block, 0, 0, true, stream, p);
    if (e != cudaSuccess) return fail(DTT_ECUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    return DTT_OK;
}

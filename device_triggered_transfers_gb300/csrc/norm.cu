// Residual addition with a root-mean-square norm or a layer norm, and their backward passes (dtt_ops.h).
//
// Each kernel has both, the layer norm where MEAN: the row's mean comes off first, and its variance is summed over
// what is left (a mean of squares less the squared mean would lose what the mean is larger than the rest by), so that
// a row is reduced twice; backward, its two sums go through one reduction, and two gradients add up over the rows.
// All f32 between the loads and the stores.  The forms of each pass:
//  - short (256 columns and less, 16-byte aligned, whole chunks of 8 columns): a row by a part of a warp;
//  - ring (longer rows that two stages in shared memory have room for; rows that are not aligned where there
//    are many): persistent CTAs whose rows come through a ring of stages, bulk copies running ahead of the
//    arithmetic.  Aligned, thread t of T holds columns 8 (i T + t) .. + 7 of chunk i, so that accesses
//    are contiguous over a warp, and a group of 32, 64 or 128 columns is 4, 8 or 16 neighbouring lanes;
//  - chunks (aligned rows too long for the ring): the same layout, from global memory;
//  - elements (what is not aligned or no whole number of chunks, and few rows of it): a warp holds 32 E
//    neighbouring columns, a thread every 32nd of them.
// Every kernel lets the next launch begin and waits for the one before it before it touches memory, so that a
// launch's set-up overlaps the end of the kernel before: 2048 x 4096 14.6 us without and 12.5 with it.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "dtt_ops.h"
#include "internal.h"
#include "ring.h"
#include "rowio.cuh"

namespace dtt {
namespace {

constexpr float kE4m3Max = 448.0f;
constexpr float kScaleMin = 0x1p-100f;     // scale of a group of zeros: its reciprocal stays finite
// Partial rows of the weight's gradient, at most: four, eight or sixteen a SM.  Rows of one warp (256
// columns and less) have several in a CTA: 20000 x 256 25 us with sixteen CTAs a SM, 20 with four.
__host__ __device__ constexpr uint32_t most_partials(uint64_t cols) { return (cols > 1024 || cols <= 256 ? 4 : cols > 512 ? 8 : 16) * kSms; }
constexpr uint32_t kFwdThreads = 1024, kBwdThreads = 512, kRingThreads = ring::kThreads;   // a row's most threads
template <bool MEAN> constexpr uint32_t kFwdOwn = MEAN ? 896 : 640;      // shared memory of a ring's CTA beside its stages, at most
template <bool MEAN> constexpr uint32_t kBwdOwn = MEAN ? 4736 : 2432;
constexpr uint32_t kWaitLimit = 1u << 18;      // looks at an mbarrier; one that fails takes 4 us: a second
// Whether row r of a ring does not arrive for thread t in time: a build of its own shows what becomes of such rows.
#ifndef DTT_NORM_ROW_LATE
#define DTT_NORM_ROW_LATE false
#endif
constexpr uint32_t kShortCols = 256;       // columns of the short form, at most
// Rows whose weight gradient is added up by columns in the same launch, at most.  By partial rows and by columns, back to
// back in a graph: 16 x 4096 (bf16) 4.6 us and 2.8, 64 x 8064 6.6 and 4.5, 152 x 4096 6.1 and 3.8, 152 x 1024 5.1 and
// 5.5, 152 x 16384 13.6 and 14.5, 304 x 8064 9.9 and 11.6.
constexpr uint32_t kFewRows = 96;
constexpr uint32_t kWideThreads = 768;     // of an unaligned row of the layer norm's backward pass, at most
constexpr uint32_t kWarpRows = 8;          // element form: rows of a CTA whose rows are one warp each
constexpr uint32_t kLong = 0;              // NCH of a row that does not fit a CTA's registers

struct FwdParams {
    const char* x;
    const char* res;            // or null
    const char* w;              // or null
    char* res_out;              // or null
    char* y;
    float* scales;
    float* rstd;                // or null
    uint64_t x_pitch, res_pitch, res_out_pitch, y_pitch;
    uint64_t rows;
    uint32_t cols, groups;
    uint32_t x_dt, res_dt, w_dt, y_dt;
    uint32_t group_lanes;       // lanes that share a scale: 4, 8, 16; 0: one scale per row
    float eps, inv_cols;
    // layer norm:
    const char* b;              // or null
    float* mean;                // or null
};

struct BwdParams {
    const char* dy;
    const char* h;
    const char* w;              // or null
    const float* rstd;
    const char* dres;           // or null
    char* dx;
    float* partial;             // [partials][cols], or null: no weight gradient, or few rows
    float* dweight;             // few rows: the CTAs after the first `partials` work it out; else null
    uint64_t dy_pitch, h_pitch, dres_pitch, dx_pitch;
    uint64_t rows;
    uint32_t cols, partials, walkers;   // walker i takes rows i, i + walkers, ...
    uint32_t dy_dt, h_dt, w_dt;
    float inv_cols;
    // layer norm:
    const float* mean;
    float* partial_b;           // as partial and dweight, of the bias's gradient
    float* dbias;
};

// The scale of a group whose largest magnitude is m.
__device__ __forceinline__ float scale_of(float m) { return max_nan(m * (1.0f / kE4m3Max), kScaleMin); }

// Division by a group's scale: the reciprocal once a group, and a quotient y * inv whose remainder, exact in
// a fused multiply-add, corrects it to the f32 quotient rounded to nearest (P. Markstein, IBM J. Res. Dev. 34
// (1), 1990).  y * inv alone turns values midway between two codes to the wrong one.  An infinite scale: d
// and inv are 0, which gives 0 for finite values and NaN for infinities.
struct Divisor {
    float d, inv;
};
__device__ __forceinline__ Divisor divisor_of(float scale) {
    Divisor v;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(scale));
    v.d = isinf(scale) ? 0.0f : scale;
    v.inv = fmaf(r, fmaf(-v.d, r, 1.0f), r);
    return v;
}
__device__ __forceinline__ float quotient(float y, const Divisor& v) {
    const float q = y * v.inv;
    return fmaf(fmaf(-v.d, q, y), v.inv, q);
}

// Over the TPR threads of a row, the same bits in each.  One warp: butterfly shuffles.  More: the warps'
// values through shared memory (`slot`: 32 words used by this reduction alone between two of the row's
// barriers).
__device__ __forceinline__ float row_sum(float v, uint32_t tpr, float* slot) {
#pragma unroll
    for (uint32_t o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (tpr == 32) return v;
    const uint32_t lane = threadIdx.x % 32;
    if (lane == 0) slot[threadIdx.x / 32] = v;
    __syncthreads();
    v = lane < tpr / 32 ? slot[lane] : 0.0f;
#pragma unroll
    for (uint32_t o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Two sums with one barrier; slot: 64 words.
__device__ __forceinline__ float2 row_sum2(float a, float b, uint32_t tpr, float* slot) {
#pragma unroll
    for (uint32_t o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
        b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    }
    if (tpr == 32) return {a, b};
    const uint32_t lane = threadIdx.x % 32;
    if (lane == 0) {
        slot[threadIdx.x / 32] = a;
        slot[32 + threadIdx.x / 32] = b;
    }
    __syncthreads();
    a = lane < tpr / 32 ? slot[lane] : 0.0f;
    b = lane < tpr / 32 ? slot[32 + lane] : 0.0f;
#pragma unroll
    for (uint32_t o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
        b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    }
    return {a, b};
}

// A row's means of g n and, for the layer norm, of g.
template <bool MEAN>
__device__ __forceinline__ float2 row_means(float dot, float all, uint32_t tpr, float* slot, float inv_cols) {
    if constexpr (!MEAN) return {row_sum(dot, tpr, slot) * inv_cols, 0.0f};
    const float2 sums = row_sum2(dot, all, tpr, slot);
    return {sums.x * inv_cols, sums.y * inv_cols};
}

// The largest of magnitudes, NaN if one is: as bits, magnitudes order like integers, with NaN on top.
__device__ __forceinline__ float warp_max(float v) {
    return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v)));
}

__device__ __forceinline__ float row_max(float v, uint32_t tpr, float* slot) {
    v = warp_max(v);
    if (tpr == 32) return v;
    const uint32_t lane = threadIdx.x % 32;
    if (lane == 0) slot[threadIdx.x / 32] = v;
    __syncthreads();
    return warp_max(lane < tpr / 32 ? slot[lane] : 0.0f);
}

// One row a CTA.  NCH chunks a thread stay in registers; kLong reads the row again for each pass over it.
// 2000 x 32768 in bf16: 141 us, 0.55 of the copy rate; loads that wait for one another bound it.  The layer norm, which reduces the row
// twice: 188 us, 0.41; 1000 x 70000, read once more for the mean, 235 us, 0.35.
template <bool MEAN, uint32_t NCH, bool VEC>
__global__ void __launch_bounds__(kFwdThreads) norm_fwd_kernel(const __grid_constant__ FwdParams p) {
    launch_next();
    wait_previous();
    __shared__ float slots[MEAN ? 3 : 2][32];
    const uint32_t tpr = blockDim.x, t = threadIdx.x;
    const uint64_t r = blockIdx.x;
    const char* x = p.x + r * p.x_pitch;
    const char* res = p.res ? p.res + r * p.res_pitch : nullptr;
    char* res_out = p.res_out ? p.res_out + r * p.res_out_pitch : nullptr;
    char* y = p.y + r * p.y_pitch;

    constexpr uint32_t HELD = NCH == kLong ? 1 : NCH;
    const uint32_t nch = NCH == kLong ? (p.cols + 8 * tpr - 1) / (8 * tpr) : NCH;
    float h[HELD][8];
    auto load = [&](uint32_t i, float (&v)[8]) {
        const uint32_t c = 8 * (i * tpr + t);
        load8<VEC>(x, p.x_dt, c, p.cols, v);
        if (res) {
            float q[8];
            load8<VEC>(res, p.res_dt, c, p.cols, q);
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k) v[k] += q[k];
        }
    };
    float sum = 0.0f;
    if constexpr (NCH != kLong) {
#pragma unroll
        for (uint32_t i = 0; i < HELD; ++i) load(i, h[i]);
    }
    float mu = 0.0f;
    if constexpr (MEAN) {
#pragma unroll HELD
        for (uint32_t i = 0; i < nch; ++i) {
            float (&v)[8] = h[NCH == kLong ? 0 : i];
            if (NCH == kLong) load(i, v);
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k) mu += v[k];
        }
        mu = row_sum(mu, tpr, slots[2]) * p.inv_cols;
        if (t == 0 && p.mean) p.mean[r] = mu;
    }
#pragma unroll HELD
    for (uint32_t i = 0; i < nch; ++i) {
        float (&v)[8] = h[NCH == kLong ? 0 : i];
        if (NCH == kLong) load(i, v);
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) {
            if (MEAN) {
                const float d = 8 * (i * tpr + t) + k < p.cols ? v[k] - mu : 0.0f;
                sum += d * d;
            } else {
                sum += v[k] * v[k];
            }
        }
    }
    const float s = rsqrtf(row_sum(sum, tpr, slots[0]) * p.inv_cols + p.eps);
    if (t == 0 && p.rstd) p.rstd[r] = s;

    auto normed = [&](uint32_t i, const float (&v)[8], float (&o)[8]) {
        const uint32_t c = 8 * (i * tpr + t);
        if (p.w) load8<VEC>(p.w, p.w_dt, c, p.cols, o);
        if constexpr (MEAN) {
            float q[8];
            if (p.b) load8<VEC>(p.b, p.w_dt, c, p.cols, q);
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k) {
                const float n = c + k < p.cols ? (v[k] - mu) * s : 0.0f;
                o[k] = p.w ? n * o[k] : n;
                if (p.b) o[k] += q[k];
            }
        } else {
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k) o[k] = p.w ? v[k] * s * o[k] : v[k] * s;
        }
    };
    auto amax8 = [&](const float (&o)[8]) {
        float m = 0.0f;
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) m = max_nan(m, fabsf(o[k]));
        return m;
    };
    Divisor by{};
    const bool e4m3 = p.y_dt == DTT_E4M3, row_scale = e4m3 && p.group_lanes == 0;
    if (row_scale) {
        float m = 0.0f;
#pragma unroll HELD
        for (uint32_t i = 0; i < nch; ++i) {
            float (&v)[8] = h[NCH == kLong ? 0 : i];
            float o[8];
            if (NCH == kLong) load(i, v);
            normed(i, v, o);
            m = max_nan(m, amax8(o));
        }
        const float scale = scale_of(row_max(m, tpr, slots[1]));
        if (t == 0) p.scales[r] = scale;
        by = divisor_of(scale);
    }
#pragma unroll HELD
    for (uint32_t i = 0; i < nch; ++i) {
        float (&v)[8] = h[NCH == kLong ? 0 : i];
        float o[8];
        const uint32_t c = 8 * (i * tpr + t);
        if (NCH == kLong) load(i, v);
        normed(i, v, o);
        if (e4m3 && !row_scale) {
            float m = amax8(o);
            for (uint32_t d = p.group_lanes >> 1; d > 0; d >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
            const float scale = scale_of(m);
            by = divisor_of(scale);
            if (t % p.group_lanes == 0 && c < p.cols)
                p.scales[r * p.groups + c / (8 * p.group_lanes)] = scale;
        }
        if (e4m3) {
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k) o[k] = quotient(o[k], by);
        }
        if (res_out) store8<VEC>(res_out, p.res_dt, c, p.cols, v);
        store8<VEC>(y, p.y_dt, c, p.cols, o);
    }
}

// The weight's gradient where there are few rows: it does not wait for the rows' means, so that CTAs of the same
// launch add it up, 32 columns at a time, a warp every `warps`-th row, the warps' sums in their order.
template <bool MEAN>
__device__ __forceinline__ void weight_columns(const BwdParams& p) {
    __shared__ float sums[MEAN ? 2 : 1][kBwdThreads / 32][32];
    constexpr uint32_t N = 4;
    wait_previous();
    const uint32_t t = threadIdx.y * blockDim.x + threadIdx.x, lane = t % 32, warp = t / 32, warps = blockDim.x * blockDim.y / 32;
    for (uint32_t b = blockIdx.x - p.partials; b < (p.cols + 31) / 32; b += gridDim.x - p.partials) {
        const uint32_t c = 32 * b + lane;
        uint32_t cs[N];
#pragma unroll
        for (uint32_t n = 0; n < N; ++n) cs[n] = min(c, p.cols - 1);
        float v = 0.0f, u = 0.0f;
        for (uint64_t r0 = warp; r0 < p.rows; r0 += N * warps) {
            const char *gs[N], *hs[N];
            float g[N], h[N], s[N], mu[N];
#pragma unroll
            for (uint32_t n = 0; n < N; ++n) {
                const uint64_t r = min(r0 + n * warps, p.rows - 1);
                gs[n] = p.dy + r * p.dy_pitch;
                hs[n] = p.h + r * p.h_pitch;
                s[n] = p.rstd[r];
                if (MEAN) mu[n] = p.mean[r];
            }
            gather(gs, p.dy_dt, cs, g);
            gather(hs, p.h_dt, cs, h);
#pragma unroll
            for (uint32_t n = 0; n < N; ++n)
                if (r0 + n * warps < p.rows) {
                    v += g[n] * ((MEAN ? h[n] - mu[n] : h[n]) * s[n]);
                    if (MEAN) u += g[n];
                }
        }
        sums[0][warp][lane] = v;
        if (MEAN) sums[MEAN][warp][lane] = u;
        __syncthreads();
        if (warp == 0) {
            for (uint32_t i = 1; i < warps; ++i) {
                v += sums[0][i][lane];
                if (MEAN) u += sums[MEAN][i][lane];
            }
            if (c < p.cols && (!MEAN || p.dweight)) p.dweight[c] = v;
            if (MEAN && c < p.cols && p.dbias) p.dbias[c] = u;
        }
        __syncthreads();
    }
}

// ---- short rows --------------------------------------------------------------------------------
// A row by `lanes` neighbouring lanes of a warp (a power of two), a chunk each; a CTA has 256 / lanes rows.  A
// thread's loads all go out before the first value is used, and many CTAs hide them: with two or four rows a
// thread under way the forward pass of 300000 x 128 (bf16 to 8 bits) took 58 and 82 us where one took 57.
// Behind another call it takes 59 (bf16 52), 0.67 (0.88) of the copy rate; the exact quotients are 2 us of it.  The layer norm
// (bf16): 67, 0.67.
template <bool MEAN>
__global__ void __launch_bounds__(256) norm_fwd_short_kernel(const __grid_constant__ FwdParams p, uint32_t lanes) {
    launch_next();
    wait_previous();
    const uint32_t t = threadIdx.x, l = t & (lanes - 1), c = 8 * l;
    const uint64_t r = (uint64_t)blockIdx.x * (256 / lanes) + t / lanes, row = min(r, p.rows - 1);
    const bool in = c < p.cols, mine = in && r < p.rows;
    const uint32_t from = in ? c : 0;               // the lanes past the row read its first chunk
    Raw8 xs = raw8(p.x + row * p.x_pitch + from * (p.x_dt == DTT_BF16 ? 2 : 4), p.x_dt), qs{}, ws{}, bs{};
    if (p.res) qs = raw8(p.res + row * p.res_pitch + from * (p.res_dt == DTT_BF16 ? 2 : 4), p.res_dt);
    if (p.w) ws = raw8(p.w + from * (p.w_dt == DTT_BF16 ? 2 : 4), p.w_dt);
    if (MEAN && p.b) bs = raw8(p.b + from * (p.w_dt == DTT_BF16 ? 2 : 4), p.w_dt);
    float h[8], o[8], sum = 0.0f;
    expand8(xs, p.x_dt, h);
    if (p.res) {
        expand8(qs, p.res_dt, o);
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) h[k] += o[k];
    }
    float mu = 0.0f;
    if constexpr (MEAN) {
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) mu += in ? h[k] : 0.0f;
        for (uint32_t d = lanes / 2; d > 0; d /= 2) mu += __shfl_xor_sync(0xFFFFFFFFu, mu, d);
        mu *= p.inv_cols;
        if (mine && l == 0 && p.mean) p.mean[r] = mu;
    }
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) {
        if (!in) h[k] = mu;
        if (MEAN) sum += (h[k] - mu) * (h[k] - mu);
        else sum += h[k] * h[k];
    }
    for (uint32_t d = lanes / 2; d > 0; d /= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    const float s = rsqrtf(sum * p.inv_cols + p.eps);
    if (mine && l == 0 && p.rstd) p.rstd[r] = s;
    if (p.w) expand8(ws, p.w_dt, o);
    float m = 0.0f, q[8];
    if (MEAN && p.b) expand8(bs, p.w_dt, q);
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) {
        const float n = MEAN ? h[k] - mu : h[k];
        o[k] = p.w ? n * s * o[k] : n * s;
        if (MEAN && p.b) o[k] += q[k];
        m = max_nan(m, fabsf(o[k]));
    }
    if (p.y_dt == DTT_E4M3) {
        const uint32_t share = p.group_lanes == 0 || p.group_lanes > lanes ? lanes : p.group_lanes;   // of a scale
        if (!in) m = 0.0f;
        for (uint32_t d = share / 2; d > 0; d /= 2) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
        const float scale = scale_of(m);
        const Divisor by = divisor_of(scale);
        if (mine && (l & (share - 1)) == 0) p.scales[p.group_lanes ? r * p.groups + l / share : r] = scale;
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) o[k] = quotient(o[k], by);
    }
    if (!mine) return;
    if (p.res_out) store8<true>(p.res_out + r * p.res_out_pitch, p.res_dt, c, p.cols, h);
    store8<true>(p.y + r * p.y_pitch, p.y_dt, c, p.cols, o);
}

// The same split; a CTA walks over rows, each thread at the same columns, whose part of the weight's gradient
// adds up in its registers; at the end the CTA's rows' sums, in their order, become its partial row.
// 300000 x 128 in bf16: 62 us, 0.73 of the copy rate; the layer norm 65, 0.70.
template <bool MEAN>
__global__ void __launch_bounds__(256, 4) norm_bwd_short_kernel(const __grid_constant__ BwdParams p, uint32_t lanes) {
    launch_next();
    if (blockIdx.x >= p.partials) return weight_columns<MEAN>(p);
    wait_previous();
    __shared__ float sums[(MEAN ? 2 : 1) * 256 * 8];
    const uint32_t t = threadIdx.x, l = t & (lanes - 1), c = 8 * l, at_a_time = 256 / lanes;
    const bool in = c < p.cols;
    const uint32_t from = in ? c : 0, ge = p.dy_dt == DTT_BF16 ? 2 : 4, he = p.h_dt == DTT_BF16 ? 2 : 4;
    float w[8], acc[8], acc_b[8];
    if (p.w) expand8(raw8(p.w + from * (p.w_dt == DTT_BF16 ? 2 : 4), p.w_dt), p.w_dt, w);
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) {
        acc[k] = acc_b[k] = 0.0f;
        if (!p.w) w[k] = 1.0f;
    }
    for (uint64_t r0 = (uint64_t)blockIdx.x * at_a_time; r0 < p.rows; r0 += (uint64_t)p.partials * at_a_time) {
        const uint64_t r = r0 + t / lanes, row = min(r, p.rows - 1);
        const bool mine = in && r < p.rows;
        const Raw8 gs = raw8(p.dy + row * p.dy_pitch + from * ge, p.dy_dt), hs = raw8(p.h + row * p.h_pitch + from * he, p.h_dt);
        Raw8 ds{};
        if (p.dres) ds = raw8(p.dres + row * p.dres_pitch + from * he, p.h_dt);
        const float s = p.rstd[row], mu = MEAN ? p.mean[row] : 0.0f;
        float g[8], n[8], dot = 0.0f, all = 0.0f;
        expand8(gs, p.dy_dt, g);
        expand8(hs, p.h_dt, n);
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) {
            n[k] = (MEAN ? n[k] - mu : n[k]) * s;
            if (mine) acc[k] += g[k] * n[k];
            if (MEAN && mine) acc_b[k] += g[k];
            g[k] *= w[k];
            if (in) dot += g[k] * n[k];
            if (MEAN && in) all += g[k];
        }
        for (uint32_t d = lanes / 2; d > 0; d /= 2) {
            dot += __shfl_xor_sync(0xFFFFFFFFu, dot, d);
            if (MEAN) all += __shfl_xor_sync(0xFFFFFFFFu, all, d);
        }
        const float m = dot * p.inv_cols, a = all * p.inv_cols;
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) g[k] = s * ((MEAN ? g[k] - a : g[k]) - n[k] * m);
        if (p.dres) {
            expand8(ds, p.h_dt, n);
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k) g[k] += n[k];
        }
        if (mine) store8<true>(p.dx + r * p.dx_pitch, p.h_dt, c, p.cols, g);
    }
    if (!p.partial) return;
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) {                              // 256 / lanes rows of 8 lanes columns
        sums[8 * t + k] = acc[k];
        if (MEAN) sums[MEAN * 256 * 8 + 8 * t + k] = acc_b[k];
    }
    __syncthreads();
    if (t < p.cols) {
        float v = 0.0f, u = 0.0f;
        for (uint32_t i = 0; i < at_a_time; ++i) {
            v += sums[i * 8 * lanes + t];
            if (MEAN) u += sums[MEAN * 256 * 8 + i * 8 * lanes + t];
        }
        p.partial[(uint64_t)blockIdx.x * p.cols + t] = v;
        if (MEAN) p.partial_b[(uint64_t)blockIdx.x * p.cols + t] = u;
    }
}

// A CTA walks over rows: each thread keeps the same columns for all of them, so the weight's gradient adds up
// in its registers and is written once, as the CTA's partial row (kLong: in the partial row itself).
// 2000 x 16384 in f32: 173 us, 0.45 of the copy rate, bound as the forward pass; the layer norm 243, 0.32.  kLong adds up in the partial rows
// in memory: the layer norm's 1000 x 70000 (bf16) 1040 us, 0.08.
template <bool MEAN, uint32_t NCH, bool VEC>
__global__ void __launch_bounds__(kBwdThreads) norm_bwd_kernel(const __grid_constant__ BwdParams p) {
    launch_next();
    if (blockIdx.x >= p.partials) return weight_columns<MEAN>(p);
    wait_previous();
    __shared__ float slots[2][64];
    const uint32_t tpr = blockDim.x, t = threadIdx.x;
    const uint32_t me = blockIdx.x;
    constexpr uint32_t HELD = NCH == kLong ? 1 : NCH;
    const uint32_t nch = NCH == kLong ? (p.cols + 8 * tpr - 1) / (8 * tpr) : NCH;
    float acc[HELD][8], acc_b[HELD][8];
#pragma unroll
    for (uint32_t i = 0; i < HELD; ++i)
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) acc[i][k] = acc_b[i][k] = 0.0f;
    float* part = p.partial ? p.partial + (uint64_t)blockIdx.x * p.cols : nullptr;
    float* part_b = MEAN && p.partial ? p.partial_b + (uint64_t)blockIdx.x * p.cols : nullptr;

    uint32_t turn = 0;
    for (uint64_t r = me; r < p.rows; r += p.walkers, turn ^= 1) {
        const char* dyr = p.dy + r * p.dy_pitch;
        const char* hr = p.h + r * p.h_pitch;
        const char* dresr = p.dres ? p.dres + r * p.dres_pitch : nullptr;
        char* dxr = p.dx + r * p.dx_pitch;
        const float s = p.rstd[r], mu = MEAN ? p.mean[r] : 0.0f;
        float g[HELD][8], n[HELD][8];               // dy, the normed row
        auto load = [&](uint32_t i, float (&gv)[8], float (&nv)[8]) {
            const uint32_t c = 8 * (i * tpr + t);
            load8<VEC>(dyr, p.dy_dt, c, p.cols, gv);
            load8<VEC>(hr, p.h_dt, c, p.cols, nv);
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k) nv[k] = (MEAN ? nv[k] - mu : nv[k]) * s;
        };
        if constexpr (NCH != kLong) {
#pragma unroll
            for (uint32_t i = 0; i < HELD; ++i) load(i, g[i], n[i]);
        }
        float dot = 0.0f, all = 0.0f;
#pragma unroll HELD
        for (uint32_t i = 0; i < nch; ++i) {
            const uint32_t j = NCH == kLong ? 0 : i, c = 8 * (i * tpr + t);
            if (NCH == kLong) load(i, g[j], n[j]);
            if (part) {
#pragma unroll
                for (uint32_t k = 0; k < 8; ++k) {
                    if (NCH != kLong) {
                        acc[j][k] += g[j][k] * n[j][k];
                        if (MEAN) acc_b[j][k] += g[j][k];
                    } else if (c + k < p.cols) {
                        part[c + k] = (r == me ? 0.0f : part[c + k]) + g[j][k] * n[j][k];
                        if (MEAN) part_b[c + k] = (r == me ? 0.0f : part_b[c + k]) + g[j][k];
                    }
                }
            }
            if (p.w) {
                float w[8];
                load8<VEC>(p.w, p.w_dt, c, p.cols, w);
#pragma unroll
                for (uint32_t k = 0; k < 8; ++k) g[j][k] *= w[k];
            }
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k) {
                dot += g[j][k] * n[j][k];
                if (MEAN) all += g[j][k];
            }
        }
        const float2 means = row_means<MEAN>(dot, all, tpr, slots[turn], p.inv_cols);
        const float m = means.x, a = means.y;
#pragma unroll HELD
        for (uint32_t i = 0; i < nch; ++i) {
            const uint32_t j = NCH == kLong ? 0 : i, c = 8 * (i * tpr + t);
            if (NCH == kLong) {
                load(i, g[j], n[j]);
                if (p.w) {
                    float w[8];
                    load8<VEC>(p.w, p.w_dt, c, p.cols, w);
#pragma unroll
                    for (uint32_t k = 0; k < 8; ++k) g[j][k] *= w[k];
                }
            }
            float o[8];
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k) o[k] = s * ((MEAN ? g[j][k] - a : g[j][k]) - n[j][k] * m);
            if (dresr) {
                float q[8];
                load8<VEC>(dresr, p.h_dt, c, p.cols, q);
#pragma unroll
                for (uint32_t k = 0; k < 8; ++k) o[k] += q[k];
            }
            store8<VEC>(dxr, p.h_dt, c, p.cols, o);
        }
    }
    if (part && NCH != kLong) {
#pragma unroll
        for (uint32_t i = 0; i < HELD; ++i)
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k) {
                const uint32_t c = 8 * (i * tpr + t) + k;
                if (c < p.cols) part[c] = acc[i][k];
                if (MEAN && c < p.cols) part_b[c] = acc_b[i][k];
            }
    }
}

// ---- elements ----------------------------------------------------------------------------------
// A warp holds 32 E neighbouring columns, a thread every 32nd of them: an access is contiguous over the
// warp, and a group of 32, 64 or 128 columns is one, two or four of each of its threads'.
template <uint32_t E>
__device__ __forceinline__ uint32_t column_of(uint32_t k) {
    return threadIdx.x / 32 * (32 * E) + 32 * k + threadIdx.x % 32;
}

// Whether the warp's columns all lie in the row: no address and no store needs a check of its own then.
template <uint32_t E>
__device__ __forceinline__ bool whole_warp(uint32_t cols) {
    return (threadIdx.x / 32 + 1) * (32 * E) <= cols;
}

// The thread's columns of a row (zeros from `cols` on).  The loads go out together (gather's reasons).
template <uint32_t E>
__device__ __forceinline__ void load_elements(const char* row, uint32_t dt, uint32_t cols, float (&v)[E]) {
    const uint32_t c0 = column_of<E>(0);
    if (whole_warp<E>(cols)) {
        if (dt == DTT_BF16) {
            const uint16_t* at = reinterpret_cast<const uint16_t*>(row) + c0;
            uint16_t raw[E];
#pragma unroll
            for (uint32_t k = 0; k < E; ++k) raw[k] = at[32 * k];
#pragma unroll
            for (uint32_t k = 0; k < E; ++k) v[k] = __uint_as_float((uint32_t)raw[k] << 16);
        } else {
            const float* at = reinterpret_cast<const float*>(row) + c0;
#pragma unroll
            for (uint32_t k = 0; k < E; ++k) v[k] = at[32 * k];
        }
        return;
    }
    const char* rows[E];
    uint32_t c[E];
#pragma unroll
    for (uint32_t k = 0; k < E; ++k) {
        rows[k] = row;
        c[k] = min(c0 + 32 * k, cols - 1);
    }
    gather(rows, dt, c, v);
#pragma unroll
    for (uint32_t k = 0; k < E; ++k)
        if (c0 + 32 * k >= cols) v[k] = 0.0f;
}

template <uint32_t E, bool WHOLE>
__device__ __forceinline__ void store_elements_as(char* row, uint32_t dt, uint32_t left, const float (&v)[E]) {
    if (dt == DTT_BF16) {
#pragma unroll
        for (uint32_t k = 0; k < E; ++k)
            if (WHOLE || 32 * k < left) reinterpret_cast<uint16_t*>(row)[32 * k] = (uint16_t)pack_bf16(v[k], 0.0f);
    } else if (dt == DTT_F32) {
#pragma unroll
        for (uint32_t k = 0; k < E; ++k)
            if (WHOLE || 32 * k < left) reinterpret_cast<float*>(row)[32 * k] = v[k];
    } else {
#pragma unroll
        for (uint32_t k = 0; k < E; ++k)
            if (WHOLE || 32 * k < left) reinterpret_cast<uint8_t*>(row)[32 * k] = (uint8_t)pack_e4m3(v[k], 0.0f);
    }
}

template <uint32_t E>
__device__ __forceinline__ void store_elements(char* row, uint32_t dt, uint32_t cols, const float (&v)[E]) {
    const uint32_t c0 = column_of<E>(0);
    char* at = row + (uint64_t)c0 * (dt == DTT_BF16 ? 2 : dt == DTT_F32 ? 4 : 1);
    if (whole_warp<E>(cols)) store_elements_as<E, true>(at, dt, 0, v);
    else store_elements_as<E, false>(at, dt, c0 < cols ? cols - c0 : 0, v);
}

// The scales of row r, and its values divided by them.
template <uint32_t E>
__device__ __forceinline__ void scale_elements(const FwdParams& p, uint64_t r, float* slot, float (&v)[E]) {
    const uint32_t c = column_of<E>(0);
    if (p.group_lanes == 0) {
        float m = 0.0f;
#pragma unroll
        for (uint32_t k = 0; k < E; ++k) m = max_nan(m, fabsf(v[k]));
        const float scale = scale_of(row_max(m, blockDim.x, slot));
        if (threadIdx.x == 0) p.scales[r] = scale;
        const Divisor by = divisor_of(scale);
#pragma unroll
        for (uint32_t k = 0; k < E; ++k) v[k] = quotient(v[k], by);
        return;
    }
    const uint32_t per = p.group_lanes / 4;                   // of a thread's columns: 1, 2 or 4
#pragma unroll
    for (uint32_t k = 0; k < E; k += 4) {
        float m[4];
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) m[i] = fabsf(v[k + i]);
        if (per >= 2) {
            m[0] = m[1] = max_nan(m[0], m[1]);
            m[2] = m[3] = max_nan(m[2], m[3]);
        }
        if (per == 4) m[0] = m[1] = m[2] = m[3] = max_nan(m[0], m[2]);
        Divisor by{};
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
            if (i % per == 0) {
                const float scale = scale_of(warp_max(m[i]));
                by = divisor_of(scale);
                if (threadIdx.x % 32 == 0 && c + 32 * (k + i) < p.cols) p.scales[r * p.groups + (c + 32 * (k + i)) / (32 * per)] = scale;
            }
            v[k + i] = quotient(v[k + i], by);
        }
    }
}

// The thread's columns past the row take its mean: they are zero once it comes off.
template <uint32_t E>
__device__ __forceinline__ void centre(float (&v)[E], float mu, uint32_t cols) {
    if (whole_warp<E>(cols)) return;
#pragma unroll
    for (uint32_t k = 0; k < E; ++k)
        if (column_of<E>(k) >= cols) v[k] = mu;
}

// A row a CTA, or a warp (blockDim.y of them).  600 x 3001 in bf16: 5.7 us back to back, the loads' latency.
template <bool MEAN, uint32_t E>
__global__ void __launch_bounds__(kFwdThreads) norm_fwd_elements_kernel(const __grid_constant__ FwdParams p) {
    launch_next();
    wait_previous();
    __shared__ float slots[MEAN ? 3 : 2][32];
    const uint64_t r = (uint64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (r >= p.rows) return;                        // a whole warp: rows share no barrier
    float h[E], o[E], b[E], mu = 0.0f;
    load_elements(p.x + r * p.x_pitch, p.x_dt, p.cols, h);
    if (p.res) {
        load_elements(p.res + r * p.res_pitch, p.res_dt, p.cols, o);
#pragma unroll
        for (uint32_t k = 0; k < E; ++k) h[k] += o[k];
    }
    if (p.w) load_elements(p.w, p.w_dt, p.cols, o);
    if (MEAN && p.b) load_elements(p.b, p.w_dt, p.cols, b);
    if constexpr (MEAN) {
#pragma unroll
        for (uint32_t k = 0; k < E; ++k) mu += h[k];
        mu = row_sum(mu, blockDim.x, slots[2]) * p.inv_cols;
        if (threadIdx.x == 0 && p.mean) p.mean[r] = mu;
        centre(h, mu, p.cols);
    }
    float sum = 0.0f;
#pragma unroll
    for (uint32_t k = 0; k < E; ++k) sum += MEAN ? (h[k] - mu) * (h[k] - mu) : h[k] * h[k];
    const float s = rsqrtf(row_sum(sum, blockDim.x, slots[0]) * p.inv_cols + p.eps);
    if (threadIdx.x == 0 && p.rstd) p.rstd[r] = s;
    if (p.res_out) store_elements(p.res_out + r * p.res_out_pitch, p.res_dt, p.cols, h);
#pragma unroll
    for (uint32_t k = 0; k < E; ++k) {
        if (MEAN) h[k] -= mu;
        h[k] = p.w ? h[k] * s * o[k] : h[k] * s;
        if (MEAN && p.b) h[k] += b[k];
    }
    if (p.y_dt == DTT_E4M3) scale_elements(p, r, slots[1], h);
    store_elements(p.y + r * p.y_pitch, p.y_dt, p.cols, h);
}

// Partial row of a CTA whose warps took rows of their own: their sums, in the warps' order.
template <uint32_t N>
__device__ __forceinline__ void add_warps(const float (&sums)[kWarpRows][N], float* part, uint32_t cols) {
    __syncthreads();
    for (uint32_t c = threadIdx.y * 32 + threadIdx.x; c < cols; c += kWarpRows * 32) {
        float v = sums[0][c];
#pragma unroll
        for (uint32_t i = 1; i < kWarpRows; ++i) v += sums[i][c];
        part[c] = v;
    }
}

// As the chunk form: a CTA or a warp walks over rows, the weight's gradient in its registers.  100 x 1021 in bf16:
// 5 us back to back with the sum of the partial rows; 300000 x 101 167 us, 0.21 of the copy rate, a 2-byte element a lane.
template <bool MEAN, uint32_t E>
__global__ void __launch_bounds__(kBwdThreads) norm_bwd_elements_kernel(const __grid_constant__ BwdParams p) {
    launch_next();
    if (blockIdx.x >= p.partials) return weight_columns<MEAN>(p);
    wait_previous();
    __shared__ float slots[2][64];
    __shared__ float sums[kWarpRows][32 * E];
    const uint32_t T = blockDim.x;
    float acc[E], acc_b[E], w[E];
#pragma unroll
    for (uint32_t k = 0; k < E; ++k) {
        acc[k] = acc_b[k] = 0.0f;
        w[k] = 1.0f;
    }
    if (p.w) load_elements(p.w, p.w_dt, p.cols, w);
    uint32_t turn = 0;
    for (uint64_t r = (uint64_t)blockIdx.x * blockDim.y + threadIdx.y; r < p.rows; r += p.walkers, turn ^= 1) {
        const float s = p.rstd[r], mu = MEAN ? p.mean[r] : 0.0f;
        float g[E], n[E], q[E];
        load_elements(p.dy + r * p.dy_pitch, p.dy_dt, p.cols, g);
        load_elements(p.h + r * p.h_pitch, p.h_dt, p.cols, n);
        if (p.dres) load_elements(p.dres + r * p.dres_pitch, p.h_dt, p.cols, q);
        float dot = 0.0f, all = 0.0f;
#pragma unroll
        for (uint32_t k = 0; k < E; ++k) {
            n[k] = (MEAN ? n[k] - mu : n[k]) * s;
            acc[k] += g[k] * n[k];
            if (MEAN) acc_b[k] += g[k];
            g[k] *= w[k];
            dot += g[k] * n[k];
            if (MEAN) all += g[k];
        }
        const float2 means = row_means<MEAN>(dot, all, T, slots[turn], p.inv_cols);
#pragma unroll
        for (uint32_t k = 0; k < E; ++k) {
            g[k] = s * ((MEAN ? g[k] - means.y : g[k]) - n[k] * means.x);
            if (p.dres) g[k] += q[k];
        }
        store_elements(p.dx + r * p.dx_pitch, p.h_dt, p.cols, g);
    }
    if (!p.partial) return;
    float* part = p.partial + (uint64_t)blockIdx.x * p.cols;
    float* part_b = MEAN ? p.partial_b + (uint64_t)blockIdx.x * p.cols : nullptr;
    if (blockDim.y == 1) {
        store_elements(reinterpret_cast<char*>(part), DTT_F32, p.cols, acc);
        if (MEAN) store_elements(reinterpret_cast<char*>(part_b), DTT_F32, p.cols, acc_b);
        return;
    }
#pragma unroll
    for (uint32_t k = 0; k < E; ++k) sums[threadIdx.y][32 * k + threadIdx.x] = acc[k];
    add_warps(sums, part, p.cols);
    if (MEAN) {
        __syncthreads();
#pragma unroll
        for (uint32_t k = 0; k < E; ++k) sums[threadIdx.y][32 * k + threadIdx.x] = acc_b[k];
        add_warps(sums, part_b, p.cols);
    }
}

// ---- ring --------------------------------------------------------------------------------------
// Bounded; false when it ran out.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity) {
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

__device__ __forceinline__ void bulk_load(uint32_t dst, const char* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

// Rows that do not arrive.  To a thread whose wait for a row runs out (`lost`) that row and all later ones are
// NaN, and through the rows' sums to the others.  Thread 0 starts copies only into stages whose last row it has
// seen arrive: where it gives up it starts no more, and waits in the end for those under way, of the CTA's
// rows before `next`.
__device__ __noinline__ void await_copies(uint64_t* full, uint32_t S, uint64_t next, uint32_t step) {
    const uint64_t started = (next - blockIdx.x) / step;
    for (uint64_t n = started > S ? started - S : 0; n < started; ++n) (void)bar_wait(saddr(full + n % S), n / S & 1);
}

constexpr float kNan = __builtin_nanf("");

template <uint32_t N>
__device__ __forceinline__ void make_nan(float (&v)[N]) {
#pragma unroll
    for (uint32_t k = 0; k < N; ++k) v[k] = kNan;
}

// Rows blockIdx.x, + gridDim.x, ... by one CTA.  Stage i % S holds the row of turn i: x, then the
// residual.  Thread 0 starts the copies of turn i + S - 1 once turn i's reduction has passed its
// barrier: every thread is then done with that stage's last row (turn i - 1).  16384 x 4096 (bf16 to 8 bits,
// groups of 128): 79 us, 0.88 of the copy rate, the issue slots 73 % full.
template <uint32_t NCH>
__global__ void __launch_bounds__(NCH == 1 ? 256 : kRingThreads, NCH == 1 ? 6 : NCH == 2 ? 2 : 1) rmsnorm_fwd_ring_kernel(const __grid_constant__ FwdParams p, uint32_t S) {
    launch_next();
    extern __shared__ __align__(128) uint8_t stages[];
    __shared__ float slots[2][2][32];
    __shared__ uint64_t full[ring::kStages];
    const uint32_t T = blockDim.x, t = threadIdx.x;
    const uint32_t xb = p.cols * (p.x_dt == DTT_BF16 ? 2 : 4), rb = p.res ? p.cols * (p.res_dt == DTT_BF16 ? 2 : 4) : 0;
    const uint32_t stage_bytes = xb + rb;
    uint64_t next = blockIdx.x;                     // thread 0: the row to be fetched next, and its stage
    uint32_t next_st = 0;
    auto start = [&] {
        if (next >= p.rows) return;
        const uint64_t r = next;
        const uint32_t bar = saddr(full + next_st), dst = saddr(stages) + next_st * stage_bytes;
        next += gridDim.x;
        if (++next_st == S) next_st = 0;
        bar_expect_tx(bar, stage_bytes);
        bulk_load(dst, p.x + r * p.x_pitch, xb, bar);
        if (rb) bulk_load(dst + xb, p.res + r * p.res_pitch, rb, bar);
    };
    if (t == 0) {
        for (uint32_t i = 0; i < S; ++i) bar_init(saddr(full + i), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    wait_previous();
    if (t == 0)
        for (uint32_t i = 0; i + 1 < S; ++i) start();
    float w[NCH][8];
#pragma unroll
    for (uint32_t i = 0; i < NCH; ++i)
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) w[i][k] = 1.0f;
    if (p.w) {
        Raw8 ws[NCH];
#pragma unroll
        for (uint32_t i = 0; i < NCH; ++i) {
            const uint32_t c = 8 * (i * T + t);
            ws[i] = raw8(p.w + (c < p.cols ? c : 0) * (p.w_dt == DTT_BF16 ? 2 : 4), p.w_dt);
        }
#pragma unroll
        for (uint32_t i = 0; i < NCH; ++i) expand8(ws[i], p.w_dt, w[i]);
    }
    __syncthreads();

    uint32_t st = 0, phase = 0;
    uint32_t turn = 0;
    bool lost = false;
    for (uint64_t r = blockIdx.x; r < p.rows; r += gridDim.x, turn ^= 1) {
        lost = lost || DTT_NORM_ROW_LATE || !bar_wait(saddr(full + st), phase);
        const char* row = reinterpret_cast<const char*>(stages) + st * stage_bytes;
        float h[NCH][8], sum = 0.0f;
#pragma unroll
        for (uint32_t i = 0; i < NCH; ++i) load8<true>(row, p.x_dt, 8 * (i * T + t), p.cols, h[i]);
        if (rb) {
#pragma unroll
            for (uint32_t i = 0; i < NCH; ++i) {
                float q[8];
                load8<true>(row + xb, p.res_dt, 8 * (i * T + t), p.cols, q);
#pragma unroll
                for (uint32_t k = 0; k < 8; ++k) h[i][k] += q[k];
            }
        }
#pragma unroll
        for (uint32_t i = 0; i < NCH; ++i)
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k) sum += h[i][k] * h[i][k];
        if (lost) sum = kNan;
        const float s = rsqrtf(row_sum(sum, T, slots[turn][0]) * p.inv_cols + p.eps);
        if (t == 0) {
            if (!lost) start();
            if (p.rstd) p.rstd[r] = s;
        }
        if (p.res_out) {
#pragma unroll
            for (uint32_t i = 0; i < NCH; ++i) {
                if (lost) make_nan(h[i]);
                store8<true>(p.res_out + r * p.res_out_pitch, p.res_dt, 8 * (i * T + t), p.cols, h[i]);
            }
        }
#pragma unroll
        for (uint32_t i = 0; i < NCH; ++i)
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k) h[i][k] = h[i][k] * s * w[i][k];      // s w alone may overflow
        if (p.y_dt == DTT_E4M3) {
            float m[NCH];
#pragma unroll
            for (uint32_t i = 0; i < NCH; ++i) {
                m[i] = 0.0f;
#pragma unroll
                for (uint32_t k = 0; k < 8; ++k) m[i] = max_nan(m[i], fabsf(h[i][k]));
            }
            if (p.group_lanes == 0) {
                float all = m[0];
#pragma unroll
                for (uint32_t i = 1; i < NCH; ++i) all = max_nan(all, m[i]);
                const float scale = scale_of(row_max(all, T, slots[turn][1]));
                if (t == 0) p.scales[r] = scale;
                const Divisor by = divisor_of(scale);
#pragma unroll
                for (uint32_t i = 0; i < NCH; ++i)
#pragma unroll
                    for (uint32_t k = 0; k < 8; ++k) h[i][k] = quotient(h[i][k], by);
            } else {
#pragma unroll
                for (uint32_t i = 0; i < NCH; ++i) {
                    for (uint32_t d = p.group_lanes >> 1; d > 0; d >>= 1)
                        m[i] = max_nan(m[i], __shfl_xor_sync(0xFFFFFFFFu, m[i], d));
                    const float scale = scale_of(m[i]);
                    const Divisor by = divisor_of(scale);
                    const uint32_t c = 8 * (i * T + t);
                    if (t % p.group_lanes == 0 && c < p.cols) p.scales[r * p.groups + c / (8 * p.group_lanes)] = scale;
#pragma unroll
                    for (uint32_t k = 0; k < 8; ++k) h[i][k] = quotient(h[i][k], by);
                }
            }
        }
#pragma unroll
        for (uint32_t i = 0; i < NCH; ++i) store8<true>(p.y + r * p.y_pitch, p.y_dt, 8 * (i * T + t), p.cols, h[i]);
        if (++st == S) { st = 0; phase ^= 1; }
    }
    if (lost && t == 0) await_copies(full, S, next, gridDim.x);
}

// ---- layer norm's ring -------------------------------------------------------------------------
// Eight columns as four pairs.  B16: the type is bf16, known when compiled.
template <bool B16>
__device__ __forceinline__ void pairs8(const char* at, uint32_t dt, Pair (&v)[4]) {
    const Raw8 q = raw8(at, B16 ? (uint32_t)DTT_BF16 : dt);
    if (B16 || dt == DTT_BF16) {
        v[0] = pair(bf16_lo(q.a.x), bf16_hi(q.a.x)), v[1] = pair(bf16_lo(q.a.y), bf16_hi(q.a.y));
        v[2] = pair(bf16_lo(q.a.z), bf16_hi(q.a.z)), v[3] = pair(bf16_lo(q.a.w), bf16_hi(q.a.w));
    } else {
        v[0] = pair(__uint_as_float(q.a.x), __uint_as_float(q.a.y)), v[1] = pair(__uint_as_float(q.a.z), __uint_as_float(q.a.w));
        v[2] = pair(__uint_as_float(q.b.x), __uint_as_float(q.b.y)), v[3] = pair(__uint_as_float(q.b.z), __uint_as_float(q.b.w));
    }
}
__device__ __forceinline__ void singles8(const Pair (&v)[4], float (&f)[8]) {
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k) {
        const float2 a = apart(v[k]);
        f[2 * k] = a.x, f[2 * k + 1] = a.y;
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (uint32_t o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// As the ring above, with the mean and the variance by one barrier: a warp takes the mean of its own columns and sums their squares
// about that, both by shuffles; the warps' sums S_w and squares Q_w then meet in shared memory, where
//     mean = sum S_w / cols,   sum (h - mean)^2 = sum Q_w + sum n_w (S_w / n_w - mean)^2
// adds what the warps' means are off by (T. F. Chan, G. H. Golub, R. J. LeVeque, 1979): no large numbers cancel.
// 16384 x 4096 (bf16 to 8 bits, groups of 128): 81 us, 0.86 of the copy rate (84 where the residual's rows stay in L2 as long as
// others).  With three CTAs of 256 threads an SM; four, whose registers spill, took 3 more, two 13, and 128 threads of four chunks
// each 12.  Two reductions with a barrier each, one value an instruction and types looked up at each access: 113.
// To bf16 95 us, 0.83; f32 throughout 185, 0.86.  Rows of 8064 columns (four chunks a thread) to bf16 175, 0.89, to 8 bits 179, 0.76;
// 30000 x 1024 51 and 53, 0.71 and 0.60.
constexpr uint32_t kLayerThreads = 256;        // of a row with two chunks a thread, at most
template <uint32_t NCH, bool B16>
__global__ void __launch_bounds__(NCH == 1 ? 128 : NCH == 2 ? kLayerThreads : kRingThreads, NCH == 1 ? 8 : NCH == 2 ? 3 : 1) layernorm_fwd_ring_kernel(const __grid_constant__ FwdParams p, uint32_t S) {
    launch_next();
    extern __shared__ __align__(128) uint8_t stages[];
    __shared__ float2 slots[2][32];
    __shared__ float tops[2][32];
    __shared__ uint64_t full[ring::kStages];
    const uint32_t T = blockDim.x, t = threadIdx.x, lane = t % 32, warp = t / 32;
    const uint32_t xe = B16 || p.x_dt == DTT_BF16 ? 2 : 4, re = B16 || p.res_dt == DTT_BF16 ? 2 : 4;
    const uint32_t xb = p.cols * xe, rb = p.res ? p.cols * re : 0;
    const uint32_t stage_bytes = xb + rb;
    uint64_t next = blockIdx.x;                     // thread 0: the row to be fetched next, and its stage
    uint32_t next_st = 0;
    auto start = [&] {
        if (next >= p.rows) return;
        const uint64_t r = next;
        const uint32_t bar = saddr(full + next_st), dst = saddr(stages) + next_st * stage_bytes;
        next += gridDim.x;
        if (++next_st == S) next_st = 0;
        bar_expect_tx(bar, stage_bytes);
        bulk_load(dst, p.x + r * p.x_pitch, xb, bar);
        if (rb) bulk_load(dst + xb, p.res + r * p.res_pitch, rb, bar);
    };
    if (t == 0) {
        for (uint32_t i = 0; i < S; ++i) bar_init(saddr(full + i), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    // columns of a warp: 256 of each of its chunks, less where the row ends
    const auto columns_of = [&](uint32_t w) {
        uint32_t n = 0;
#pragma unroll
        for (uint32_t i = 0; i < NCH; ++i) {
            const uint32_t c = 8 * (i * T + 32 * w);
            if (c < p.cols) n += min(p.cols - c, 256u);
        }
        return (float)n;
    };
    const float mine_inv = 1.0f / fmaxf(columns_of(warp), 1.0f);
    const float lanes_n = lane < T / 32 ? columns_of(lane) : 0.0f, lanes_inv = 1.0f / fmaxf(lanes_n, 1.0f);   // warp `lane`'s
    uint32_t c[NCH], scale_at[NCH];
    bool in[NCH], scales[NCH];
#pragma unroll
    for (uint32_t i = 0; i < NCH; ++i) {
        c[i] = 8 * (i * T + t);
        in[i] = c[i] < p.cols;
        scale_at[i] = p.group_lanes ? c[i] / 8 / p.group_lanes : 0;
        scales[i] = p.group_lanes ? in[i] && t % p.group_lanes == 0 : t == 0 && i == 0;
    }
    wait_previous();
    if (t == 0)
        for (uint32_t i = 0; i + 1 < S; ++i) start();
    Pair w[NCH][4], b[NCH][4];
#pragma unroll
    for (uint32_t i = 0; i < NCH; ++i) {
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) w[i][k] = both(1.0f), b[i][k] = both(0.0f);
        const uint32_t we = B16 || p.w_dt == DTT_BF16 ? 2 : 4;
        if (p.w && in[i]) pairs8<B16>(p.w + c[i] * we, p.w_dt, w[i]);
        if (p.b && in[i]) pairs8<B16>(p.b + c[i] * we, p.w_dt, b[i]);
    }
    __syncthreads();

    uint32_t st = 0, phase = 0, turn = 0;
    bool lost = false;
    for (uint64_t r = blockIdx.x; r < p.rows; r += gridDim.x, turn ^= 1) {
        lost = lost || DTT_NORM_ROW_LATE || !bar_wait(saddr(full + st), phase);
        const char* row = reinterpret_cast<const char*>(stages) + st * stage_bytes;
        Pair h[NCH][4], sum = both(0.0f);
#pragma unroll
        for (uint32_t i = 0; i < NCH; ++i) {
            // a thread past the row's end takes its first chunk, and leaves it out
            const uint32_t from = in[i] ? c[i] : 0;
            pairs8<B16>(row + from * xe, p.x_dt, h[i]);
            if (rb) {
                Pair q[4];
                pairs8<B16>(row + xb + from * re, p.res_dt, q);
#pragma unroll
                for (uint32_t k = 0; k < 4; ++k) h[i][k] = h[i][k] + q[k];
            }
        }
        if (lost) {
#pragma unroll
            for (uint32_t i = 0; i < NCH; ++i)
#pragma unroll
                for (uint32_t k = 0; k < 4; ++k) h[i][k] = both(kNan);
        }
#pragma unroll
        for (uint32_t i = 0; i < NCH; ++i) {
            if (!in[i]) continue;
            if (p.res_out) {
                float f[8];
                singles8(h[i], f);
                store8_first_out(p.res_out + r * p.res_out_pitch, B16 ? (uint32_t)DTT_BF16 : p.res_dt, c[i], f);
            }
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k) sum = sum + h[i][k];
        }
        const float2 part = apart(sum);
        const float own = warp_sum(part.x + part.y);
        const Pair centre = both(-own * mine_inv);
        Pair squares = both(0.0f);
#pragma unroll
        for (uint32_t i = 0; i < NCH; ++i) {
            if (!in[i]) continue;
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k) {
                const Pair d = h[i][k] + centre;
                squares = fma2(d, d, squares);
            }
        }
        const float2 part2 = apart(squares);
        const float own2 = warp_sum(part2.x + part2.y);
        if (lane == 0) slots[turn][warp] = make_float2(own, own2);
        __syncthreads();
        const float2 from_warp = lane < T / 32 ? slots[turn][lane] : make_float2(0.0f, 0.0f);
        const float mu = warp_sum(from_warp.x) * p.inv_cols;
        const float off = from_warp.x * lanes_inv - mu;
        const float s = rsqrtf(warp_sum(fmaf(lanes_n * off, off, from_warp.y)) * p.inv_cols + p.eps);
        if (t == 0) {
            if (!lost) start();
            if (p.mean) p.mean[r] = mu;
            if (p.rstd) p.rstd[r] = s;
        }
        const Pair less = both(-mu), by = both(s);
#pragma unroll
        for (uint32_t i = 0; i < NCH; ++i)
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k) h[i][k] = fma2((h[i][k] + less) * by, w[i][k], b[i][k]);
        if (p.y_dt == DTT_E4M3) {
            float m[NCH];
#pragma unroll
            for (uint32_t i = 0; i < NCH; ++i) {
                float f[8];
                singles8(h[i], f);
                m[i] = max3_nan(max3_nan(fabsf(f[0]), fabsf(f[1]), fabsf(f[2])), fabsf(f[3]), fabsf(f[4]));
                m[i] = max3_nan(max_nan(m[i], fabsf(f[5])), fabsf(f[6]), fabsf(f[7]));
                if (!in[i]) m[i] = 0.0f;
            }
            if (p.group_lanes == 0) {
#pragma unroll
                for (uint32_t i = 1; i < NCH; ++i) m[0] = max_nan(m[0], m[i]);
                m[0] = row_max(m[0], T, tops[turn]);
#pragma unroll
                for (uint32_t i = 1; i < NCH; ++i) m[i] = m[0];
            } else {
#pragma unroll
                for (uint32_t i = 0; i < NCH; ++i)
                    for (uint32_t d = p.group_lanes >> 1; d > 0; d >>= 1) m[i] = max_nan(m[i], __shfl_xor_sync(0xFFFFFFFFu, m[i], d));
            }
#pragma unroll
            for (uint32_t i = 0; i < NCH; ++i) {
                const float scale = scale_of(m[i]);
                const Divisor v = divisor_of(scale);
                if (scales[i]) p.scales[r * p.groups + scale_at[i]] = scale;
                // quotient() of two at a time
                const Pair inv = both(v.inv), less_d = both(-v.d);
                float f[8];
#pragma unroll
                for (uint32_t k = 0; k < 4; ++k) {
                    const Pair q = h[i][k] * inv;
                    const float2 a = apart(fma2(fma2(less_d, q, h[i][k]), inv, q));
                    f[2 * k] = a.x, f[2 * k + 1] = a.y;
                }
                if (in[i]) store8<true>(p.y + r * p.y_pitch, DTT_E4M3, c[i], p.cols, f);
            }
        } else {
#pragma unroll
            for (uint32_t i = 0; i < NCH; ++i) {
                float f[8];
                singles8(h[i], f);
                if (in[i]) store8<true>(p.y + r * p.y_pitch, p.y_dt, c[i], p.cols, f);
            }
        }
        if (++st == S) { st = 0; phase ^= 1; }
    }
    if (lost && t == 0) await_copies(full, S, next, gridDim.x);
}

// The backward pass the same way: a stage holds dy, h, then dres.  A row's latency is what the few CTAs of an SM have
// to hide, so rstd is read a turn ahead and a thread's loads from the stage go out together: 16384 x 8064 in
// bf16 153 us and not 201.  16384 x 4096 83 us with the weight's gradient, 0.95 of the copy rate; 2048 x 4096
// 18.6 us, 0.53: seven rows a CTA, then the sum of the partial rows.
template <uint32_t NCH>
__global__ void __launch_bounds__(NCH == 1 ? 256 : kRingThreads, NCH == 1 ? 4 : 1) rmsnorm_bwd_ring_kernel(const __grid_constant__ BwdParams p, uint32_t S) {
    launch_next();
    if (blockIdx.x >= p.partials) return weight_columns<false>(p);
    extern __shared__ __align__(128) uint8_t stages[];
    __shared__ float slots[2][32];
    __shared__ uint64_t full[ring::kStages];
    const uint32_t T = blockDim.x, t = threadIdx.x;
    const uint32_t gb = p.cols * (p.dy_dt == DTT_BF16 ? 2 : 4), hb = p.cols * (p.h_dt == DTT_BF16 ? 2 : 4);
    const uint32_t stage_bytes = gb + hb + (p.dres ? hb : 0);
    uint64_t next = blockIdx.x;                     // thread 0: the row to be fetched next, and its stage
    uint32_t next_st = 0;
    auto start = [&] {
        if (next >= p.rows) return;
        const uint64_t r = next;
        const uint32_t bar = saddr(full + next_st), dst = saddr(stages) + next_st * stage_bytes;
        next += p.partials;
        if (++next_st == S) next_st = 0;
        bar_expect_tx(bar, stage_bytes);
        bulk_load(dst, p.dy + r * p.dy_pitch, gb, bar);
        bulk_load(dst + gb, p.h + r * p.h_pitch, hb, bar);
        if (p.dres) bulk_load(dst + gb + hb, p.dres + r * p.dres_pitch, hb, bar);
    };
    if (t == 0) {
        for (uint32_t i = 0; i < S; ++i) bar_init(saddr(full + i), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    wait_previous();
    if (t == 0)
        for (uint32_t i = 0; i + 1 < S; ++i) start();
    float w[NCH][8], acc[NCH][8];
#pragma unroll
    for (uint32_t i = 0; i < NCH; ++i)
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) {
            w[i][k] = 1.0f;
            acc[i][k] = 0.0f;
        }
    if (p.w) {
        Raw8 ws[NCH];
#pragma unroll
        for (uint32_t i = 0; i < NCH; ++i) {
            const uint32_t c = 8 * (i * T + t);
            ws[i] = raw8(p.w + (c < p.cols ? c : 0) * (p.w_dt == DTT_BF16 ? 2 : 4), p.w_dt);
        }
#pragma unroll
        for (uint32_t i = 0; i < NCH; ++i) expand8(ws[i], p.w_dt, w[i]);
    }
    __syncthreads();

    uint32_t st = 0, phase = 0;
    uint32_t turn = 0;
    bool lost = false;
    float s_next = p.rstd[blockIdx.x];              // a turn ahead of its use
    for (uint64_t r = blockIdx.x; r < p.rows; r += p.partials, turn ^= 1) {
        const float s = s_next;
        if (r + p.partials < p.rows) s_next = p.rstd[r + p.partials];
        lost = lost || DTT_NORM_ROW_LATE || !bar_wait(saddr(full + st), phase);
        const char* row = reinterpret_cast<const char*>(stages) + st * stage_bytes;
        float g[NCH][8], n[NCH][8], dot = 0.0f;
        constexpr uint32_t G = NCH > 2 ? 1 : NCH;   // chunks whose loads go out together: what the registers allow
#pragma unroll
        for (uint32_t i0 = 0; i0 < NCH; i0 += G) {
            Raw8 gs[G], hs[G];
#pragma unroll
            for (uint32_t i = 0; i < G; ++i) {
                const uint32_t c = 8 * ((i0 + i) * T + t), from = c < p.cols ? c : 0;
                gs[i] = raw8(row + from * (p.dy_dt == DTT_BF16 ? 2 : 4), p.dy_dt);
                hs[i] = raw8(row + gb + from * (p.h_dt == DTT_BF16 ? 2 : 4), p.h_dt);
            }
#pragma unroll
            for (uint32_t i = 0; i < G; ++i) {
                float (&gi)[8] = g[i0 + i], (&ni)[8] = n[i0 + i];
                const bool in = 8 * ((i0 + i) * T + t) < p.cols;
                expand8(gs[i], p.dy_dt, gi);
                expand8(hs[i], p.h_dt, ni);
#pragma unroll
                for (uint32_t k = 0; k < 8; ++k) {
                    gi[k] = in ? gi[k] : 0.0f;
                    ni[k] = in ? ni[k] * s : 0.0f;
                    acc[i0 + i][k] += gi[k] * ni[k];
                    gi[k] *= w[i0 + i][k];
                    dot += gi[k] * ni[k];
                }
            }
        }
        if (lost) dot = kNan;
        const float m = row_sum(dot, T, slots[turn]) * p.inv_cols;
        if (t == 0 && !lost) start();
#pragma unroll
        for (uint32_t i = 0; i < NCH; ++i) {
            const uint32_t c = 8 * (i * T + t);
            float o[8];
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k) o[k] = s * (g[i][k] - n[i][k] * m);
            if (p.dres) {
                float q[8];
                load8<true>(row + gb + hb, p.h_dt, c, p.cols, q);
#pragma unroll
                for (uint32_t k = 0; k < 8; ++k) o[k] += q[k];
            }
            store8<true>(p.dx + r * p.dx_pitch, p.h_dt, c, p.cols, o);
        }
        if (++st == S) { st = 0; phase ^= 1; }
    }
    if (lost) {                                     // acc has taken rows that had not arrived
        if (t == 0) await_copies(full, S, next, p.partials);
#pragma unroll
        for (uint32_t i = 0; i < NCH; ++i) make_nan(acc[i]);
    }
    if (p.partial) {
        float* part = p.partial + (uint64_t)blockIdx.x * p.cols;
#pragma unroll
        for (uint32_t i = 0; i < NCH; ++i) store8<true>(reinterpret_cast<char*>(part), DTT_F32, 8 * (i * T + t), p.cols, acc[i]);
    }
}

// The layer norm's the same way, two values an instruction.  16384 x 4096 (bf16) 85 us, 0.93 of the copy rate, with the parameters' gradients.
template <uint32_t NCH, bool B16>
__global__ void __launch_bounds__(NCH == 1 ? 256 : kRingThreads, NCH == 1 ? 4 : 1) layernorm_bwd_ring_kernel(const __grid_constant__ BwdParams p, uint32_t S) {
    launch_next();
    if (blockIdx.x >= p.partials) return weight_columns<true>(p);
    extern __shared__ __align__(128) uint8_t stages[];
    __shared__ float slots[2][64];
    __shared__ uint64_t full[ring::kStages];
    const uint32_t T = blockDim.x, t = threadIdx.x;
    const uint32_t ge = B16 || p.dy_dt == DTT_BF16 ? 2 : 4, he = B16 || p.h_dt == DTT_BF16 ? 2 : 4;
    const uint32_t gb = p.cols * ge, hb = p.cols * he, stage_bytes = gb + hb + (p.dres ? hb : 0);
    uint64_t next = blockIdx.x;                     // thread 0: the row to be fetched next, and its stage
    uint32_t next_st = 0;
    auto start = [&] {
        if (next >= p.rows) return;
        const uint64_t r = next;
        const uint32_t bar = saddr(full + next_st), dst = saddr(stages) + next_st * stage_bytes;
        next += p.partials;
        if (++next_st == S) next_st = 0;
        bar_expect_tx(bar, stage_bytes);
        bulk_load(dst, p.dy + r * p.dy_pitch, gb, bar);
        bulk_load(dst + gb, p.h + r * p.h_pitch, hb, bar);
        if (p.dres) bulk_load(dst + gb + hb, p.dres + r * p.dres_pitch, hb, bar);
    };
    if (t == 0) {
        for (uint32_t i = 0; i < S; ++i) bar_init(saddr(full + i), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    wait_previous();
    if (t == 0)
        for (uint32_t i = 0; i + 1 < S; ++i) start();
    Pair w[NCH][4], acc[NCH][4], acc_b[NCH][4];
    uint32_t c[NCH];
    bool in[NCH];
#pragma unroll
    for (uint32_t i = 0; i < NCH; ++i) {
        c[i] = 8 * (i * T + t);
        in[i] = c[i] < p.cols;
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) w[i][k] = both(1.0f), acc[i][k] = acc_b[i][k] = both(0.0f);
        if (p.w && in[i]) pairs8<B16>(p.w + c[i] * (B16 || p.w_dt == DTT_BF16 ? 2 : 4), p.w_dt, w[i]);
    }
    __syncthreads();

    uint32_t st = 0, phase = 0, turn = 0;
    bool lost = false;
    float s_next = p.rstd[blockIdx.x], mu_next = p.mean[blockIdx.x];      // a turn ahead of their use
    for (uint64_t r = blockIdx.x; r < p.rows; r += p.partials, turn ^= 1) {
        const float s = s_next, mu = mu_next;
        if (r + p.partials < p.rows) {
            s_next = p.rstd[r + p.partials];
            mu_next = p.mean[r + p.partials];
        }
        lost = lost || DTT_NORM_ROW_LATE || !bar_wait(saddr(full + st), phase);
        const char* row = reinterpret_cast<const char*>(stages) + st * stage_bytes;
        const Pair less = both(-mu), by = both(s);
        Pair g[NCH][4], n[NCH][4], dots = both(0.0f), alls = both(0.0f);
#pragma unroll
        for (uint32_t i = 0; i < NCH; ++i) {
            if (!in[i]) continue;
            pairs8<B16>(row + c[i] * ge, p.dy_dt, g[i]);
            pairs8<B16>(row + gb + c[i] * he, p.h_dt, n[i]);
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k) {
                n[i][k] = (n[i][k] + less) * by;
                acc[i][k] = fma2(g[i][k], n[i][k], acc[i][k]);
                acc_b[i][k] = acc_b[i][k] + g[i][k];
                g[i][k] = g[i][k] * w[i][k];
                dots = fma2(g[i][k], n[i][k], dots);
                alls = alls + g[i][k];
            }
        }
        const float2 d = apart(dots), a = apart(alls);
        const float2 means = row_means<true>(lost ? kNan : d.x + d.y, a.x + a.y, T, slots[turn], p.inv_cols);
        if (t == 0 && !lost) start();
        const Pair less_m = both(-means.x), less_a = both(-means.y);
#pragma unroll
        for (uint32_t i = 0; i < NCH; ++i) {
            if (!in[i]) continue;
            Pair o[4];
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k) o[k] = fma2(n[i][k], less_m, g[i][k] + less_a);
            if (p.dres) {
                Pair q[4];
                pairs8<B16>(row + gb + hb + c[i] * he, p.h_dt, q);
#pragma unroll
                for (uint32_t k = 0; k < 4; ++k) o[k] = fma2(o[k], by, q[k]);
            } else {
#pragma unroll
                for (uint32_t k = 0; k < 4; ++k) o[k] = o[k] * by;
            }
            float f[8];
            singles8(o, f);
            store8<true>(p.dx + r * p.dx_pitch, B16 ? (uint32_t)DTT_BF16 : p.h_dt, c[i], p.cols, f);
        }
        if (++st == S) { st = 0; phase ^= 1; }
    }
    if (lost && t == 0) await_copies(full, S, next, p.partials);
    if (!p.partial) return;
#pragma unroll
    for (uint32_t i = 0; i < NCH; ++i) {
        if (!in[i]) continue;
        float f[8], e[8];
        singles8(acc[i], f);
        singles8(acc_b[i], e);
        if (lost) {                                 // they have taken rows that had not arrived
            make_nan(f);
            make_nan(e);
        }
        store8<true>(reinterpret_cast<char*>(p.partial + (uint64_t)blockIdx.x * p.cols), DTT_F32, c[i], p.cols, f);
        store8<true>(reinterpret_cast<char*>(p.partial_b + (uint64_t)blockIdx.x * p.cols), DTT_F32, c[i], p.cols, e);
    }
}

// ---- ring of unaligned rows --------------------------------------------------------------------
// The ring for rows at any alignment, an element a thread.  A bulk copy moves whole 16-byte
// words: from the one that holds the row's first byte to the one that holds its last.  The few bytes
// beside the row in these two are copied with it and not looked at (an allocation never ends within
// such a word).  4093 x 5001 (bf16 with an f32 residual): 41.6 us, 0.87 of the copy rate; the layer norm, with its second reduction, 51,
// 0.71.
struct Words {
    uint64_t from;              // address of the first
    uint32_t bytes;             // of all
};

__device__ __forceinline__ Words words_of(const char* row, uint32_t bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(row), first = a & ~15ull;
    return {first, ((uint32_t)(a - first) + bytes + 15) & ~15u};
}

// Where a row begins in its first word.
__device__ __forceinline__ uint32_t skip_of(const char* base, uint64_t r, uint64_t pitch) {
    return ((uint32_t)reinterpret_cast<uint64_t>(base) + (uint32_t)r * (uint32_t)pitch) & 15u;
}

__host__ __device__ __forceinline__ uint32_t words_room(uint32_t bytes) { return (bytes + 30) & ~15u; }

template <bool MEAN, uint32_t E>
__global__ void __launch_bounds__(kRingThreads, 2) norm_fwd_ring_elements_kernel(const __grid_constant__ FwdParams p, uint32_t S) {
    launch_next();
    extern __shared__ __align__(128) uint8_t stages[];
    __shared__ float slots[2][MEAN ? 3 : 2][32];
    __shared__ uint64_t full[ring::kStages];
    const uint32_t T = blockDim.x, t = threadIdx.x;
    const uint32_t xb = p.cols * (p.x_dt == DTT_BF16 ? 2 : 4), rb = p.res ? p.cols * (p.res_dt == DTT_BF16 ? 2 : 4) : 0;
    const uint32_t x_room = words_room(xb), stage_bytes = x_room + (rb ? words_room(rb) : 0);
    uint64_t next = blockIdx.x;                     // thread 0: the row to be fetched next, and its stage
    uint32_t next_st = 0;
    auto start = [&] {
        if (next >= p.rows) return;
        const uint64_t r = next;
        const uint32_t bar = saddr(full + next_st), dst = saddr(stages) + next_st * stage_bytes;
        next += gridDim.x;
        if (++next_st == S) next_st = 0;
        const Words x = words_of(p.x + r * p.x_pitch, xb);
        Words res{0, 0};
        if (rb) res = words_of(p.res + r * p.res_pitch, rb);
        bar_expect_tx(bar, x.bytes + res.bytes);
        bulk_load(dst, reinterpret_cast<const char*>(x.from), x.bytes, bar);
        if (rb) bulk_load(dst + x_room, reinterpret_cast<const char*>(res.from), res.bytes, bar);
    };
    if (t == 0) {
        for (uint32_t i = 0; i < S; ++i) bar_init(saddr(full + i), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    wait_previous();
    if (t == 0)
        for (uint32_t i = 0; i + 1 < S; ++i) start();
    float w[E], b[MEAN ? E : 1];
#pragma unroll
    for (uint32_t k = 0; k < E; ++k) {
        w[k] = 1.0f;
        if (MEAN) b[k] = 0.0f;
    }
    if (p.w) load_elements(p.w, p.w_dt, p.cols, w);
    if constexpr (MEAN)
        if (p.b) load_elements(p.b, p.w_dt, p.cols, b);
    __syncthreads();

    uint32_t st = 0, phase = 0;
    uint32_t turn = 0;
    bool lost = false;
    for (uint64_t r = blockIdx.x; r < p.rows; r += gridDim.x, turn ^= 1) {
        lost = lost || DTT_NORM_ROW_LATE || !bar_wait(saddr(full + st), phase);
        const char* row = reinterpret_cast<const char*>(stages) + st * stage_bytes;
        float h[E], sum = 0.0f;
        load_elements(row + skip_of(p.x, r, p.x_pitch), p.x_dt, p.cols, h);
        if (rb) {
            float q[E];
            load_elements(row + x_room + skip_of(p.res, r, p.res_pitch), p.res_dt, p.cols, q);
#pragma unroll
            for (uint32_t k = 0; k < E; ++k) h[k] += q[k];
        }
        float mu = 0.0f;
        if constexpr (MEAN) {
#pragma unroll
            for (uint32_t k = 0; k < E; ++k) mu += h[k];
            if (lost) mu = kNan;
            mu = row_sum(mu, T, slots[turn][2]) * p.inv_cols;
            if (t == 0 && p.mean) p.mean[r] = mu;
            centre(h, mu, p.cols);
        }
#pragma unroll
        for (uint32_t k = 0; k < E; ++k) sum += MEAN ? (h[k] - mu) * (h[k] - mu) : h[k] * h[k];
        if (lost) sum = kNan;
        const float s = rsqrtf(row_sum(sum, T, slots[turn][0]) * p.inv_cols + p.eps);
        if (t == 0) {
            if (!lost) start();
            if (p.rstd) p.rstd[r] = s;
        }
        if (p.res_out) {
            if (lost) make_nan(h);
            store_elements(p.res_out + r * p.res_out_pitch, p.res_dt, p.cols, h);
        }
#pragma unroll
        for (uint32_t k = 0; k < E; ++k) {
            if (MEAN) h[k] -= mu;
            h[k] = h[k] * s * w[k];
            if (MEAN) h[k] += b[k];
        }
        if (p.y_dt == DTT_E4M3) scale_elements(p, r, slots[turn][1], h);
        store_elements(p.y + r * p.y_pitch, p.y_dt, p.cols, h);
        if (++st == S) { st = 0; phase ^= 1; }
    }
    if (lost && t == 0) await_copies(full, S, next, gridDim.x);
}

// 16384 x 4001 in f32: 179 us, 0.86 of the copy rate (layer norm 171, 0.90); 1021 x 5001 in f32 19 us, 0.63 (layer norm 22, 0.54): one CTA a SM
// (60 KiB a stage), seven rows each.
template <bool MEAN, uint32_t E>
__global__ void __launch_bounds__(MEAN && E == 8 ? kWideThreads : kRingThreads) norm_bwd_ring_elements_kernel(const __grid_constant__ BwdParams p, uint32_t S) {
    launch_next();
    if (blockIdx.x >= p.partials) return weight_columns<MEAN>(p);
    extern __shared__ __align__(128) uint8_t stages[];
    __shared__ float slots[2][MEAN ? 64 : 32];
    __shared__ uint64_t full[ring::kStages];
    const uint32_t T = blockDim.x, t = threadIdx.x;
    const uint32_t gb = p.cols * (p.dy_dt == DTT_BF16 ? 2 : 4), hb = p.cols * (p.h_dt == DTT_BF16 ? 2 : 4);
    const uint32_t g_room = words_room(gb), h_room = words_room(hb), stage_bytes = g_room + (p.dres ? 2 : 1) * h_room;
    uint64_t next = blockIdx.x;                     // thread 0: the row to be fetched next, and its stage
    uint32_t next_st = 0;
    auto start = [&] {
        if (next >= p.rows) return;
        const uint64_t r = next;
        const uint32_t bar = saddr(full + next_st), dst = saddr(stages) + next_st * stage_bytes;
        next += p.partials;
        if (++next_st == S) next_st = 0;
        const Words g = words_of(p.dy + r * p.dy_pitch, gb), h = words_of(p.h + r * p.h_pitch, hb);
        Words d{0, 0};
        if (p.dres) d = words_of(p.dres + r * p.dres_pitch, hb);
        bar_expect_tx(bar, g.bytes + h.bytes + d.bytes);
        bulk_load(dst, reinterpret_cast<const char*>(g.from), g.bytes, bar);
        bulk_load(dst + g_room, reinterpret_cast<const char*>(h.from), h.bytes, bar);
        if (p.dres) bulk_load(dst + g_room + h_room, reinterpret_cast<const char*>(d.from), d.bytes, bar);
    };
    if (t == 0) {
        for (uint32_t i = 0; i < S; ++i) bar_init(saddr(full + i), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    wait_previous();
    if (t == 0)
        for (uint32_t i = 0; i + 1 < S; ++i) start();
    float w[E], acc[E], acc_b[MEAN ? E : 1];
#pragma unroll
    for (uint32_t k = 0; k < E; ++k) {
        w[k] = 1.0f;
        acc[k] = 0.0f;
        if (MEAN) acc_b[k] = 0.0f;
    }
    if (p.w) load_elements(p.w, p.w_dt, p.cols, w);
    __syncthreads();

    uint32_t st = 0, phase = 0;
    uint32_t turn = 0;
    bool lost = false;
    for (uint64_t r = blockIdx.x; r < p.rows; r += p.partials, turn ^= 1) {
        const float s = p.rstd[r], mu = MEAN ? p.mean[r] : 0.0f;
        lost = lost || DTT_NORM_ROW_LATE || !bar_wait(saddr(full + st), phase);
        const char* row = reinterpret_cast<const char*>(stages) + st * stage_bytes;
        float g[E], n[E], dot = 0.0f, all = 0.0f;
        load_elements(row + skip_of(p.dy, r, p.dy_pitch), p.dy_dt, p.cols, g);
        load_elements(row + g_room + skip_of(p.h, r, p.h_pitch), p.h_dt, p.cols, n);
#pragma unroll
        for (uint32_t k = 0; k < E; ++k) {
            n[k] = (MEAN ? n[k] - mu : n[k]) * s;
            acc[k] += g[k] * n[k];
            if (MEAN) acc_b[k] += g[k];
            g[k] *= w[k];
            dot += g[k] * n[k];
            if (MEAN) all += g[k];
        }
        if (lost) dot = kNan;
        const float2 means = row_means<MEAN>(dot, all, T, slots[turn], p.inv_cols);
        if (t == 0 && !lost) start();
#pragma unroll
        for (uint32_t k = 0; k < E; ++k) g[k] = s * ((MEAN ? g[k] - means.y : g[k]) - n[k] * means.x);
        if (p.dres) {
            load_elements(row + g_room + h_room + skip_of(p.dres, r, p.dres_pitch), p.h_dt, p.cols, n);
#pragma unroll
            for (uint32_t k = 0; k < E; ++k) g[k] += n[k];
        }
        store_elements(p.dx + r * p.dx_pitch, p.h_dt, p.cols, g);
        if (++st == S) { st = 0; phase ^= 1; }
    }
    if (lost) {                                     // acc has taken rows that had not arrived
        if (t == 0) await_copies(full, S, next, p.partials);
        make_nan(acc);
        if (MEAN) make_nan(acc_b);
    }
    if (p.partial) store_elements(reinterpret_cast<char*>(p.partial + (uint64_t)blockIdx.x * p.cols), DTT_F32, p.cols, acc);
    if constexpr (MEAN)
        if (p.partial) store_elements(reinterpret_cast<char*>(p.partial_b + (uint64_t)blockIdx.x * p.cols), DTT_F32, p.cols, acc_b);
}

// dweight[c] = the partial rows' sum.  32 columns a CTA; its 32 warps take every 32nd partial row, and
// their sums are added in warp order.  304 partial rows of 4096: about 4 us, from L2.
// blockIdx.y 1: the bias's partial rows and gradient.
__global__ void __launch_bounds__(1024) norm_dweight_kernel(const float* partial_w, const float* partial_b, uint32_t partials, uint32_t cols, float* dweight, float* dbias) {
    const float* partial = blockIdx.y ? partial_b : partial_w;
    float* out = blockIdx.y ? dbias : dweight;
    if (!out) return;
    __shared__ float part[32][33];
    const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const uint64_t c = (uint64_t)blockIdx.x * 32 + lane;
    float v = 0.0f;
    wait_previous();
    if (c < cols) {
#pragma unroll 10
        for (uint32_t i = warp; i < partials; i += 32) v += partial[(uint64_t)i * cols + c];
    }
    part[warp][lane] = v;
    __syncthreads();
    v = part[lane][warp];                            // warp w adds column w
#pragma unroll
    for (uint32_t o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (lane == 0 && (uint64_t)blockIdx.x * 32 + warp < cols) out[(uint64_t)blockIdx.x * 32 + warp] = v;
}

uint32_t short_lanes(uint32_t cols) {
    uint32_t n = 1;
    while (8 * n < cols) n *= 2;
    return n;
}

uint32_t sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 1;
    return (uint32_t)std::max(sms, 1);
}

// Threads of the element form: E elements each, `threads` at most; 0: the row is longer.
uint32_t element_threads(uint32_t cols, uint32_t E, uint32_t threads) {
    const uint32_t t = ((cols + E - 1) / E + 31) / 32 * 32;
    return t <= threads ? t : 0;
}

using RingKernel = void (*)(FwdParams, uint32_t);
RingKernel layernorm_ring(uint32_t nch, bool b16) {
    if (b16) return nch == 1 ? layernorm_fwd_ring_kernel<1, true> : nch == 2 ? layernorm_fwd_ring_kernel<2, true> : layernorm_fwd_ring_kernel<4, true>;
    return nch == 1 ? layernorm_fwd_ring_kernel<1, false> : nch == 2 ? layernorm_fwd_ring_kernel<2, false> : layernorm_fwd_ring_kernel<4, false>;
}

using BackwardRingKernel = void (*)(BwdParams, uint32_t);
BackwardRingKernel layernorm_bwd_ring(uint32_t nch, bool b16) {
    if (b16) return nch == 1 ? layernorm_bwd_ring_kernel<1, true> : nch == 2 ? layernorm_bwd_ring_kernel<2, true> : layernorm_bwd_ring_kernel<4, true>;
    return nch == 1 ? layernorm_bwd_ring_kernel<1, false> : nch == 2 ? layernorm_bwd_ring_kernel<2, false> : layernorm_bwd_ring_kernel<4, false>;
}

template <bool MEAN>
cudaError_t launch_fwd(const FwdParams& p, bool vec, cudaStream_t stream) {
    const uint32_t xe = p.x_dt == DTT_BF16 ? 2 : 4, re = p.res ? (p.res_dt == DTT_BF16 ? 2 : 4) : 0;
    const uint32_t sms = sm_count();
    const uint64_t xb = (uint64_t)p.cols * xe, rb = (uint64_t)p.cols * re;
    if (vec && p.cols <= kShortCols) {
        const uint32_t lanes = short_lanes(p.cols);
        const uint64_t each = 256 / lanes;
        return launch(norm_fwd_short_kernel<MEAN>, (uint32_t)((p.rows + each - 1) / each), 256, 0, 0, true, stream, p, lanes);
    }
    // two stages where a CTA has many rows: reads that run further ahead of the writes cost more than they
    // hide (40000 x 2048 to 8 bits: 104 us with three, 90 with two; 2048 x 4096, three rows a CTA: 14.7 and
    // 16.5; the backward pass, 30000 x 1024: 63 with eight, 76 with two)
    const ring::Plan g = MEAN && vec ? ring::plan(p.cols, vec, xb + rb, kFwdOwn<MEAN>, 1024, {1024, 768, 512}, 2, p.rows >= 32 * sms ? 2 : ring::kStages, 16 * kLayerThreads)
                                     : ring::plan(p.cols, vec, vec ? xb + rb : xb + rb + 60, kFwdOwn<MEAN>, vec ? 1024 : 2048, {vec ? 1536u : 1024u, 1024, 512}, 2, p.rows >= 32 * sms ? 2 : ring::kStages);
    // The chunk form's loads wait for one another, the ring's do not: 152 x 8064 (bf16) 6.7 us by chunks, 3.7 by
    // the ring.  The element form's go out together, and it is the faster one while there are few rows:
    // 600 x 3001 5.7 us and 6.6, 2400 x 3001 22.2 and 18.4.
    if (g.ctas && (vec || p.rows >= 8 * sms)) {
        const uint32_t grid = (uint32_t)std::min<uint64_t>(p.rows, g.ctas * sms);
        if (!vec) return launch(g.nch == 1 ? norm_fwd_ring_elements_kernel<MEAN, 8> : norm_fwd_ring_elements_kernel<MEAN, 16>, grid, g.threads, g.smem, 0, true, stream, p, g.stages);
        if constexpr (MEAN) {
            const bool b16 = p.x_dt == DTT_BF16 && (!p.res || p.res_dt == DTT_BF16) && (!p.res_out || p.res_dt == DTT_BF16) && ((!p.w && !p.b) || p.w_dt == DTT_BF16);
            return launch(layernorm_ring(g.nch, b16), grid, g.threads, g.smem, 0, true, stream, p, g.stages);
        }
        auto kernel = g.nch == 1 ? rmsnorm_fwd_ring_kernel<1> : g.nch == 2 ? rmsnorm_fwd_ring_kernel<2> : rmsnorm_fwd_ring_kernel<4>;
        return launch(kernel, grid, g.threads, g.smem, 0, true, stream, p, g.stages);
    }
    if (!vec) {
        if (const uint32_t t = element_threads(p.cols, 8, kFwdThreads)) {
            const uint32_t each = t == 32 ? kWarpRows : 1;
            return launch(norm_fwd_elements_kernel<MEAN, 8>, (uint32_t)((p.rows + each - 1) / each), dim3(t, each), 0, 0, true, stream, p);
        }
        if (const uint32_t t = element_threads(p.cols, 16, kFwdThreads))
            return launch(norm_fwd_elements_kernel<MEAN, 16>, (uint32_t)p.rows, t, 0, 0, true, stream, p);
        return launch(norm_fwd_kernel<MEAN, kLong, false>, (uint32_t)p.rows, kFwdThreads, 0, 0, true, stream, p);
    }
    if (p.cols <= 32 * kFwdThreads) return launch(norm_fwd_kernel<MEAN, 4, true>, (uint32_t)p.rows, kFwdThreads, 0, 0, true, stream, p);
    return launch(norm_fwd_kernel<MEAN, kLong, true>, (uint32_t)p.rows, kFwdThreads, 0, 0, true, stream, p);
}

// Sets p.partials, the CTAs that take rows, and as many partial rows of the weight's gradient.
template <bool MEAN>
cudaError_t launch_bwd(BwdParams& p, bool vec, cudaStream_t stream) {
    const uint32_t columns = p.dweight || p.dbias ? (uint32_t)std::min<uint64_t>((p.cols + 31) / 32, 4 * sm_count()) : 0;
    const uint32_t ge = p.dy_dt == DTT_BF16 ? 2 : 4, he = p.h_dt == DTT_BF16 ? 2 : 4;
    const uint32_t sms = sm_count();
    if (vec && p.cols <= kShortCols) {
        const uint32_t lanes = short_lanes(p.cols);
        const uint64_t each = 256 / lanes;
        p.partials = (uint32_t)std::min<uint64_t>((p.rows + each - 1) / each, most_partials(p.cols));
        return launch(norm_bwd_short_kernel<MEAN>, p.partials + columns, 256, 0, 0, true, stream, p, lanes);
    }
    const uint64_t stage = (uint64_t)p.cols * (ge + (p.dres ? 2 : 1) * he);
    ring::Plan g = ring::plan(p.cols, vec, vec ? stage : stage + 90, kBwdOwn<MEAN>, 2048, {1024, 512, 256}, 1, ring::kStages);
    // where an SM has room for one CTA the layer norm gives it more threads: 1021 x 5001 (f32) 23 us with 16 elements a
    // thread, 22 with 8
    if (MEAN && !vec && g.ctas == 1 && g.nch == 2 && p.cols <= 8 * kWideThreads && p.rows > kFewRows) {
        g.nch = 1;
        g.threads = (p.cols + 255) / 256 * 32;
    }
    // by chunks and by the ring: 200 x 4096 (bf16) 11.2 us and 7.6, 16384 x 4096 255 and 92; by elements and by
    // the ring: 152 x 1021 (f32) 5.5 and 5.6, 460 x 5001 (f32) 15.3 and 10.8
    if (g.ctas && (vec || p.rows > sms)) {
        p.partials = (uint32_t)std::min<uint64_t>({p.rows, (uint64_t)g.ctas * sms, (uint64_t)most_partials(p.cols)});
        if (MEAN && vec) {
            const bool b16 = p.dy_dt == DTT_BF16 && p.h_dt == DTT_BF16 && (!p.w || p.w_dt == DTT_BF16);
            return launch(layernorm_bwd_ring(g.nch, b16), p.partials + columns, g.threads, g.smem, 0, true, stream, p, g.stages);
        }
        auto kernel = vec ? (g.nch == 1 ? rmsnorm_bwd_ring_kernel<1> : g.nch == 2 ? rmsnorm_bwd_ring_kernel<2> : rmsnorm_bwd_ring_kernel<4>)
                          : (g.nch == 1 ? norm_bwd_ring_elements_kernel<MEAN, 8> : norm_bwd_ring_elements_kernel<MEAN, 16>);
        return launch(kernel, p.partials + columns, g.threads, g.smem, 0, true, stream, p, g.stages);
    }
    auto walk = [&](uint32_t each) {       // walkers a CTA
        p.partials = (uint32_t)std::min<uint64_t>((p.rows + each - 1) / each, most_partials(p.cols));
        p.walkers = p.partials * each;
    };
    walk(1);
    if (!vec) {
        if (const uint32_t t = element_threads(p.cols, 8, kBwdThreads)) {
            const uint32_t each = t == 32 ? kWarpRows : 1;
            walk(each);
            return launch(norm_bwd_elements_kernel<MEAN, 8>, p.partials + columns, dim3(t, each), 0, 0, true, stream, p);
        }
        if (const uint32_t t = element_threads(p.cols, 16, kBwdThreads))
            return launch(norm_bwd_elements_kernel<MEAN, 16>, p.partials + columns, t, 0, 0, true, stream, p);
        return launch(norm_bwd_kernel<MEAN, kLong, false>, p.partials + columns, kBwdThreads, 0, 0, true, stream, p);
    }
    if (p.cols <= 32 * kBwdThreads) return launch(norm_bwd_kernel<MEAN, 4, true>, p.partials + columns, kBwdThreads, 0, 0, true, stream, p);
    return launch(norm_bwd_kernel<MEAN, kLong, true>, p.partials + columns, kBwdThreads, 0, 0, true, stream, p);
}

uint32_t elem_bytes(uint32_t dt) { return dt == DTT_BF16 ? 2 : dt == DTT_F32 ? 4 : 1; }

int check_desc(const char* who, const dtt_rmsnorm_desc* d) {
    if (!d) return fail(DTT_EINVAL, "%s: null desc", who);
    for (uint32_t t : {d->x_dtype, d->residual_dtype, d->weight_dtype})
        if (t != DTT_BF16 && t != DTT_F32) return fail(DTT_EINVAL, "%s: x, residual and weight are bf16 or f32", who);
    if (d->y_dtype != DTT_BF16 && d->y_dtype != DTT_F32 && d->y_dtype != DTT_E4M3)
        return fail(DTT_EINVAL, "%s: y is bf16, f32 or e4m3", who);
    if (d->y_dtype == DTT_E4M3 ? (d->group != 0 && d->group != 32 && d->group != 64 && d->group != 128) : d->group != 0)
        return fail(DTT_EINVAL, "%s: group is 0, 32, 64 or 128 with an e4m3 y, else 0", who);
    if (!(d->eps >= 0.0f) || !std::isfinite(d->eps)) return fail(DTT_EINVAL, "%s: eps must be finite and not negative", who);
    if (d->cols == 0 || d->cols > (1u << 24)) return fail(DTT_EINVAL, "%s: cols must be 1 .. 2^24", who);
    return DTT_OK;
}

// A tensor argument: present unless optional, aligned to its element, rows that do not overlap.
int check_rows(const char* who, const char* name, const void* ptr, uint64_t pitch, uint64_t rows, uint64_t cols,
               uint32_t dt, bool optional) {
    if (!ptr) return optional ? DTT_OK : fail(DTT_EINVAL, "%s: %s is missing", who, name);
    const uint32_t e = elem_bytes(dt);
    if (reinterpret_cast<uintptr_t>(ptr) % e || pitch % e)
        return fail(DTT_EINVAL, "%s: %s must be aligned to its %u-byte elements", who, name, e);
    if (rows > 1 && pitch < cols * e) return fail(DTT_EINVAL, "%s: %s: the pitch is less than a row", who, name);
    return DTT_OK;
}

bool aligned(const void* ptr, uint64_t pitch, uint32_t to) {
    return reinterpret_cast<uintptr_t>(ptr) % to == 0 && pitch % to == 0;      // null: aligned
}

// own: what the launches take a kernel's shared memory beside the stages to be, at most.
cudaError_t prepare(const void* kernel, uint32_t own = ~0u) {
    cudaFuncAttributes a;
    cudaError_t e = cudaFuncGetAttributes(&a, kernel);
    if (e == cudaSuccess && a.sharedSizeBytes > own) return cudaErrorInvalidConfiguration;
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, kCarveout);
    return e;
}

}  // namespace

namespace {

template <bool MEAN>
cudaError_t preload_norm() {
    const void* kernels[] = {
        (const void*)norm_fwd_short_kernel<MEAN>, (const void*)norm_bwd_short_kernel<MEAN>,
        (const void*)norm_fwd_kernel<MEAN, 4, true>, (const void*)norm_fwd_kernel<MEAN, kLong, true>,
        (const void*)norm_fwd_kernel<MEAN, kLong, false>, (const void*)norm_fwd_elements_kernel<MEAN, 8>,
        (const void*)norm_fwd_elements_kernel<MEAN, 16>,
        (const void*)norm_bwd_kernel<MEAN, 4, true>, (const void*)norm_bwd_kernel<MEAN, kLong, true>,
        (const void*)norm_bwd_kernel<MEAN, kLong, false>, (const void*)norm_bwd_elements_kernel<MEAN, 8>,
        (const void*)norm_bwd_elements_kernel<MEAN, 16>, (const void*)norm_dweight_kernel};
    for (const void* k : kernels) {
        const cudaError_t e = prepare(k);
        if (e != cudaSuccess) return e;
    }
    const void* fwd_rings[] = {(const void*)(MEAN ? layernorm_ring(1, true) : rmsnorm_fwd_ring_kernel<1>), (const void*)(MEAN ? layernorm_ring(2, true) : rmsnorm_fwd_ring_kernel<2>),
                               (const void*)(MEAN ? layernorm_ring(4, true) : rmsnorm_fwd_ring_kernel<4>), (const void*)norm_fwd_ring_elements_kernel<MEAN, 8>,
                               (const void*)norm_fwd_ring_elements_kernel<MEAN, 16>, (const void*)layernorm_ring(1, false), (const void*)layernorm_ring(2, false),
                               (const void*)layernorm_ring(4, false)};
    const void* bwd_rings[] = {(const void*)(MEAN ? layernorm_bwd_ring(1, true) : rmsnorm_bwd_ring_kernel<1>), (const void*)(MEAN ? layernorm_bwd_ring(2, true) : rmsnorm_bwd_ring_kernel<2>),
                               (const void*)(MEAN ? layernorm_bwd_ring(4, true) : rmsnorm_bwd_ring_kernel<4>), (const void*)norm_bwd_ring_elements_kernel<MEAN, 8>,
                               (const void*)norm_bwd_ring_elements_kernel<MEAN, 16>, (const void*)layernorm_bwd_ring(1, false), (const void*)layernorm_bwd_ring(2, false),
                               (const void*)layernorm_bwd_ring(4, false)};
    auto ring = [](const void* k, uint32_t own) {
        const cudaError_t e = prepare(k, own);
        return e == cudaSuccess ? cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ring::kSmem) : e;
    };
    for (uint32_t i = 0; i < (MEAN ? 8 : 5); ++i) {
        cudaError_t e = ring(fwd_rings[i], kFwdOwn<MEAN>);
        if (e == cudaSuccess) e = ring(bwd_rings[i], kBwdOwn<MEAN>);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t preload_norm_kernels() {
    const cudaError_t e = preload_norm<false>();
    return e == cudaSuccess ? preload_norm<true>() : e;
}

}  // namespace dtt

using namespace dtt;

extern "C" int dtt_rmsnorm_workspace(const dtt_rmsnorm_desc* d, uint64_t* bytes) {
    const int rc = check_desc("dtt_rmsnorm_workspace", d);
    if (rc) return rc;
    if (!bytes) return fail(DTT_EINVAL, "dtt_rmsnorm_workspace: null bytes");
    *bytes = (uint64_t)most_partials(d->cols) * d->cols * 4;
    return DTT_OK;
}

extern "C" int dtt_layernorm_workspace(const dtt_layernorm_desc* d, uint64_t* bytes) {
    const int rc = check_desc("dtt_layernorm_workspace", d);
    if (rc) return rc;
    if (!bytes) return fail(DTT_EINVAL, "dtt_layernorm_workspace: null bytes");
    *bytes = 2 * (uint64_t)most_partials(d->cols) * d->cols * 4;
    return DTT_OK;
}

namespace {

// bias and mean: the layer norm's.
template <bool MEAN>
int forward(const char* who, const dtt_rmsnorm_desc* d, uint64_t rows, const void* x, uint64_t x_pitch, const void* residual,
            uint64_t residual_pitch, const void* weight, const void* bias, void* residual_out, uint64_t residual_out_pitch, void* y,
            uint64_t y_pitch, float* scales, float* mean, float* rstd, cudaStream_t stream) {
    int rc = check_desc(who, d);
    if (rc) return rc;
    if (rows >= (1ull << 31)) return fail(DTT_EINVAL, "%s: 2^31 rows or more", who);
    if (rows == 0) return DTT_OK;
    const bool e4m3 = d->y_dtype == DTT_E4M3;
    if ((rc = check_rows(who, "x", x, x_pitch, rows, d->cols, d->x_dtype, false)) ||
        (rc = check_rows(who, "residual", residual, residual_pitch, rows, d->cols, d->residual_dtype, true)) ||
        (rc = check_rows(who, "weight", weight, 0, 1, d->cols, d->weight_dtype, true)) ||
        (rc = check_rows(who, "bias", bias, 0, 1, d->cols, d->weight_dtype, true)) ||
        (rc = check_rows(who, "residual_out", residual_out, residual_out_pitch, rows, d->cols, d->residual_dtype, true)) ||
        (rc = check_rows(who, "y", y, y_pitch, rows, d->cols, d->y_dtype, false)) ||
        (rc = check_rows(who, "scales", scales, 0, 1, 0, DTT_F32, !e4m3)) ||
        (rc = check_rows(who, "mean", mean, 0, 1, 0, DTT_F32, true)) ||
        (rc = check_rows(who, "rstd", rstd, 0, 1, 0, DTT_F32, true)))
        return rc;
    if (scales && !e4m3) return fail(DTT_EINVAL, "%s: scales go with an e4m3 y alone", who);
    if (residual && residual == residual_out && residual_pitch != residual_out_pitch)
        return fail(DTT_EINVAL, "%s: in place, residual and residual_out have one pitch", who);
    if ((rc = preload_once())) return rc;
    FwdParams p{};
    p.x = static_cast<const char*>(x);
    p.res = static_cast<const char*>(residual);
    p.w = static_cast<const char*>(weight);
    p.b = static_cast<const char*>(bias);
    p.res_out = static_cast<char*>(residual_out);
    p.y = static_cast<char*>(y);
    p.scales = scales;
    p.mean = mean;
    p.rstd = rstd;
    p.x_pitch = x_pitch;
    p.res_pitch = residual_pitch;
    p.res_out_pitch = residual_out_pitch;
    p.y_pitch = y_pitch;
    p.rows = rows;
    p.cols = (uint32_t)d->cols;
    p.groups = d->group ? (uint32_t)((d->cols + d->group - 1) / d->group) : 1;
    p.x_dt = d->x_dtype;
    p.res_dt = d->residual_dtype;
    p.w_dt = d->weight_dtype;
    p.y_dt = d->y_dtype;
    p.group_lanes = d->group / 8;
    p.eps = d->eps;
    p.inv_cols = 1.0f / (float)d->cols;
    const bool vec = d->cols % 8 == 0 && aligned(x, x_pitch, 16) && aligned(residual, residual ? residual_pitch : 0, 16) &&
                     aligned(weight, 0, 16) && aligned(bias, 0, 16) && aligned(residual_out, residual_out ? residual_out_pitch : 0, 16) &&
                     aligned(y, y_pitch, e4m3 ? 8 : 16);
    const cudaError_t e = launch_fwd<MEAN>(p, vec, stream);
    if (e != cudaSuccess) return fail(DTT_ECUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    return DTT_OK;
}

// mean and dbias: the layer norm's.
template <bool MEAN>
int backward(const char* who, const dtt_rmsnorm_desc* d, uint64_t rows, const void* dy, uint64_t dy_pitch, const void* h, uint64_t h_pitch,
             const void* weight, const float* mean, const float* rstd, const void* dres, uint64_t dres_pitch, void* dx, uint64_t dx_pitch,
             float* dweight, float* dbias, void* workspace, uint64_t workspace_bytes, cudaStream_t stream) {
    const uint64_t part_bytes = d ? (uint64_t)most_partials(d->cols) * d->cols * 4 : 0;
    int rc = check_desc(who, d);
    if (rc) return rc;
    if (rows >= (1ull << 31)) return fail(DTT_EINVAL, "%s: 2^31 rows or more", who);
    if (dweight && !weight) return fail(DTT_EINVAL, "%s: a weight's gradient without a weight", who);
    if ((rc = check_rows(who, "weight", weight, 0, 1, d->cols, d->weight_dtype, true)) ||
        (rc = check_rows(who, "dweight", dweight, 0, 1, 0, DTT_F32, true)) ||
        (rc = check_rows(who, "dbias", dbias, 0, 1, 0, DTT_F32, true)))
        return rc;
    if ((dweight || dbias) && (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16 || workspace_bytes < (MEAN ? 2 : 1) * part_bytes))
        return fail(DTT_EINVAL, "%s: the workspace is missing, misaligned or short", who);
    if (rows == 0) {
        for (float* out : {dweight, dbias})
            if (out) DTT_CUDA_TRY(cudaMemsetAsync(out, 0, d->cols * 4, stream));
        return DTT_OK;
    }
    if ((rc = check_rows(who, "dy", dy, dy_pitch, rows, d->cols, d->x_dtype, false)) ||
        (rc = check_rows(who, "h", h, h_pitch, rows, d->cols, d->residual_dtype, false)) ||
        (rc = check_rows(who, "mean", mean, 0, 1, 0, DTT_F32, !MEAN)) ||
        (rc = check_rows(who, "rstd", rstd, 0, 1, 0, DTT_F32, false)) ||
        (rc = check_rows(who, "dres", dres, dres_pitch, rows, d->cols, d->residual_dtype, true)) ||
        (rc = check_rows(who, "dx", dx, dx_pitch, rows, d->cols, d->residual_dtype, false)))
        return rc;
    if (dres && dres == dx && dres_pitch != dx_pitch)
        return fail(DTT_EINVAL, "%s: in place, dres and dx have one pitch", who);
    if ((rc = preload_once())) return rc;
    BwdParams p{};
    p.dy = static_cast<const char*>(dy);
    p.h = static_cast<const char*>(h);
    p.w = static_cast<const char*>(weight);
    p.mean = mean;
    p.rstd = rstd;
    p.dres = static_cast<const char*>(dres);
    p.dx = static_cast<char*>(dx);
    const bool few = rows <= kFewRows;
    p.partial = (dweight || dbias) && !few ? static_cast<float*>(workspace) : nullptr;
    p.partial_b = MEAN && p.partial ? p.partial + part_bytes / 4 : nullptr;
    p.dweight = few ? dweight : nullptr;
    p.dbias = few ? dbias : nullptr;
    p.dy_pitch = dy_pitch;
    p.h_pitch = h_pitch;
    p.dres_pitch = dres_pitch;
    p.dx_pitch = dx_pitch;
    p.rows = rows;
    p.cols = (uint32_t)d->cols;
    p.dy_dt = d->x_dtype;
    p.h_dt = d->residual_dtype;
    p.w_dt = d->weight_dtype;
    p.inv_cols = 1.0f / (float)d->cols;
    const bool vec = d->cols % 8 == 0 && aligned(dy, dy_pitch, 16) && aligned(h, h_pitch, 16) && aligned(weight, 0, 16) &&
                     aligned(dres, dres ? dres_pitch : 0, 16) && aligned(dx, dx_pitch, 16);
    cudaError_t e = launch_bwd<MEAN>(p, vec, stream);
    if (e == cudaSuccess && p.partial)
        e = launch(norm_dweight_kernel, dim3((p.cols + 31) / 32, MEAN ? 2 : 1), 1024, 0, 0, true, stream, p.partial, p.partial_b, p.partials, p.cols, dweight, dbias);
    if (e != cudaSuccess) return fail(DTT_ECUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    return DTT_OK;
}

}  // namespace

extern "C" int dtt_rmsnorm_forward(const dtt_rmsnorm_desc* d, uint64_t rows, const void* x, uint64_t x_pitch,
                                   const void* residual, uint64_t residual_pitch, const void* weight,
                                   void* residual_out, uint64_t residual_out_pitch, void* y, uint64_t y_pitch,
                                   float* scales, float* rstd, cudaStream_t stream) {
    return forward<false>("dtt_rmsnorm_forward", d, rows, x, x_pitch, residual, residual_pitch, weight, nullptr, residual_out,
                          residual_out_pitch, y, y_pitch, scales, nullptr, rstd, stream);
}

extern "C" int dtt_layernorm_forward(const dtt_layernorm_desc* d, uint64_t rows, const void* x, uint64_t x_pitch,
                                     const void* residual, uint64_t residual_pitch, const void* weight, const void* bias,
                                     void* residual_out, uint64_t residual_out_pitch, void* y, uint64_t y_pitch,
                                     float* scales, float* mean, float* rstd, cudaStream_t stream) {
    return forward<true>("dtt_layernorm_forward", d, rows, x, x_pitch, residual, residual_pitch, weight, bias, residual_out,
                         residual_out_pitch, y, y_pitch, scales, mean, rstd, stream);
}

extern "C" int dtt_rmsnorm_backward(const dtt_rmsnorm_desc* d, uint64_t rows, const void* dy, uint64_t dy_pitch,
                                    const void* h, uint64_t h_pitch, const void* weight, const float* rstd,
                                    const void* dres, uint64_t dres_pitch, void* dx, uint64_t dx_pitch,
                                    float* dweight, void* workspace, uint64_t workspace_bytes, cudaStream_t stream) {
    return backward<false>("dtt_rmsnorm_backward", d, rows, dy, dy_pitch, h, h_pitch, weight, nullptr, rstd, dres, dres_pitch, dx,
                           dx_pitch, dweight, nullptr, workspace, workspace_bytes, stream);
}

extern "C" int dtt_layernorm_backward(const dtt_layernorm_desc* d, uint64_t rows, const void* dy, uint64_t dy_pitch,
                                      const void* h, uint64_t h_pitch, const void* weight, const float* mean, const float* rstd,
                                      const void* dres, uint64_t dres_pitch, void* dx, uint64_t dx_pitch, float* dweight,
                                      float* dbias, void* workspace, uint64_t workspace_bytes, cudaStream_t stream) {
    return backward<true>("dtt_layernorm_backward", d, rows, dy, dy_pitch, h, h_pitch, weight, mean, rstd, dres, dres_pitch, dx,
                          dx_pitch, dweight, dbias, workspace, workspace_bytes, stream);
}

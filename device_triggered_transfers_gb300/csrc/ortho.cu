// Orthogonalising an update by Newton-Schulz products (dtt_ops.h): X <- a X + (b A + c A A) X with
// A = X X^T, a few times over, for a batch of S x L matrices (S <= L: the smaller side first).
//
// Precision.  The tensor cores take f16 operands and add in f32.  X is held in f32 (x32) and only
// its operand copy (x16) is rounded: f16 has 11 significant bits where bf16 has 8, at the same
// rate, and every value here is below 3 in magnitude.  Rounding X itself would put noise of 2^-12 |X|
// into the singular directions that the update lacks, where a step multiplies it by a = 3.44: for a
// rank-1 update five steps in f16 end 10 % off, in bf16 75 %, with X in f32 0.2 % (the bf16 output).
// Rounded operands meet their noise only through b A + c A A, whose range holds nothing of it.
//
// A and b A + c A A are symmetric: only tiles on and below the diagonal are computed, and each is
// stored twice, once transposed.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>

#include <cuda_fp16.h>

#include "dtt_ops.h"
#include "internal.h"
#include "rowio.cuh"

namespace dtt {
namespace {

constexpr uint32_t TM = 128, TN = 128, BK = 64, UMMA_K = 16;
constexpr uint32_t TILE_STAGE = TM * BK * 2;         // 16 KiB an operand and stage
constexpr uint32_t STAGES = 6;
constexpr uint32_t ACC_BUFS = 2;
constexpr uint32_t TMEM_COLS = ACC_BUFS * TN;
constexpr uint32_t EPI_THREADS = 128;
constexpr uint32_t THREADS = EPI_THREADS + 64;       // + TMA warp + MMA warp
constexpr uint32_t TMA_WARP = 4, MMA_WARP = 5;
constexpr uint32_t WAIT_LIMIT = 1u << 22;
constexpr uint32_t SMEM_BYTES = 1024 /* alignment slack */ + STAGES * 2 * TILE_STAGE + 256;
// instruction descriptor (kind::f16): f32 accumulator, f16 operands, N = TN, M = TM
constexpr uint32_t IDESC = (1u << 4) | ((TN >> 3) << 17) | ((TM >> 4) << 24);
constexpr uint32_t IDESC_B_MN = 1u << 16;            // B stored with N contiguous

constexpr uint32_t kStartTile = 64;                  // ortho_start_tiles_kernel: elements a side
constexpr uint32_t kMaxParts = 1216;                 // ortho_update_kernel: CTAs a matrix at most, eight a SM

enum Product { GRAM, POLY, APPLY };

struct GemmParams {
    CUtensorMap tmA, tmB;
    uint32_t S, L, K;            // output rows S and columns (GRAM, POLY: S; APPLY: L)
    uint32_t batch, tiles_m, tiles_n, tiles;   // tiles: of one matrix
    uint64_t s_pitch, l_pitch;   // elements between rows of the S-wide and L-wide arrays
    float a, b, c;
    const __half* gram;          // POLY: A
    __half* out16;               // GRAM: A; POLY: b A + c A A; APPLY: the next x16
    float* x32;                  // APPLY
    // APPLY, last step: the result
    char* out;                   // or null: not the last step
    uint64_t out_pitch, out_stride;
    float scale;
    uint32_t transposed, out_vec;
    uint32_t* err;
};

__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Bounded wait for the phase of the given parity; false when the limit ran out or another role
// already reported an error.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile uint32_t* abort) {
    for (uint32_t i = 0; i < WAIT_LIMIT; ++i) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done) : "r"(bar), "r"(parity) : "memory");
        if (done) return true;
        if ((i & 255) == 255 && *abort) return false;
    }
    return false;
}

// AND of v over the epilogue's threads (named barrier 1), the same result in each.
__device__ __forceinline__ bool epi_all(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.and.pred q, 1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r) : "r"((uint32_t)v), "n"(EPI_THREADS) : "memory");
    return r != 0;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}

// Shared-memory matrix descriptors with the 128-byte swizzle.  K contiguous: rows of 64 k, groups of
// 8 rows 1024 bytes apart.  N contiguous: blocks of 64 n by 64 k (8 KiB, one box of the tensor map
// each), within one the groups of 8 k 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_of(uint32_t addr, uint32_t leading, uint32_t stride) {
    uint64_t d = 0;
    d |= (uint64_t)((addr & 0x3FFFFu) >> 4);          // start address
    d |= (uint64_t)(leading >> 4) << 16;              // leading byte offset
    d |= (uint64_t)(stride >> 4) << 32;               // stride byte offset
    d |= (uint64_t)1 << 46;                           // descriptor version
    d |= (uint64_t)2 << 61;                           // 128-byte swizzle
    return d;
}
__device__ __forceinline__ uint64_t desc_k(uint32_t addr) { return desc_of(addr, 16, 1024); }
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr) { return desc_of(addr, 64 * BK * 2, 1024); }

__device__ __forceinline__ void umma(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}

__device__ __forceinline__ void umma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 consecutive f32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
    uint32_t u[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
          "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
          "=r"(u[14]), "=r"(u[15]), "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]),
          "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]), "=r"(u[25]),
          "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (uint32_t k = 0; k < 32; ++k) v[k] = __uint_as_float(u[k]);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Tile t of a lower triangle counted row by row: (0,0), (1,0), (1,1), (2,0), ...
__device__ __forceinline__ void triangle(uint32_t t, uint32_t& i, uint32_t& j) {
    i = (uint32_t)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
    while (i * (i + 1) / 2 > t) --i;
    while ((i + 1) * (i + 2) / 2 <= t) ++i;
    j = t - i * (i + 1) / 2;
}

// The tile of place u: its matrix and its tile row and column.
template <Product P>
__device__ __forceinline__ void tile_of(const GemmParams& p, uint32_t u, uint32_t& m, uint32_t& i, uint32_t& j) {
    m = u / p.tiles;
    const uint32_t t = u % p.tiles;
    if (P == APPLY) {
        i = t % p.tiles_m;
        j = t / p.tiles_m;
    } else {
        triangle(t, i, j);
    }
}

// 32 columns from column c of output row r of matrix m, in the thread that holds them.
template <Product P>
__device__ __forceinline__ void finish(const GemmParams& p, uint32_t m, uint32_t r, uint32_t c, bool mirror, float (&v)[32]) {
    if (P == APPLY) {
        if (r >= p.S || c >= p.L) return;
        float4* x = reinterpret_cast<float4*>(p.x32 + ((uint64_t)m * p.S + r) * p.l_pitch + c);
#pragma unroll
        for (uint32_t q = 0; q < 8; ++q) {
            const float4 o = x[q];
            v[4 * q] += p.a * o.x;
            v[4 * q + 1] += p.a * o.y;
            v[4 * q + 2] += p.a * o.z;
            v[4 * q + 3] += p.a * o.w;
        }
        if (!p.out) {
#pragma unroll
            for (uint32_t q = 0; q < 8; ++q) x[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        } else {
            char* out = p.out + (uint64_t)m * p.out_stride;
#pragma unroll
            for (uint32_t k = 0; k < 32; ++k) v[k] *= p.scale;
            if (p.transposed) {
#pragma unroll
                for (uint32_t k = 0; k < 32; ++k)       // neighbouring lanes hold neighbouring columns of `out`
                    if (c + k < p.L)
                        *reinterpret_cast<uint16_t*>(out + (uint64_t)(c + k) * p.out_pitch + (uint64_t)r * 2) =
                            (uint16_t)pack_bf16(v[k], 0.0f);
            } else if (p.out_vec && c + 32 <= p.L) {
                uint4* o = reinterpret_cast<uint4*>(out + (uint64_t)r * p.out_pitch + (uint64_t)c * 2);
#pragma unroll
                for (uint32_t q = 0; q < 4; ++q)
                    o[q] = make_uint4(pack_bf16(v[8 * q], v[8 * q + 1]), pack_bf16(v[8 * q + 2], v[8 * q + 3]),
                                      pack_bf16(v[8 * q + 4], v[8 * q + 5]), pack_bf16(v[8 * q + 6], v[8 * q + 7]));
            } else {
#pragma unroll
                for (uint32_t k = 0; k < 32; ++k)
                    if (c + k < p.L)
                        *reinterpret_cast<uint16_t*>(out + (uint64_t)r * p.out_pitch + (uint64_t)(c + k) * 2) =
                            (uint16_t)pack_bf16(v[k], 0.0f);
            }
            return;
        }
    } else {
        if (r >= p.S || c >= p.S) return;
        if (P == POLY) {
            const uint4* g = reinterpret_cast<const uint4*>(p.gram + ((uint64_t)m * p.S + r) * p.s_pitch + c);
#pragma unroll
            for (uint32_t q = 0; q < 4; ++q) {
                const uint4 w = g[q];
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (uint32_t k = 0; k < 4; ++k) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[k]));
                    v[8 * q + 2 * k] = p.c * v[8 * q + 2 * k] + p.b * f.x;
                    v[8 * q + 2 * k + 1] = p.c * v[8 * q + 2 * k + 1] + p.b * f.y;
                }
            }
        }
    }
    const uint64_t pitch = P == APPLY ? p.l_pitch : p.s_pitch;
    uint4* o = reinterpret_cast<uint4*>(p.out16 + ((uint64_t)m * p.S + r) * pitch + c);
#pragma unroll
    for (uint32_t q = 0; q < 4; ++q)       // rows are padded to 64 elements: the whole chunk is the array's
        o[q] = make_uint4(pack_f16(v[8 * q], v[8 * q + 1]), pack_f16(v[8 * q + 2], v[8 * q + 3]),
                          pack_f16(v[8 * q + 4], v[8 * q + 5]), pack_f16(v[8 * q + 6], v[8 * q + 7]));
    if (P != APPLY && mirror) {
#pragma unroll
        for (uint32_t k = 0; k < 32; ++k)  // neighbouring lanes hold neighbouring columns of the mirrored rows
            if (c + k < p.S)
                *reinterpret_cast<uint16_t*>(p.out16 + ((uint64_t)m * p.S + c + k) * p.s_pitch + r) =
                    (uint16_t)pack_f16(v[k], 0.0f);
    }
}

// Persistent: CTA q takes tiles q, q + gridDim, ... of all matrices.  Warp 4 loads 128 x 64 tiles of
// both operands into a ring of stages (TMA, out-of-range rows and columns as zeros), one thread of warp
// 5 issues the MMAs into one of two TMEM accumulators, and warps 0-3 drain the other.
template <Product P>
__global__ void __launch_bounds__(THREADS, 1) ortho_gemm_kernel(const __grid_constant__ GemmParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = smem + STAGES * TILE_STAGE;
    uint64_t* full = reinterpret_cast<uint64_t*>(sB + STAGES * TILE_STAGE);   // [STAGES]  TMA -> MMA
    uint64_t* empty = full + STAGES;              // [STAGES]  MMA -> TMA
    uint64_t* acc_full = empty + STAGES;          // [2]       MMA -> epilogue
    uint64_t* acc_empty = acc_full + ACC_BUFS;    // [2]       epilogue -> MMA
    uint64_t* drain = acc_empty + ACC_BUFS;       // [1]       MMA teardown
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile uint32_t* abort_flag = tmem_slot + 1;

    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < STAGES; ++i) {
            bar_init(saddr(full + i), 1);
            bar_init(saddr(empty + i), 1);
        }
        for (uint32_t i = 0; i < ACC_BUFS; ++i) {
            bar_init(saddr(acc_full + i), 1);
            bar_init(saddr(acc_empty + i), EPI_THREADS);
        }
        bar_init(saddr(drain), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(saddr(tmem_slot)), "r"(TMEM_COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    const uint32_t places = p.batch * p.tiles, kblocks = (p.K + BK - 1) / BK;
    auto fail = [&]() {
        *abort_flag = 1;
        atomicAdd(p.err, 1u);
    };

    if (warp == TMA_WARP) {
        if (lane == 0) {
            uint32_t stage = 0, phase = 0, issued = 0;
            bool ok = true;
            for (uint32_t u = blockIdx.x; u < places && ok; u += gridDim.x) {
                uint32_t m, i, j;
                tile_of<P>(p, u, m, i, j);
                for (uint32_t kb = 0; kb < kblocks; ++kb) {
                    if (!bar_wait(saddr(empty + stage), phase ^ 1, abort_flag)) { fail(); ok = false; break; }
                    const uint32_t bar = saddr(full + stage), k = kb * BK;
                    const uint32_t dA = saddr(sA + stage * TILE_STAGE), dB = saddr(sB + stage * TILE_STAGE);
                    bar_expect_tx(bar, 2 * TILE_STAGE);
                    tma_load_3d(dA, &p.tmA, (int32_t)k, (int32_t)(i * TM), (int32_t)m, bar);
                    if (P == APPLY) {             // X: rows k, 64 columns a box
                        tma_load_3d(dB, &p.tmB, (int32_t)(j * TN), (int32_t)k, (int32_t)m, bar);
                        tma_load_3d(dB + TILE_STAGE / 2, &p.tmB, (int32_t)(j * TN + 64), (int32_t)k, (int32_t)m, bar);
                    } else {
                        tma_load_3d(dB, &p.tmB, (int32_t)k, (int32_t)(j * TN), (int32_t)m, bar);
                    }
                    ++issued;
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                }
            }
            // the last loads of every stage have landed before the CTA can leave
            volatile uint32_t never = 0;
            for (uint32_t i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i)
                (void)bar_wait(saddr(full + i % STAGES), (i / STAGES) & 1, &never);
        }
    } else if (warp == MMA_WARP) {
        if (lane == 0) {
            uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
            bool ok = true;
            for (uint32_t u = blockIdx.x; u < places && ok; u += gridDim.x) {
                if (!bar_wait(saddr(acc_empty + acc), acc_phase ^ 1, abort_flag)) { fail(); break; }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + acc * TN;
                for (uint32_t kb = 0; kb < kblocks; ++kb) {
                    if (!bar_wait(saddr(full + stage), phase, abort_flag)) { fail(); ok = false; break; }
                    tc_fence_after();
                    const uint64_t da = desc_k(saddr(sA + stage * TILE_STAGE));
                    const uint32_t b0 = saddr(sB + stage * TILE_STAGE);
                    const uint64_t db = P == APPLY ? desc_mn(b0) : desc_k(b0);
                    // 16 k further: 32 bytes along a K-contiguous row, 16 rows of 128 bytes otherwise
                    constexpr uint32_t step_b = P == APPLY ? UMMA_K * 128 / 16 : UMMA_K * 2 / 16;
#pragma unroll
                    for (uint32_t k = 0; k < BK / UMMA_K; ++k)
                        umma(d_tmem, da + 2 * k, db + step_b * k, P == APPLY ? IDESC | IDESC_B_MN : IDESC, (kb | k) != 0);
                    umma_commit(saddr(empty + stage));     // the stage is free once these finish
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                }
                if (!ok) break;
                umma_commit(saddr(acc_full + acc));        // the tile is complete in TMEM
                if (++acc == ACC_BUFS) { acc = 0; acc_phase ^= 1; }
            }
            // every MMA this thread issued has finished before TMEM is released
            umma_commit(saddr(drain));
            volatile uint32_t never = 0;
            (void)bar_wait(saddr(drain), 0, &never);
        }
    } else {
        // epilogue: thread t of warp w owns row 32 w + t of every tile
        uint32_t acc = 0, acc_phase = 0;
        for (uint32_t u = blockIdx.x; u < places; u += gridDim.x) {
            uint32_t m, i, j;
            tile_of<P>(p, u, m, i, j);
            const bool mine = bar_wait(saddr(acc_full + acc), acc_phase, abort_flag);
            if (!mine) fail();
            if (!epi_all(mine && !*abort_flag)) break;
            tc_fence_after();
            const uint32_t taddr = tmem_base + ((warp * 32u) << 16) + acc * TN;
#pragma unroll 1
            for (uint32_t g = 0; g < TN / 32; ++g) {
                float v[32];
                tmem_ld32(taddr + g * 32, v);
                finish<P>(p, m, i * TM + warp * 32 + lane, j * TN + g * 32, i != j, v);
            }
            tc_fence_before();
            bar_arrive(saddr(acc_empty + acc));            // the accumulator may be overwritten
            if (++acc == ACC_BUFS) { acc = 0; acc_phase ^= 1; }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(TMEM_COLS) : "memory");
}

struct UpdateParams {
    const char* x;
    uint64_t x_pitch, x_stride;
    char* mom;                   // f32, or null
    uint64_t mom_pitch, mom_stride;
    float mu, eps;
    uint32_t nesterov, x_dt;
    uint32_t rows, cols, parts;
    float* sums;                 // [batch][parts]
    float* x32;
    __half* x16;
    uint64_t l_pitch;
    uint32_t S;
};

// Sum over a CTA's 256 threads, in one fixed order, the same bits in each.
__device__ __forceinline__ float cta_sum(float v, float (&slot)[8]) {
#pragma unroll
    for (uint32_t o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (threadIdx.x % 32 == 0) slot[threadIdx.x / 32] = v;
    __syncthreads();
    v = slot[0];
#pragma unroll
    for (uint32_t w = 1; w < 8; ++w) v += slot[w];
    return v;
}

// The momentum's update, and a part of |u|^2 from each of `parts` CTAs a matrix, which stride over its
// rows in chunks of 8 columns (VEC) or single elements.
template <bool VEC>
__global__ void __launch_bounds__(256) ortho_update_kernel(const __grid_constant__ UpdateParams p) {
    __shared__ float slot[8];
    constexpr uint32_t W = VEC ? 8 : 1;
    const uint32_t m = blockIdx.y, per_row = (p.cols + W - 1) / W;
    const char* x = p.x + (uint64_t)m * p.x_stride;
    char* mom = p.mom ? p.mom + (uint64_t)m * p.mom_stride : nullptr;
    const uint64_t total = (uint64_t)p.rows * per_row;
    float sum = 0.0f;
#pragma unroll 4
    for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (uint64_t)p.parts * 256) {
        const uint32_t r = (uint32_t)(i / per_row), c = (uint32_t)(i - (uint64_t)r * per_row) * W;
        float u[8], v[8];
        if (VEC) load8<true>(x + r * p.x_pitch, p.x_dt, c, p.cols, u);
        else u[0] = load1(x + r * p.x_pitch, p.x_dt, c);
        if (mom) {
            char* row = mom + r * p.mom_pitch;
            if (VEC) load8<true>(row, DTT_F32, c, p.cols, v);
            else v[0] = load1(row, DTT_F32, c);
#pragma unroll
            for (uint32_t k = 0; k < W; ++k) {
                v[k] = p.mu * v[k] + u[k];
                u[k] = p.nesterov ? u[k] + p.mu * v[k] : v[k];
            }
            if (VEC) store8<true>(row, DTT_F32, c, p.cols, v);
            else store1(row, DTT_F32, c, v[0]);
        }
#pragma unroll
        for (uint32_t k = 0; k < W; ++k) sum += u[k] * u[k];
    }
    sum = cta_sum(sum, slot);
    if (threadIdx.x == 0) p.sums[(uint64_t)m * p.parts + blockIdx.x] = sum;
}

// 1 / (|u| + eps) of matrix m, from its parts; 0 where that overflows (u is then 0 in f16 as well).
__device__ __forceinline__ float inverse_norm(const UpdateParams& p, uint32_t m, float (&slot)[8]) {
    float sum = 0.0f;
#pragma unroll 4
    for (uint32_t i = threadIdx.x; i < p.parts; i += 256) sum += p.sums[(uint64_t)m * p.parts + i];
    const float inv = 1.0f / (sqrtf(cta_sum(sum, slot)) + p.eps);
    return isinf(inv) ? 0.0f : inv;
}

// u again (the momentum is updated by now) and X = u / (|u| + eps), in f32 and as the f16 operand: rows
// <= cols, 16-byte aligned.  A thread has two chunks of 8 columns under way.
__global__ void __launch_bounds__(256) ortho_start_kernel(const __grid_constant__ UpdateParams p) {
    __shared__ float slot[8];
    const uint32_t m = blockIdx.y, per_row = p.cols / 8, total = p.rows * per_row, step = gridDim.x * 256;
    const char* x = p.x + (uint64_t)m * p.x_stride;
    const char* mom = p.mom ? p.mom + (uint64_t)m * p.mom_stride : nullptr;
    float* x32 = p.x32 + (uint64_t)m * p.S * p.l_pitch;
    __half* x16 = p.x16 + (uint64_t)m * p.S * p.l_pitch;
    const float inv = inverse_norm(p, m, slot);
    for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < total; i += 2 * step) {
        float u[2][8], v[2][8];
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
            const uint32_t j = min(i + h * step, total - 1), r = j / per_row, c = 8 * (j - r * per_row);
            load8<true>(x + r * p.x_pitch, p.x_dt, c, p.cols, u[h]);
            if (mom) load8<true>(mom + r * p.mom_pitch, DTT_F32, c, p.cols, v[h]);
        }
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
            const uint32_t j = i + h * step, r = j / per_row, c = 8 * (j - r * per_row);
            if (j >= total) break;
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k) {
                if (mom) u[h][k] = p.nesterov ? u[h][k] + p.mu * v[h][k] : v[h][k];
                u[h][k] *= inv;
            }
            store8<true>(reinterpret_cast<char*>(x32 + r * p.l_pitch), DTT_F32, c, p.cols, u[h]);
            *reinterpret_cast<uint4*>(x16 + r * p.l_pitch + c) =
                make_uint4(pack_f16(u[h][0], u[h][1]), pack_f16(u[h][2], u[h][3]), pack_f16(u[h][4], u[h][5]),
                           pack_f16(u[h][6], u[h][7]));
        }
    }
}

// The same for any alignment, and for rows > cols (TALL: turned over in shared memory): a tile of 64 x
// 64 elements a CTA.
template <bool TALL>
__global__ void __launch_bounds__(256) ortho_start_tiles_kernel(const __grid_constant__ UpdateParams p) {
    __shared__ float slot[8];
    __shared__ float tile[TALL ? kStartTile : 1][kStartTile + 1];
    const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32, m = blockIdx.z;
    const uint32_t r0 = blockIdx.y * kStartTile, c0 = blockIdx.x * kStartTile;
    const char* x = p.x + (uint64_t)m * p.x_stride;
    const char* mom = p.mom ? p.mom + (uint64_t)m * p.mom_stride : nullptr;
    float u[kStartTile / 8][2];
#pragma unroll
    for (uint32_t k = 0; k < kStartTile / 8; ++k)
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
            const uint32_t r = r0 + warp + 8 * k, c = c0 + lane + 32 * h;
            u[k][h] = 0.0f;
            if (r < p.rows && c < p.cols) {
                if (!mom || p.nesterov) u[k][h] = load1(x + r * p.x_pitch, p.x_dt, c);
                if (mom) {
                    const float v = load1(mom + r * p.mom_pitch, DTT_F32, c);
                    u[k][h] = p.nesterov ? u[k][h] + p.mu * v : v;
                }
            }
        }
    const float inv = inverse_norm(p, m, slot);
    float* x32 = p.x32 + (uint64_t)m * p.S * p.l_pitch;
    __half* x16 = p.x16 + (uint64_t)m * p.S * p.l_pitch;
    if (TALL) {
#pragma unroll
        for (uint32_t k = 0; k < kStartTile / 8; ++k)
#pragma unroll
            for (uint32_t h = 0; h < 2; ++h) tile[warp + 8 * k][lane + 32 * h] = u[k][h];
        __syncthreads();
    }
#pragma unroll
    for (uint32_t k = 0; k < kStartTile / 8; ++k)
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
            const uint32_t a = warp + 8 * k, b = lane + 32 * h;      // TALL: column a, row b of the tile
            const uint32_t r = r0 + (TALL ? b : a), c = c0 + (TALL ? a : b);
            if (r < p.rows && c < p.cols) {
                const float v = (TALL ? tile[b][a] : u[k][h]) * inv;
                const uint64_t at = TALL ? c * p.l_pitch + r : r * p.l_pitch + c;
                x32[at] = v;
                x16[at] = __float2half_rn(v);
            }
        }
}

// A batch of matrices rows x cols f16, `pitch` elements a row, in boxes of 64 columns (128 bytes,
// swizzled) by box_rows rows.
bool make_map(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint64_t batch, uint64_t pitch,
              uint32_t box_rows) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    const cuuint64_t dims[3] = {cols, rows, batch};
    const cuuint64_t strides[2] = {pitch * 2, rows * pitch * 2};
    const cuuint32_t box[3] = {64, box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Layout {
    uint64_t S, L, s_pitch, l_pitch;                 // elements
    uint64_t x32, x16[2], gram, poly, sums, bytes;   // byte offsets in the workspace
};

Layout layout_of(const dtt_ortho_desc& d) {
    Layout l{};
    l.S = std::min(d.rows, d.cols);
    l.L = std::max(d.rows, d.cols);
    l.s_pitch = (l.S + 63) / 64 * 64;
    l.l_pitch = (l.L + 63) / 64 * 64;
    uint64_t at = 0;
    auto take = [&](uint64_t bytes) {
        const uint64_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    l.x32 = take(d.batch * l.S * l.l_pitch * 4);
    l.x16[0] = take(d.batch * l.S * l.l_pitch * 2);
    l.x16[1] = take(d.batch * l.S * l.l_pitch * 2);
    l.gram = take(d.batch * l.S * l.s_pitch * 2);
    l.poly = take(d.batch * l.S * l.s_pitch * 2);
    l.sums = take((uint64_t)d.batch * kMaxParts * 4);
    l.bytes = at;
    return l;
}

int check_desc(const char* who, const dtt_ortho_desc* d) {
    if (!d) return fail(DTT_EINVAL, "%s: null desc", who);
    if (d->x_dtype != DTT_BF16 && d->x_dtype != DTT_F32) return fail(DTT_EINVAL, "%s: x is bf16 or f32", who);
    if (d->rows == 0 || d->cols == 0 || d->rows > 65536 || d->cols > 65536)
        return fail(DTT_EINVAL, "%s: rows and cols must be 1 .. 65536", who);
    if (d->batch == 0 || d->batch > 65535) return fail(DTT_EINVAL, "%s: batch must be 1 .. 65535", who);
    if (((d->rows + TM - 1) / TM) * ((d->cols + TN - 1) / TN) * d->batch >= (1ull << 31))
        return fail(DTT_EINVAL, "%s: 2^31 tiles of 128 x 128 or more", who);
    if (d->steps == 0 || d->steps > DTT_ORTHO_MAX_STEPS)
        return fail(DTT_EINVAL, "%s: steps must be 1 .. %d", who, DTT_ORTHO_MAX_STEPS);
    if (d->momentum > 1 || d->nesterov > 1 || (d->nesterov && !d->momentum))
        return fail(DTT_EINVAL, "%s: momentum and nesterov are 0 or 1, nesterov with momentum alone", who);
    if (!std::isfinite(d->mu) || !std::isfinite(d->scale) || !std::isfinite(d->eps) || !(d->eps > 0.0f))
        return fail(DTT_EINVAL, "%s: mu, scale and eps must be finite and eps positive", who);
    // the iterate's largest singular value, step by step: its operands must stay within f16
    double bound = 1.0;
    for (uint32_t k = 0; k < d->steps; ++k) {
        const double a = d->coeffs[k][0], b = d->coeffs[k][1], c = d->coeffs[k][2];
        if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c))
            return fail(DTT_EINVAL, "%s: step %u has a coefficient that is not finite", who, k);
        if (std::fabs(b) * bound * bound + std::fabs(c) * bound * bound * bound * bound > 1024.0)
            return fail(DTT_EINVAL, "%s: step %u's coefficients leave f16's range", who, k);
        double next = 0.0;
        for (int i = 0; i <= 1024; ++i) {
            const double s = bound * i / 1024, q = s * s;
            next = std::max(next, std::fabs(s * (a + q * (b + q * c))));
        }
        bound = next;
        if (bound > 16.0) return fail(DTT_EINVAL, "%s: step %u's coefficients let the iterate grow past 16", who, k);
    }
    return DTT_OK;
}

template <Product P>
cudaError_t prepare_gemm() {
    cudaError_t e = prepare_kernel(ortho_gemm_kernel<P>);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(ortho_gemm_kernel<P>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
    return e;
}

}  // namespace

cudaError_t preload_ortho_kernels() {
    cudaError_t e = prepare_gemm<GRAM>();
    if (e == cudaSuccess) e = prepare_gemm<POLY>();
    if (e == cudaSuccess) e = prepare_gemm<APPLY>();
    if (e == cudaSuccess) e = prepare_kernel(ortho_update_kernel<true>);
    if (e == cudaSuccess) e = prepare_kernel(ortho_update_kernel<false>);
    if (e == cudaSuccess) e = prepare_kernel(ortho_start_kernel);
    if (e == cudaSuccess) e = prepare_kernel(ortho_start_tiles_kernel<true>);
    if (e == cudaSuccess) e = prepare_kernel(ortho_start_tiles_kernel<false>);
    return e;
}

}  // namespace dtt

using namespace dtt;

struct dtt_ortho {
    dtt_ortho_desc d;
    Layout l;
    char* ws;
    uint32_t sms;
    CUtensorMap x_rows[2];       // x16, K-major operand of A = X X^T: boxes of 64 x 128
    CUtensorMap x_cols[2];       // x16, N-contiguous operand of the last product: boxes of 64 x 64
    CUtensorMap gram, poly;      // boxes of 64 x 128
};

extern "C" int dtt_ortho_workspace(const dtt_ortho_desc* d, uint64_t* bytes) {
    const int rc = check_desc("dtt_ortho_workspace", d);
    if (rc) return rc;
    if (!bytes) return fail(DTT_EINVAL, "dtt_ortho_workspace: null bytes");
    *bytes = layout_of(*d).bytes;
    return DTT_OK;
}

extern "C" int dtt_ortho_create(const dtt_ortho_desc* d, void* workspace, uint64_t workspace_bytes, dtt_ortho** out) {
    const char* who = "dtt_ortho_create";
    int rc = check_desc(who, d);
    if (rc) return rc;
    if (!out) return fail(DTT_EINVAL, "%s: null out", who);
    *out = nullptr;
    const Layout l = layout_of(*d);
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 || workspace_bytes < l.bytes)
        return fail(DTT_EINVAL, "%s: the workspace is missing, misaligned or shorter than %llu bytes", who,
                    (unsigned long long)l.bytes);
    if ((rc = preload_once())) return rc;
    int dev = 0, sms = 0;
    DTT_CUDA_TRY(cudaGetDevice(&dev));
    DTT_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    dtt_ortho* o = new (std::nothrow) dtt_ortho;
    if (!o) return fail(DTT_ENOMEM, "%s: out of host memory", who);
    o->d = *d;
    o->l = l;
    o->ws = static_cast<char*>(workspace);
    o->sms = (uint32_t)sms;
    bool ok = make_map(&o->gram, o->ws + l.gram, l.S, l.S, d->batch, l.s_pitch, TM) &&
              make_map(&o->poly, o->ws + l.poly, l.S, l.S, d->batch, l.s_pitch, TM);
    for (int i = 0; i < 2 && ok; ++i)
        ok = make_map(&o->x_rows[i], o->ws + l.x16[i], l.L, l.S, d->batch, l.l_pitch, TM) &&
             make_map(&o->x_cols[i], o->ws + l.x16[i], l.L, l.S, d->batch, l.l_pitch, BK);
    if (!ok) {
        delete o;
        return fail(DTT_ECUDA, "%s: cannot encode the tensor maps", who);
    }
    *out = o;
    return DTT_OK;
}

extern "C" void dtt_ortho_destroy(dtt_ortho* o) { delete o; }

extern "C" int dtt_ortho_run(dtt_ortho* o, const void* x, uint64_t x_pitch, uint64_t x_stride, float* momentum,
                             uint64_t momentum_pitch, uint64_t momentum_stride, void* out, uint64_t out_pitch,
                             uint64_t out_stride, uint32_t* err, cudaStream_t stream) {
    const char* who = "dtt_ortho_run";
    if (!o || !x || !out || !err) return fail(DTT_EINVAL, "%s: null argument", who);
    const dtt_ortho_desc& d = o->d;
    const Layout& l = o->l;
    if ((momentum != nullptr) != (d.momentum != 0))
        return fail(DTT_EINVAL, "%s: momentum is an argument exactly where the desc has it", who);
    const struct { const char* name; const void* p; uint64_t pitch, stride, e; } args[] = {
        {"x", x, x_pitch, x_stride, d.x_dtype == DTT_BF16 ? 2ull : 4ull},
        {"momentum", momentum, momentum_pitch, momentum_stride, 4},
        {"out", out, out_pitch, out_stride, 2}};
    for (const auto& a : args) {
        if (!a.p) continue;
        if (reinterpret_cast<uintptr_t>(a.p) % a.e || a.pitch % a.e || a.stride % a.e)
            return fail(DTT_EINVAL, "%s: %s must be aligned to its elements", who, a.name);
        if (d.rows > 1 && a.pitch < d.cols * a.e) return fail(DTT_EINVAL, "%s: %s: the pitch is less than a row", who, a.name);
        if (d.batch > 1 && a.stride < (d.rows - 1) * a.pitch + d.cols * a.e)
            return fail(DTT_EINVAL, "%s: %s: the stride is less than a matrix", who, a.name);
    }
    if (reinterpret_cast<uintptr_t>(err) % 4) return fail(DTT_EINVAL, "%s: err is misaligned", who);

    float* x32 = reinterpret_cast<float*>(o->ws + l.x32);
    UpdateParams up{};
    up.x = static_cast<const char*>(x);
    up.x_pitch = x_pitch;
    up.x_stride = x_stride;
    up.mom = reinterpret_cast<char*>(momentum);
    up.mom_pitch = momentum_pitch;
    up.mom_stride = momentum_stride;
    up.mu = d.mu;
    up.eps = d.eps;
    up.nesterov = d.nesterov;
    up.x_dt = d.x_dtype;
    up.rows = (uint32_t)d.rows;
    up.cols = (uint32_t)d.cols;
    up.sums = reinterpret_cast<float*>(o->ws + l.sums);
    up.x32 = x32;
    up.x16 = reinterpret_cast<__half*>(o->ws + l.x16[0]);
    up.l_pitch = l.l_pitch;
    up.S = (uint32_t)l.S;
    const bool tall = d.rows > d.cols;
    bool vec = d.cols % 8 == 0;
    for (const auto& a : args)
        if (a.p != out && a.p) vec = vec && reinterpret_cast<uintptr_t>(a.p) % 16 == 0 && a.pitch % 16 == 0 && a.stride % 16 == 0;
    const uint64_t items = d.rows * (vec ? d.cols / 8 : d.cols);
    up.parts = (uint32_t)std::min<uint64_t>((items + 1023) / 1024, std::max(kMaxParts / d.batch, 1u));
    if (vec) ortho_update_kernel<true><<<dim3(up.parts, d.batch), 256, 0, stream>>>(up);
    else ortho_update_kernel<false><<<dim3(up.parts, d.batch), 256, 0, stream>>>(up);
    if (vec && !tall) {
        const uint32_t ctas = (uint32_t)std::min<uint64_t>((items + 511) / 512, std::max(8 * o->sms / d.batch, 1u));
        ortho_start_kernel<<<dim3(ctas, d.batch), 256, 0, stream>>>(up);
    } else {
        const dim3 tiles((up.cols + kStartTile - 1) / kStartTile, (up.rows + kStartTile - 1) / kStartTile, d.batch);
        if (tall) ortho_start_tiles_kernel<true><<<tiles, 256, 0, stream>>>(up);
        else ortho_start_tiles_kernel<false><<<tiles, 256, 0, stream>>>(up);
    }

    GemmParams g{};
    g.S = (uint32_t)l.S;
    g.batch = d.batch;
    g.s_pitch = l.s_pitch;
    g.l_pitch = l.l_pitch;
    g.x32 = x32;
    g.err = err;
    g.scale = d.scale;
    g.transposed = tall;
    g.out_vec = reinterpret_cast<uintptr_t>(out) % 16 == 0 && out_pitch % 16 == 0 && (d.batch == 1 || out_stride % 16 == 0);
    g.out_pitch = out_pitch;
    g.out_stride = out_stride;
    g.tiles_m = (uint32_t)((l.S + TM - 1) / TM);
    const uint32_t triangle_tiles = g.tiles_m * (g.tiles_m + 1) / 2;
    auto grid = [&](uint64_t tiles) { return (uint32_t)std::min<uint64_t>(tiles * d.batch, o->sms); };
    for (uint32_t k = 0; k < d.steps; ++k) {
        const uint32_t now = k & 1;
        g.a = d.coeffs[k][0];
        g.b = d.coeffs[k][1];
        g.c = d.coeffs[k][2];
        g.L = g.S;
        g.tiles_n = g.tiles_m;
        g.tiles = triangle_tiles;
        g.tmA = g.tmB = o->x_rows[now];
        g.K = (uint32_t)l.L;
        g.out16 = reinterpret_cast<__half*>(o->ws + l.gram);
        ortho_gemm_kernel<GRAM><<<grid(g.tiles), THREADS, SMEM_BYTES, stream>>>(g);
        g.tmA = g.tmB = o->gram;
        g.K = g.S;
        g.gram = g.out16;
        g.out16 = reinterpret_cast<__half*>(o->ws + l.poly);
        ortho_gemm_kernel<POLY><<<grid(g.tiles), THREADS, SMEM_BYTES, stream>>>(g);
        g.tmA = o->poly;
        g.tmB = o->x_cols[now];
        g.L = (uint32_t)l.L;
        g.tiles_n = (uint32_t)((l.L + TN - 1) / TN);
        g.tiles = g.tiles_m * g.tiles_n;
        g.out16 = reinterpret_cast<__half*>(o->ws + l.x16[now ^ 1]);
        g.out = k + 1 == d.steps ? static_cast<char*>(out) : nullptr;
        ortho_gemm_kernel<APPLY><<<grid(g.tiles), THREADS, SMEM_BYTES, stream>>>(g);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(DTT_ECUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    return DTT_OK;
}

// Orthogonalising an update by Newton-Schulz products (dtt_ops.h): X <- a X + (b A + c A A) X with
// A = X X^T, a few times over, for a batch of S x L matrices (S <= L: the smaller side first).
//
// Precision.  The tensor cores take f16 operands and add in f32: f16 has 11 significant bits where
// bf16 has 8, at the same rate, and every value here is below 3 in magnitude.  X is held in 32 bits,
// as its f16 operand (hi) and the rest of it times 2^11 in f16 (lo): 22 significant bits, and nothing
// below 2^-35 is lost.  An X of one f16 would carry noise of 2^-12 |X| in the singular directions that
// the update lacks, where a step multiplies it by a = 3.44: for a rank-1 update five steps in f16 end
// 10 % off, in bf16 75 %, with 32 bits 0.17 % (the bf16 output).  The noise of rounded operands meets X
// only through b A + c A A, whose range holds nothing of those directions.
//
// A and b A + c A A are symmetric: only tiles on and below the diagonal are computed, and each is
// stored twice, once transposed (not in the resident form).
//
// Four forms, the smallest matrices first: resident (S <= 128, L <= 4096: one launch, X in the shared memory
// of a cluster); a launch a product on tiles of 128 x 128 split over clusters along k (up to S = 256 with
// the second product within the third); a launch a product by CTA pairs on tiles of 256 rows; and all
// products of all steps in one launch of such pairs.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <new>
#include <type_traits>

#include <cuda_fp16.h>

#include "dtt_ops.h"
#include "internal.h"
#include "rowio.cuh"

namespace dtt {
namespace {

constexpr uint32_t BK = 64, UMMA_K = 16;
constexpr uint32_t HALF_STAGE = 128 * BK * 2;        // 16 KiB: 128 rows or columns of an operand
constexpr uint32_t STAGES = 5;
constexpr uint32_t ACC_BUFS = 2;                     // TMEM accumulators of the pair form
constexpr uint32_t EPI_WARPS = 8;                    // two for each 32 lanes of TMEM: half of the columns each
constexpr uint32_t THREADS = EPI_WARPS * 32 + 96;    // + TMA warp, MMA warp, slab warp
constexpr uint32_t TMA_WARP = EPI_WARPS, MMA_WARP = EPI_WARPS + 1, SLAB_WARP = EPI_WARPS + 2;
constexpr uint32_t SLAB = 64;                        // pair form: columns that its epilogue takes at a time
constexpr uint32_t SLAB_BYTES = 128 * SLAB * 2;      // of one f16 array: 16 KiB
constexpr uint32_t SLAB_BUFS = 2;
constexpr uint32_t TILES = 160;                      // of a cluster of the pair form, worked out beforehand
// Looks at an mbarrier, at most: one that fails takes 4 us, so some seconds.  A build of its own makes the waits of
// some threads run out (DTT_ORTHO_LATE), or all of them sooner.
#ifndef DTT_ORTHO_WAIT_LIMIT
#define DTT_ORTHO_WAIT_LIMIT (1u << 20)
#endif
#ifndef DTT_ORTHO_LATE
#define DTT_ORTHO_LATE false
#endif
constexpr uint32_t WAIT_LIMIT = DTT_ORTHO_WAIT_LIMIT;
constexpr uint32_t SMEM_BYTES = 1024 /* alignment slack */ + STAGES * 2 * HALF_STAGE + SLAB_BUFS * 2 * SLAB_BYTES + 256 + TILES * 8;
// instruction descriptor (kind::f16): f32 accumulator, f16 operands, M = m, N = n
__host__ __device__ constexpr uint32_t idesc(uint32_t m, uint32_t n) { return (1u << 4) | ((n >> 3) << 17) | ((m >> 4) << 24); }
constexpr uint32_t IDESC_B_MN = 1u << 16;            // B stored with N contiguous
// split form: the tile's f32 sums, and its f16 or bf16 rows, in the shared memory of the stages
constexpr uint32_t T16_PITCH = 130;                  // 16-bit elements: columns fall on different banks
constexpr uint32_t T16_OFFSET = 128 * 128 * 4;
static_assert(T16_OFFSET + 128 * T16_PITCH * 2 <= STAGES * 2 * HALF_STAGE && 128 * 128 * 4 <= SLAB_BUFS * 2 * SLAB_BYTES,
              "the tile fits the stages, the sums of the cluster the slabs");

constexpr uint32_t kStartTile = 64;                  // ortho_start_tiles_kernel: elements a side
constexpr uint32_t START_CTAS = 8;                   // of the update and start kernels on a SM
constexpr uint32_t kMaxParts = kSms * START_CTAS;     // CTAs of the update's launch at most: all run at once

enum Product { GRAM, POLY, APPLY };

// A product in the split form.
struct GemmParams {
    CUtensorMap tmA, tmB;        // operands
    uint32_t S, L, K;            // output rows S and columns (GRAM, POLY: S; APPLY: L)
    uint32_t batch, tiles_m, tiles;   // tiles: of one matrix
    uint64_t s_pitch, l_pitch;   // elements between rows of the S-wide and L-wide arrays
    float a, b, c;
    const __half* gram;          // POLY: A
    __half* out16;               // GRAM: A; POLY: b A + c A A; APPLY: the next hi
    const __half* hi;            // APPLY
    __half* lo;                  // APPLY, in place
    char* out;                   // APPLY, last step: the result (see Result); null: not the last step
    uint64_t out_pitch, out_stride;
    float scale;
    uint32_t transposed, out_vec;
    uint32_t* err;
};

// Where the result goes: scale X, rounded to bf16, by rows or (transposed) by columns of X.
struct Result {
    char* out;                   // of one matrix
    uint64_t pitch;
    uint32_t S, L;
    float scale;
    uint32_t transposed, vec;    // vec: rows of 16-byte words
};

__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Bounded wait for the phase of the given parity; false when the limit ran out or another role
// already reported an error (abort; null: a wait for what is under way, before a CTA leaves, which
// nothing cuts short).
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile uint32_t* abort) {
    if (abort && (DTT_ORTHO_LATE)) return false;
    for (uint32_t i = 0; i < WAIT_LIMIT; ++i) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done) : "r"(bar), "r"(parity) : "memory");
        if (done) return true;
        if (abort && (i & 255) == 0 && *abort) return false;
    }
    return false;
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
// 16 k further, in the descriptor's units: 32 bytes along a K-contiguous row, 16 rows of 128 bytes else
constexpr uint32_t STEP_K = UMMA_K * 2 / 16, STEP_MN = UMMA_K * 128 / 16;
template <Product P>
__device__ __forceinline__ constexpr uint32_t step_b() { return P == APPLY ? STEP_MN : STEP_K; }

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

// The iterate's two halves: x = hi + 2^-11 lo.
constexpr float LO_SCALE = 2048.0f;
__device__ __forceinline__ float2 join(uint32_t hi, uint32_t lo) {
    const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi)), l = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    return make_float2(h.x + l.x * (1.0f / LO_SCALE), h.y + l.y * (1.0f / LO_SCALE));
}
__device__ __forceinline__ void part(float x, float y, uint32_t& hi, uint32_t& lo) {
    hi = pack_f16(x, y);
    const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    lo = pack_f16((x - h.x) * LO_SCALE, (y - h.y) * LO_SCALE);
}

// Two f16 terms of each value: x = hi + below, to 22 bits.
__device__ __forceinline__ void two_terms(float x, float y, uint32_t& hi, uint32_t& below) {
    hi = pack_f16(x, y);
    const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    below = pack_f16(x - h.x, y - h.y);
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

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// The shared::cluster address of the same shared-memory offset in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t at_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// ---- pair form ---------------------------------------------------------------------------------
// The products first .. last of `steps` steps in one launch.  Alone (first == last, one step) a product
// follows the launch before it.  With counters, all products of all steps are one sequence of tiles that
// the clusters, all resident, take in turn, and a tile waits for what it reads: each row block of 256 rows
// counts, per matrix and product, the CTAs that have stored into it.
struct PairParams {
    CUtensorMap hi_rows[2], lo_rows, gram, poly;             // boxes of 64 x 128 (columns x rows)
    CUtensorMap hi_cols[2], gram_blocks, poly_blocks;        // boxes of 64 x 64
    uint32_t S, L, batch;
    uint32_t n, across, tn;      // row blocks of S; tiles of tn columns (256 or 128) across L
    uint32_t first, last;
    uint32_t step, steps;        // the first step of this launch (its parity names the hi that is read), and how many
    uint32_t* counters;          // [batch][GRAM, POLY, APPLY][n], then [batch][tiles of A] for the parts; or null
    uint32_t splits;             // of A's k blocks, over as many places; 1 without counters
    float* parts;                // the f32 sums of all but the last of them: [batch][tiles of A][splits - 1][256 x 256]
    char* out;                   // the result of the launch's last step (see Result); null: another launch follows
    uint64_t out_pitch, out_stride;
    float scale;
    uint32_t transposed, out_vec;
    uint32_t* err;
    float coeffs[DTT_ORTHO_MAX_STEPS][3];                    // of this launch's steps
};

// Place u of the sequence: its step (of this launch), product, matrix and tile.  A by rows and b A + c A A
// by columns, and the last product by rows again, because then the first row blocks of each are complete
// while the last tiles of it still run.  4096 x 4096 fills 7.0 rounds of the clusters a step, where a launch
// a product takes 2 + 2 + 4: 990 us for five steps with these, 915 in one sequence.
struct Tile {
    uint32_t k, product, m, i, j;
    uint32_t split, place;       // A: which part of its k blocks, and its place in the triangle
};

__device__ __forceinline__ Tile pair_tile(const PairParams& p, uint32_t u) {
    const uint32_t square = p.n * (p.n + 1) / 2, oblong = p.n * p.across;
    uint32_t per_step = 0;
    auto places = [&](uint32_t q) { return q == APPLY ? oblong : q == GRAM ? square * p.splits : square; };   // of a matrix
    for (uint32_t q = p.first; q <= p.last; ++q) per_step += p.batch * places(q);
    Tile t{};
    t.k = u / per_step;
    uint32_t r = u % per_step;
    for (t.product = p.first;; ++t.product) {
        const uint32_t all = p.batch * places(t.product);
        if (r < all) break;
        r -= all;
    }
    const uint32_t each = places(t.product);
    t.m = r / each;
    r %= each;
    if (t.product == APPLY) {
        t.i = r / p.across;
        t.j = r % p.across;
    } else if (t.product == GRAM) {
        t.split = r % p.splits;
        t.place = r / p.splits;
        triangle(t.place, t.i, t.j);
    } else {
        triangle(square - 1 - r, t.i, t.j);       // the columns of a triangle are the rows of it turned over
        const uint32_t i = p.n - 1 - t.j;
        t.j = p.n - 1 - t.i;
        t.i = i;
    }
    return t;
}

// A tile in 8 bytes: steps 5 bits, matrices 16, tiles a side 9 each.  (Worked out by each warp at its turn:
// eight of 1024 x 1024 262 us and not 229.)
__device__ __forceinline__ uint2 packed(const Tile& t) {
    return make_uint2(t.k | t.product << 5 | t.split << 7 | t.m << 16, t.i | t.j << 16);
}
__device__ __forceinline__ Tile unpacked(uint2 v) {
    Tile t{v.x & 31, v.x >> 5 & 3, v.x >> 16, v.y & 0xFFFF, v.y >> 16, v.x >> 7 & 7, 0};
    t.place = t.i * (t.i + 1) / 2 + t.j;
    return t;
}

__device__ __forceinline__ uint32_t pair_tiles(const PairParams& p) {
    uint32_t per_step = 0;
    for (uint32_t q = p.first; q <= p.last; ++q)
        per_step += p.batch * (q == APPLY ? p.n * p.across : p.n * (p.n + 1) / 2 * (q == GRAM ? p.splits : 1));
    return per_step * p.steps;
}

// Wait (bounded) until a counter has reached `target`.
__device__ __forceinline__ bool reached(const uint32_t* c, uint32_t target, volatile uint32_t* abort) {
    for (uint32_t polls = 0; polls < 4 * WAIT_LIMIT; ++polls) {
        uint32_t v;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(c) : "memory");
        if (v >= target) return true;
        if ((polls & 63) == 63 && *abort) return false;
        __nanosleep(64);
    }
    return false;
}

// The same for `target` CTAs that have stored into row block i of product q of matrix m.
__device__ __forceinline__ bool stored(const PairParams& p, uint32_t m, uint32_t q, uint32_t i, uint32_t target, volatile uint32_t* abort) {
    return reached(p.counters + (m * 3 + q) * p.n + i, target, abort);
}

// Everything that tile t reads is there, for copies too.  X of step k was complete before b A + c A A of any
// of its rows could be, so the last product waits for these alone; and whoever read what a tile
// overwrites had stored before what the tile waits for could be stored.
__device__ __forceinline__ bool inputs_ready(const PairParams& p, const Tile& t, volatile uint32_t* abort) {
    if (!p.counters) return true;
    bool ok = true;
    if (t.product == GRAM && t.k > 0) {
        const uint32_t target = 2 * p.across * t.k;
        ok = stored(p, t.m, APPLY, t.i, target, abort) && stored(p, t.m, APPLY, t.j, target, abort);
    } else if (t.product == POLY) {
        const uint32_t target = 2 * p.n * (t.k + 1);
        ok = stored(p, t.m, GRAM, t.i, target, abort) && stored(p, t.m, GRAM, t.j, target, abort);
    } else if (t.product == APPLY) {
        ok = stored(p, t.m, POLY, t.i, 2 * p.n * (t.k + 1), abort);
    }
    asm volatile("fence.proxy.async.global;" ::: "memory");
    return ok;
}

// This thread's copies of tile t have been written: count the CTA.
__device__ __forceinline__ void count_stored(const PairParams& p, const Tile& t) {
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    asm volatile("fence.proxy.async.global;" ::: "memory");
    uint32_t* c = p.counters + (t.m * 3 + t.product) * p.n;
    asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(c + t.i) : "memory");
    if (t.product != APPLY && t.i != t.j) asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(c + t.j) : "memory");
}

// The k blocks of tile t, `all` of them in its product: first and one past the last.
__device__ __forceinline__ uint2 k_blocks(const PairParams& p, const Tile& t, uint32_t all) {
    if (t.product != GRAM) return make_uint2(0, all);
    const uint32_t each = (all + p.splits - 1) / p.splits;
    return make_uint2(t.split * each, min((t.split + 1) * each, all));
}

// Sums of a part of A's k blocks: what warp `warp` of CTA q holds of columns 64 g .., as its lanes hold it.  The
// tile's last part adds the others in their order.
__device__ __forceinline__ float4* part_of(const PairParams& p, const Tile& t, uint32_t split, uint32_t q, uint32_t warp, uint32_t g) {
    const uint64_t tile = (uint64_t)t.m * (p.n * (p.n + 1) / 2) + t.place;
    return reinterpret_cast<float4*>(p.parts + (tile * (p.splits - 1) + split) * 65536) + ((q * EPI_WARPS + warp) * 4 + g) * 256;
}
__device__ __forceinline__ uint32_t* parts_counter(const PairParams& p, const Tile& t) {
    return p.counters + p.batch * 3 * p.n + t.m * (p.n * (p.n + 1) / 2) + t.place;
}

// A slab is 128 rows by 64 columns of f16 in shared memory, rows of 128 bytes with their 16-byte words
// swizzled by the row, as the tensor maps move it.  The epilogue's thread with lane `lane` of warp w
// holds row 32 (w % 4) + lane and columns 32 (w / 4) .. of it: words 4 (w / 4) .. + 3.
__device__ __forceinline__ uint4& slab_word(uint8_t* slab, uint32_t row, uint32_t word) {
    return *reinterpret_cast<uint4*>(slab + row * 128 + ((word ^ (row & 7)) << 4));
}

// A, or b A + c A A of the slab's A: the thread's 32 columns into the slab and, for the mirrored part, into
// the two blocks of 64 columns by 64 rows behind it, as rows.
template <bool POLYNOMIAL>
__device__ __forceinline__ void finish(float b, float c, uint8_t* slab, uint32_t row, uint32_t half, bool mirror, float (&v)[32]) {
    uint8_t* turned = slab + SLAB_BYTES + row / 64 * (SLAB_BYTES / 2);
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k) {
        uint4& word = slab_word(slab, row, 4 * half + k);
        if (POLYNOMIAL) {
            const uint32_t g[4] = {word.x, word.y, word.z, word.w};
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&g[e]));
                v[8 * k + 2 * e] = c * v[8 * k + 2 * e] + b * f.x;
                v[8 * k + 2 * e + 1] = c * v[8 * k + 2 * e + 1] + b * f.y;
            }
        }
        word = make_uint4(pack_f16(v[8 * k], v[8 * k + 1]), pack_f16(v[8 * k + 2], v[8 * k + 3]),
                          pack_f16(v[8 * k + 4], v[8 * k + 5]), pack_f16(v[8 * k + 6], v[8 * k + 7]));
    }
    if (mirror) {
#pragma unroll
        for (uint32_t k = 0; k < 32; ++k) {        // neighbouring lanes: neighbouring elements of row 32 half + k
            uint8_t* to = turned + (32 * half + k) * 128 + ((((row % 64) / 8) ^ (k & 7)) << 4) + (row & 7) * 2;
            *reinterpret_cast<uint16_t*>(to) = (uint16_t)pack_f16(v[k], 0.0f);
        }
    }
}

// APPLY: a X of the two slabs added to the thread's 32 columns, and the next iterate left in the slabs
// (keep).
__device__ __forceinline__ void finish_apply(float a, uint8_t* hi, uint8_t* lo, uint32_t row, uint32_t half, float (&v)[32], bool keep) {
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k) {
        uint4& wh = slab_word(hi, row, 4 * half + k);
        uint4& wl = slab_word(lo, row, 4 * half + k);
        uint32_t h[4] = {wh.x, wh.y, wh.z, wh.w}, l[4] = {wl.x, wl.y, wl.z, wl.w};
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e) {
            const float2 x = join(h[e], l[e]);
            v[8 * k + 2 * e] += a * x.x;
            v[8 * k + 2 * e + 1] += a * x.y;
            part(v[8 * k + 2 * e], v[8 * k + 2 * e + 1], h[e], l[e]);
        }
        if (keep) {
            wh = make_uint4(h[0], h[1], h[2], h[3]);
            wl = make_uint4(l[0], l[1], l[2], l[3]);
        }
    }
}

// The thread's 32 columns, from column c of row r, of the result; all lanes of a warp, at neighbouring rows and
// the same columns.  Rows that are no whole 16-byte words go through the thread's words of the slab, and
// a row at a time to memory: an element of 32 rows at a time cost 1500 x 3500 65 us of 404.
__device__ __forceinline__ void store_result(const Result& o, uint32_t r, uint32_t c, uint8_t* slab, uint32_t row, uint32_t half, float (&v)[32]) {
#pragma unroll
    for (uint32_t k = 0; k < 32; ++k) v[k] *= o.scale;
    if (o.transposed) {
        if (r >= o.S) return;
#pragma unroll
        for (uint32_t k = 0; k < 32; ++k)          // neighbouring lanes hold neighbouring columns of `out`
            if (c + k < o.L)
                *reinterpret_cast<uint16_t*>(o.out + (uint64_t)(c + k) * o.pitch + (uint64_t)r * 2) = (uint16_t)pack_bf16(v[k], 0.0f);
        return;
    }
    uint4 word[4];
#pragma unroll
    for (uint32_t q = 0; q < 4; ++q)
        word[q] = make_uint4(pack_bf16(v[8 * q], v[8 * q + 1]), pack_bf16(v[8 * q + 2], v[8 * q + 3]),
                             pack_bf16(v[8 * q + 4], v[8 * q + 5]), pack_bf16(v[8 * q + 6], v[8 * q + 7]));
    if (o.vec && c + 32 <= o.L) {
        if (r >= o.S) return;
        uint4* to = reinterpret_cast<uint4*>(o.out + (uint64_t)r * o.pitch + (uint64_t)c * 2);
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q) to[q] = word[q];
        return;
    }
#pragma unroll
    for (uint32_t q = 0; q < 4; ++q) slab_word(slab, row, 4 * half + q) = word[q];
    __syncwarp();
    const uint32_t lane = threadIdx.x % 32, r0 = r - lane, row0 = row - lane;
    if (c + lane < o.L) {
#pragma unroll 8
        for (uint32_t k = 0; k < 32; ++k)
            if (r0 + k < o.S)
                *reinterpret_cast<uint16_t*>(o.out + (uint64_t)(r0 + k) * o.pitch + (uint64_t)(c + lane) * 2) =
                    reinterpret_cast<const uint16_t*>(&slab_word(slab, row0 + k, 4 * half + lane / 8))[lane % 8];
    }
    __syncwarp();
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, int32_t x, int32_t y, int32_t z, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(src) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

__device__ __forceinline__ void bar_arrive_at(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// A tile load into this CTA's shared memory that completes on the leader's mbarrier.
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z,
                                                 uint32_t cluster_bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 "
        "[%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(cluster_bar) : "memory");
}

__device__ __forceinline__ void umma_pair(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a), "l"(b), "r"(id), "r"(accumulate) : "memory");
}

// Arrive once on the mbarrier at this offset in both CTAs when the MMAs issued so far finish.
__device__ __forceinline__ void umma_commit_both(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        ::"r"(bar), "h"((uint16_t)0x3) : "memory");
}

__device__ __forceinline__ void umma_commit_local2(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// Clusters of two CTAs on two SMs, persistent: cluster c takes tiles c, c + clusters, ... of all
// matrices.  A tile is 256 rows by p.tn columns of one tcgen05.mma.cta_group::2: each CTA holds 128 of
// the rows and half of the columns.  At 256 columns an SM takes in 32 KiB for 512 cycles of MMA, about
// the 64 bytes a cycle that it can, so everything else is kept off that path as far as it goes.
//   warp 8      loads the CTA's operand halves into a ring of stages (TMA, out-of-range rows and
//               columns as zeros);
//   warp 9      one thread of the leader issues the MMAs into one of two TMEM accumulators (its
//               mbarriers count both CTAs' loads and both epilogues);
//   warps 0-7   drain the CTA's 128 rows of the other accumulator, a slab of 64 columns at a time,
//               into one of two slab buffers;
//   warp 10     fills the slab buffers with what a slab needs (two slabs ahead) and stores them, in
//               whole 128-byte lines: stored by the threads that hold the rows, a tile took 14,000
//               cycles instead of 6,000.
// 4096 x 4096, five steps in one launch: ~870 us for 1.37 TFLOP of products (half of each symmetric
// one), the tensor pipe active 75 % of the time.  Back to back the power limit takes the SM clock from 2.07
// to 1.67 GHz, and a call from 910 us to 1010.
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
ortho_pair_kernel(const __grid_constant__ PairParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = smem + STAGES * HALF_STAGE;
    uint8_t* slabs = sB + STAGES * HALF_STAGE;    // [2] x 32 KiB
    uint64_t* full = reinterpret_cast<uint64_t*>(slabs + SLAB_BUFS * 2 * SLAB_BYTES);   // [STAGES]  leader: both CTAs' loads -> MMA
    uint64_t* empty = full + STAGES;              // [STAGES]  each CTA: MMA -> its TMA warp
    uint64_t* acc_full = empty + STAGES;          // [2]       each CTA: MMA -> its epilogue
    uint64_t* acc_empty = acc_full + ACC_BUFS;    // [2]       leader: both epilogues -> MMA
    uint64_t* slab_in = acc_empty + ACC_BUFS;     // [2]       slab warp: free, and what it needs is there -> epilogue
    uint64_t* slab_out = slab_in + SLAB_BUFS;     // [2]       epilogue: to be stored -> slab warp
    uint64_t* drain = slab_out + SLAB_BUFS;       // [1]       leader: MMA teardown
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    uint2* tiles = reinterpret_cast<uint2*>(tmem_slot + 2);   // [TILES] the cluster's first: worked out by a thread each

    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32, q = cluster_rank();
    const uint32_t c0 = blockIdx.x / 2, NC = gridDim.x / 2;
    const bool leader = q == 0;
    if (threadIdx.x < TILES) tiles[threadIdx.x] = packed(pair_tile(p, c0 + threadIdx.x * NC));
    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < STAGES; ++i) {
            bar_init(saddr(full + i), 1);            // the leader's expect_tx covers both CTAs' bytes
            bar_init(saddr(empty + i), 1);
        }
        for (uint32_t i = 0; i < ACC_BUFS; ++i) {
            bar_init(saddr(acc_full + i), 1);
            bar_init(saddr(acc_empty + i), 2 * EPI_WARPS);
        }
        for (uint32_t i = 0; i < SLAB_BUFS; ++i) {
            bar_init(saddr(slab_in + i), 1);
            bar_init(saddr(slab_out + i), EPI_WARPS);
        }
        bar_init(saddr(drain), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(saddr(tmem_slot)), "r"(ACC_BUFS * 256) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    if (warp == TMA_WARP && lane == 0) {
        prefetch_map(p.first == GRAM ? &p.hi_rows[p.step & 1] : p.first == POLY ? &p.gram : &p.poly);
        if (p.first == APPLY) prefetch_map(&p.hi_cols[p.step & 1]);
    }
    tc_fence_before();
    cluster_sync_all();          // both CTAs' barriers exist before either arrives remotely
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    launch_next();
    const uint32_t places = pair_tiles(p), k_long = (p.L + BK - 1) / BK, k_short = (p.S + BK - 1) / BK;   // k blocks: GRAM; else
    auto tile_at = [&](uint32_t u) { return u < c0 + TILES * NC ? unpacked(tiles[(u - c0) / NC]) : pair_tile(p, u); };
    wait_previous();

    const uint32_t peer_abort = at_rank(saddr(tmem_slot + 1), q ^ 1);
    auto fail = [&]() {
        *abort_flag = 1;
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer_abort), "r"(1u) : "memory");
        atomicAdd(p.err, 1u);
    };

    if (warp == TMA_WARP) {
        if (lane == 0) {
            uint32_t stage = 0, phase = 0, issued = 0;
            bool ok = true;
            for (uint32_t u = c0; u < places && ok; u += NC) {
                const Tile t = tile_at(u);
                if (!inputs_ready(p, t, abort_flag)) { fail(); ok = false; break; }
                const uint32_t now = (p.step + t.k) & 1, tn = t.product == APPLY ? p.tn : 256;
                const CUtensorMap* mA = t.product == GRAM ? &p.hi_rows[now] : t.product == POLY ? &p.gram : &p.poly;
                const CUtensorMap* mB = t.product == APPLY ? &p.hi_cols[now] : mA;
                const int32_t row = (int32_t)(t.i * 256 + q * 128), col = (int32_t)(t.j * tn + q * (tn / 2)), z = (int32_t)t.m;
                const uint2 ks = k_blocks(p, t, t.product == GRAM ? k_long : k_short);
                for (uint32_t kb = ks.x; kb < ks.y; ++kb) {
                    if (!bar_wait(saddr(empty + stage), phase ^ 1, abort_flag)) { fail(); ok = false; break; }
                    // The peer's loads may land before the leader's expect_tx (the barrier's
                    // transaction count goes below zero for a while), but never a phase early: its
                    // stage is free only once the MMA has consumed that stage.
                    const uint32_t bar = at_rank(saddr(full + stage), 0);
                    const int32_t k = (int32_t)(kb * BK);
                    const uint32_t dA = saddr(sA + stage * HALF_STAGE), dB = saddr(sB + stage * HALF_STAGE);
                    if (leader) bar_expect_tx(saddr(full + stage), tn == 128 ? 3 * HALF_STAGE : 4 * HALF_STAGE);
                    tma_load_3d_pair(dA, mA, k, row, z, bar);
                    if (t.product == APPLY) {     // X: rows k, 64 columns a box
                        tma_load_3d_pair(dB, mB, col, k, z, bar);
                        if (tn > 128) tma_load_3d_pair(dB + HALF_STAGE / 2, mB, col + 64, k, z, bar);
                    } else {
                        tma_load_3d_pair(dB, mB, k, col, z, bar);
                    }
                    ++issued;
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                }
            }
            // the leader's full barriers count both CTAs' loads: once its last phases complete, every
            // load of the pair has landed
            if (leader) {
                for (uint32_t i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i)
                    (void)bar_wait(saddr(full + i % STAGES), (i / STAGES) & 1, nullptr);
            } else if (!ok) {
                // the leader may have given up before it counted this CTA's last loads: 0.2 ms for a few us of them
                for (uint32_t i = 0; i < 256; ++i) __nanosleep(1000);
            }
        }
    } else if (warp == MMA_WARP) {
        if (lane == 0 && leader) {
            uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
            bool ok = true;
            for (uint32_t u = c0; u < places && ok; u += NC) {
                const Tile t = tile_at(u);
                const uint32_t product = t.product;
                const uint32_t id = product == APPLY ? idesc(256, p.tn) | IDESC_B_MN : idesc(256, 256);
                const uint32_t step = product == APPLY ? STEP_MN : STEP_K;
                const uint2 ks = k_blocks(p, t, product == GRAM ? k_long : k_short);
                if (!bar_wait(saddr(acc_empty + acc), acc_phase ^ 1, abort_flag)) { fail(); break; }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + acc * 256;
                for (uint32_t kb = ks.x; kb < ks.y; ++kb) {
                    if (!bar_wait(saddr(full + stage), phase, abort_flag)) { fail(); ok = false; break; }
                    tc_fence_after();
                    const uint64_t da = desc_k(saddr(sA + stage * HALF_STAGE));
                    const uint32_t b0 = saddr(sB + stage * HALF_STAGE);
                    const uint64_t db = product == APPLY ? desc_mn(b0) : desc_k(b0);
#pragma unroll
                    for (uint32_t k = 0; k < BK / UMMA_K; ++k) umma_pair(d_tmem, da + STEP_K * k, db + step * k, id, kb != ks.x || k != 0);
                    umma_commit_both(saddr(empty + stage));   // both CTAs' stages are free
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                }
                if (!ok) break;
                umma_commit_both(saddr(acc_full + acc));      // the tile is in both TMEMs
                if (++acc == ACC_BUFS) { acc = 0; acc_phase ^= 1; }
            }
            // every MMA has finished before either CTA releases TMEM or shared memory
            umma_commit_local2(saddr(drain));
            (void)bar_wait(saddr(drain), 0, nullptr);
        }
    } else if (warp == SLAB_WARP) {
        if (lane == 0 && c0 < places) {
            uint32_t loaded = 0, stored_slabs = 0;
            bool ok = true;
            for (uint32_t u = c0; u < places && ok; u += NC) {
                const Tile t = tile_at(u);
                if (t.product == GRAM && t.split + 1 < p.splits) continue;    // its sums leave as they are
                const bool apply = t.product == APPLY, result = p.out && t.k + 1 == p.steps;
                const uint32_t count = (apply ? p.tn : 256) / SLAB;
                const int32_t y = (int32_t)(t.i * 256 + q * 128), m = (int32_t)t.m;
                auto column = [&](uint32_t g) { return (int32_t)(t.j * count * SLAB + g * SLAB); };
                auto inside = [&](uint32_t g) { return (uint32_t)column(g) < (apply ? p.L : p.S) && (uint32_t)y < p.S; };
                auto load = [&](uint32_t g) {
                    const uint32_t bar = saddr(slab_in + loaded % SLAB_BUFS), to = saddr(slabs) + loaded % SLAB_BUFS * 2 * SLAB_BYTES;
                    if (t.product == GRAM || !inside(g)) {
                        bar_arrive(bar);
                    } else {
                        bar_expect_tx(bar, apply ? 2 * SLAB_BYTES : SLAB_BYTES);
                        tma_load_3d(to, apply ? &p.hi_rows[(p.step + t.k) & 1] : &p.gram, column(g), y, m, bar);
                        if (apply) tma_load_3d(to + SLAB_BYTES, &p.lo_rows, column(g), y, m, bar);
                    }
                    ++loaded;
                };
                // not before the last tile has been stored and counted: this one may wait for it
                if (!inputs_ready(p, t, abort_flag)) { ok = false; break; }
                for (uint32_t g = 0; g < SLAB_BUFS; ++g) load(g);
                for (uint32_t g = 0; g < count; ++g, ++stored_slabs) {
                    if (!bar_wait(saddr(slab_out + stored_slabs % SLAB_BUFS), stored_slabs / SLAB_BUFS & 1, abort_flag)) { ok = false; break; }
                    const int32_t x = column(g);
                    const uint32_t from = saddr(slabs) + stored_slabs % SLAB_BUFS * 2 * SLAB_BYTES;
                    if (!apply) {
                        const bool gram = t.product == GRAM;
                        if (inside(g)) tma_store_3d(gram ? &p.gram : &p.poly, x, y, m, from);
                        if (t.i != t.j && (uint32_t)x < p.S)                 // as rows x .., columns y ..
                            for (int32_t h = 0; h < 2; ++h)
                                if ((uint32_t)(y + 64 * h) < p.S)
                                    tma_store_3d(gram ? &p.gram_blocks : &p.poly_blocks, y + 64 * h, x, m, from + SLAB_BYTES + h * (SLAB_BYTES / 2));
                    } else if (!result && inside(g)) {
                        tma_store_3d(&p.hi_rows[(p.step + t.k + 1) & 1], x, y, m, from);
                        tma_store_3d(&p.lo_rows, x, y, m, from + SLAB_BYTES);
                    }
                    bulk_commit();
                    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                    if (g + SLAB_BUFS < count) load(g + SLAB_BUFS);
                }
                if (ok && p.counters && !(apply && result)) count_stored(p, t);
            }
            if (!ok) fail();
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
            // every load has landed before the CTA can leave
            for (uint32_t n = loaded > SLAB_BUFS ? loaded - SLAB_BUFS : 0; n < loaded; ++n)
                (void)bar_wait(saddr(slab_in + n % SLAB_BUFS), n / SLAB_BUFS & 1, nullptr);
        }
    } else {
        // epilogue
        uint32_t acc = 0, acc_phase = 0, s = 0;
        const uint32_t row = 32 * (warp % 4) + lane, half = warp / 4;
        bool ok = true;
        for (uint32_t u = c0; u < places && ok; u += NC) {
            const Tile t = tile_at(u);
            const float a = p.coeffs[t.k][0], b = p.coeffs[t.k][1], c = p.coeffs[t.k][2];
            const bool result = p.out && t.k + 1 == p.steps;
            const uint32_t tn = t.product == APPLY ? p.tn : 256;
            ok = __all_sync(0xFFFFFFFFu, bar_wait(saddr(acc_full + acc), acc_phase, abort_flag));
            tc_fence_after();
            const uint32_t taddr = tmem_base + ((32u * (warp % 4)) << 16) + acc * 256 + 32 * half;
            const bool parted = t.product == GRAM && p.splits > 1;
            if (ok && parted) {
                if (t.split + 1 < p.splits) {
                    for (uint32_t g = 0; g < tn / SLAB; ++g) {
                        float v[32];
                        tmem_ld32(taddr + g * SLAB, v);
                        float4* to = part_of(p, t, t.split, q, warp, g);
#pragma unroll
                        for (uint32_t k = 0; k < 8; ++k) to[k * 32 + lane] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(parts_counter(p, t)) : "memory");
                        bar_arrive_at(at_rank(saddr(acc_empty + acc), 0));
                    }
                    if (++acc == ACC_BUFS) { acc = 0; acc_phase ^= 1; }
                    continue;
                }
                ok = __all_sync(0xFFFFFFFFu, lane != 0 || reached(parts_counter(p, t), (t.k + 1) * (p.splits - 1) * 2 * EPI_WARPS, abort_flag));
                __syncwarp();          // what lane 0 acquired is there for all lanes: a vote orders no memory
            }
            for (uint32_t g = 0; g < tn / SLAB && ok; ++g, ++s) {
                uint8_t* slab = slabs + s % SLAB_BUFS * 2 * SLAB_BYTES;
                float v[32];
                tmem_ld32(taddr + g * SLAB, v);
                if (parted) {
                    for (uint32_t n = 0; n + 1 < p.splits; ++n) {
                        const float4* from = part_of(p, t, n, q, warp, g);
#pragma unroll
                        for (uint32_t k = 0; k < 8; ++k) {
                            const float4 f = __ldcg(from + k * 32 + lane);
                            v[4 * k] += f.x;
                            v[4 * k + 1] += f.y;
                            v[4 * k + 2] += f.z;
                            v[4 * k + 3] += f.w;
                        }
                    }
                }
                ok = __all_sync(0xFFFFFFFFu, bar_wait(saddr(slab_in + s % SLAB_BUFS), s / SLAB_BUFS & 1, abort_flag));
                if (!ok) break;
                if (t.product == APPLY) {
                    finish_apply(a, slab, slab + SLAB_BYTES, row, half, v, !result);
                    if (result)
                        store_result({p.out + (uint64_t)t.m * p.out_stride, p.out_pitch, p.S, p.L, p.scale, p.transposed, p.out_vec},
                                     t.i * 256 + q * 128 + row, t.j * tn + g * SLAB + 32 * half, slab, row, half, v);
                } else if (t.product == GRAM) {
                    finish<false>(b, c, slab, row, half, t.i != t.j, v);
                } else {
                    finish<true>(b, c, slab, row, half, t.i != t.j, v);
                }
                // the slab warp's stores read what every lane wrote
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) bar_arrive(saddr(slab_out + s % SLAB_BUFS));
            }
            if (!ok) {
                if (lane == 0) fail();
                break;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive_at(at_rank(saddr(acc_empty + acc), 0));   // this warp's TMEM reads are done
            if (++acc == ACC_BUFS) { acc = 0; acc_phase ^= 1; }
        }
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync_all();          // no CTA leaves while the pair's MMAs or loads may touch it
    tc_fence_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(ACC_BUFS * 256) : "memory");
}

// ---- split form --------------------------------------------------------------------------------
// A copy to a CTA of the cluster that counts, in bytes, on an mbarrier of that CTA.
__device__ __forceinline__ void push(uint32_t to, uint32_t from, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(to), "r"(from), "r"(bytes), "r"(bar) : "memory");
}
// What the threads wrote to shared memory is there for copies and MMAs that start after a barrier.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Four columns from column c of output row r of matrix m, a lane's share of a tile's row: v with what the
// product adds to it (held, rest: A, or hi and lo, of the same place), stored, and kept in `turn` (or null)
// for store_turned.
template <Product P>
__device__ __forceinline__ void store_four(const GemmParams& p, uint32_t m, uint32_t r, uint32_t c, float4 v, uint2 held, uint2 rest, uint32_t* turn) {
    const uint32_t cols = P == APPLY ? p.L : p.S;
    const bool in = r < p.S && c < cols;          // rows are padded to 64 elements: then all four are the array's
    const uint64_t to = ((uint64_t)m * p.S + r) * (P == APPLY ? p.l_pitch : p.s_pitch) + c;
    if (P == POLY && in) {
        const float2 g0 = __half22float2(*reinterpret_cast<const __half2*>(&held.x)), g1 = __half22float2(*reinterpret_cast<const __half2*>(&held.y));
        v = make_float4(p.c * v.x + p.b * g0.x, p.c * v.y + p.b * g0.y, p.c * v.z + p.b * g1.x, p.c * v.w + p.b * g1.y);
    }
    if (P == APPLY && in) {
        const float2 x0 = join(held.x, rest.x), x1 = join(held.y, rest.y);
        v = make_float4(v.x + p.a * x0.x, v.y + p.a * x0.y, v.z + p.a * x1.x, v.w + p.a * x1.y);
        if (!p.out) {
            uint32_t unused;
            uint2 l;
            part(v.x, v.y, unused, l.x);
            part(v.z, v.w, unused, l.y);
            *reinterpret_cast<uint2*>(p.lo + to) = l;
        }
    }
    uint32_t e01, e23;                            // the four as stored
    if (P == APPLY && p.out) {
        e01 = pack_bf16(v.x * p.scale, v.y * p.scale);
        e23 = pack_bf16(v.z * p.scale, v.w * p.scale);
    } else {
        e01 = pack_f16(v.x, v.y);
        e23 = pack_f16(v.z, v.w);
    }
    if (turn) {
        turn[0] = in ? e01 : 0;
        turn[1] = in ? e23 : 0;
    }
    if (!in || (P == APPLY && p.out && p.transposed)) return;
    if (P == APPLY && p.out) {
        char* out = p.out + (uint64_t)m * p.out_stride + (uint64_t)r * p.out_pitch + (uint64_t)c * 2;
        if (p.out_vec && c + 4 <= p.L) {
            *reinterpret_cast<uint2*>(out) = make_uint2(e01, e23);
        } else {
            const uint32_t e[4] = {e01 & 0xFFFF, e01 >> 16, e23 & 0xFFFF, e23 >> 16};
#pragma unroll
            for (uint32_t x = 0; x < 4; ++x)
                if (c + x < p.L) reinterpret_cast<uint16_t*>(out)[x] = (uint16_t)e[x];
        }
    } else {
        *reinterpret_cast<uint2*>(p.out16 + to) = make_uint2(e01, e23);
    }
}

// `rows` rows from row r0 (of the columns c0 .. + 127) as columns: a thread a column, whose elements
// neighbour each other in row c0 + thread of the result.
template <Product P>
__device__ __forceinline__ void store_turned(const GemmParams& p, uint32_t m, uint32_t r0, uint32_t c0, uint32_t rows, const uint16_t* turn) {
    const uint32_t c = c0 + threadIdx.x;
    if (threadIdx.x >= 128 || c >= (P == APPLY ? p.L : p.S)) return;
    for (uint32_t n = 0; n < rows && r0 + n < p.S; n += 8) {
        const uint32_t r = r0 + n;
        uint32_t e[8];
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) e[k] = turn[(n + k) * T16_PITCH + threadIdx.x];
        const uint4 w = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
        if (P != APPLY) {
            *reinterpret_cast<uint4*>(p.out16 + ((uint64_t)m * p.S + c) * p.s_pitch + r) = w;
        } else {
            char* out = p.out + (uint64_t)m * p.out_stride + (uint64_t)c * p.out_pitch + (uint64_t)r * 2;
            if (p.out_vec && r + 8 <= p.S) {
                *reinterpret_cast<uint4*>(out) = w;
            } else {
#pragma unroll
                for (uint32_t k = 0; k < 8; ++k)
                    if (r + k < p.S) reinterpret_cast<uint16_t*>(out)[k] = (uint16_t)e[k];
            }
        }
    }
}

// What store_four needs for the thread's rows of a tile (rows first + warp + 8 k), fetched ahead.
template <Product P, uint32_t N>
__device__ __forceinline__ void fetch_fours(const GemmParams& p, uint32_t m, uint32_t r0, uint32_t c, uint2 (&held)[N], uint2 (&rest)[N]) {
    if (P == GRAM || threadIdx.x / 32 >= EPI_WARPS || c >= (P == APPLY ? p.L : p.S)) return;
#pragma unroll
    for (uint32_t k = 0; k < N; ++k) {
        const uint32_t r = r0 + threadIdx.x / 32 + EPI_WARPS * k;
        if (r < p.S) {
            const uint64_t at = ((uint64_t)m * p.S + r) * (P == APPLY ? p.l_pitch : p.s_pitch) + c;
            held[k] = *reinterpret_cast<const uint2*>((P == POLY ? p.gram : p.hi) + at);
            if (P == APPLY) rest[k] = *reinterpret_cast<const uint2*>(p.lo + at);
        }
    }
}

// One 128 x 128 tile a cluster, its k blocks shared out over the cluster's CTAs (CTAS: one, two, four
// or eight).  Each CTA leaves its f32 sums in its shared memory; CTA q then adds rows q 128 / CTAs .. of
// all of them, in the CTAs' order, through distributed shared memory, and stores those rows.  A of two 1024 x
// 4096: 18 us, the tensor pipe active 30 %: what an SM can load bounds it (0.36 us a k block of 32 KiB), and
// 3 us between the launch and the first MMA.
template <Product P, uint32_t CTAS>
__global__ void __launch_bounds__(THREADS, 1) ortho_split_kernel(const __grid_constant__ GemmParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = smem + STAGES * HALF_STAGE;
    // f32 sums, rows of 32 words of four columns, words swizzled by the row: the CTA's own [128] in place of
    // the stages, and [CTAS sources][128 / CTAS]
    float4* tile = reinterpret_cast<float4*>(smem);
    float4* from = reinterpret_cast<float4*>(sB + STAGES * HALF_STAGE);
    uint64_t* full = reinterpret_cast<uint64_t*>(from + 128 * 32);   // [STAGES]  TMA -> MMA
    uint64_t* empty = full + STAGES;              // [STAGES]  MMA -> TMA
    uint64_t* done = empty + STAGES;              // [1]       every MMA of the tile
    uint64_t* sums_full = done + 1;               // [1]       the other CTAs' sums
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sums_full + 1);
    volatile uint32_t* abort_flag = tmem_slot + 1;

    constexpr uint32_t rows = 128 / CTAS, SLICE = rows * 512, MAX_ROWS = rows / EPI_WARPS;
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32, q = cluster_rank();
    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < STAGES; ++i) {
            bar_init(saddr(full + i), 1);
            bar_init(saddr(empty + i), 1);
        }
        bar_init(saddr(done), 1);
        bar_init(saddr(sums_full), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        bar_expect_tx(saddr(sums_full), (CTAS - 1) * SLICE);
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tmem_slot)), "r"(128) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (warp == TMA_WARP && lane == 0) {
        prefetch_map(&p.tmA);
        prefetch_map(&p.tmB);
    }
    tc_fence_before();
    if (CTAS > 1) cluster_sync_all();             // the barriers of all CTAs exist
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    launch_next();
    wait_previous();

    uint32_t m, i, j;
    tile_of<P>(p, blockIdx.x / CTAS, m, i, j);
    const uint32_t kblocks = (p.K + BK - 1) / BK, k0 = kblocks * q / CTAS, k1 = kblocks * (q + 1) / CTAS;
    // the rows that this CTA stores: a warp a row, four columns a lane, and what they need besides the sums
    const uint32_t first = q * rows, c = j * 128 + 4 * lane;
    uint2 held[MAX_ROWS], rest[MAX_ROWS];
    fetch_fours<P>(p, m, i * 128 + first, c, held, rest);
    auto fail = [&]() {
        *abort_flag = 1;
        atomicAdd(p.err, 1u);
    };
    if (warp == TMA_WARP) {
        if (lane == 0) {
            uint32_t issued = 0;
            for (uint32_t kb = k0; kb < k1; ++kb, ++issued) {
                const uint32_t stage = issued % STAGES;
                if (!bar_wait(saddr(empty + stage), (issued / STAGES & 1) ^ 1, abort_flag)) { fail(); break; }
                const uint32_t bar = saddr(full + stage);
                const int32_t k = (int32_t)(kb * BK), row = (int32_t)(i * 128), col = (int32_t)(j * 128), z = (int32_t)m;
                const uint32_t dA = saddr(sA + stage * HALF_STAGE), dB = saddr(sB + stage * HALF_STAGE);
                bar_expect_tx(bar, 2 * HALF_STAGE);
                tma_load_3d(dA, &p.tmA, k, row, z, bar);
                if (P == APPLY) {                 // X: rows k, 64 columns a box
                    tma_load_3d(dB, &p.tmB, col, k, z, bar);
                    tma_load_3d(dB + HALF_STAGE / 2, &p.tmB, col + 64, k, z, bar);
                } else {
                    tma_load_3d(dB, &p.tmB, k, col, z, bar);
                }
            }
            // the last loads of every stage have landed before the stages are used for the tile
            for (uint32_t n = issued > STAGES ? issued - STAGES : 0; n < issued; ++n)
                (void)bar_wait(saddr(full + n % STAGES), (n / STAGES) & 1, nullptr);
        }
    } else if (warp == MMA_WARP) {
        if (lane == 0) {
            for (uint32_t n = 0; n < k1 - k0; ++n) {
                const uint32_t stage = n % STAGES;
                if (!bar_wait(saddr(full + stage), n / STAGES & 1, abort_flag)) { fail(); break; }
                tc_fence_after();
                const uint64_t da = desc_k(saddr(sA + stage * HALF_STAGE));
                const uint32_t b0 = saddr(sB + stage * HALF_STAGE);
                const uint64_t db = P == APPLY ? desc_mn(b0) : desc_k(b0);
                constexpr uint32_t id = idesc(128, 128) | (P == APPLY ? IDESC_B_MN : 0);
#pragma unroll
                for (uint32_t k = 0; k < BK / UMMA_K; ++k) umma(tmem_base, da + STEP_K * k, db + step_b<P>() * k, id, (n | k) != 0);
                umma_commit(saddr(empty + stage));     // the stage is free once these finish
            }
            umma_commit(saddr(done));
            (void)bar_wait(saddr(done), 0, nullptr);
        }
    }
    __syncwarp();
    __syncthreads();                              // the MMAs are done and no load is under way
    tc_fence_after();
    if (warp < EPI_WARPS) {                       // a lane a row, 64 columns a warp
        const uint32_t row = 32 * (warp % 4) + lane;
#pragma unroll
        for (uint32_t g = 0; g < 2; ++g) {
            float v[32];
            tmem_ld32(tmem_base + ((32 * (warp % 4)) << 16) + 64 * (warp / 4) + 32 * g, v);
#pragma unroll
            for (uint32_t w = 0; w < 8; ++w)
                tile[row * 32 + ((16 * (warp / 4) + 8 * g + w) ^ (row & 7))] = make_float4(v[4 * w], v[4 * w + 1], v[4 * w + 2], v[4 * w + 3]);
        }
    }
    fence_async();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(128) : "memory");
    if (CTAS > 1) {
        if (threadIdx.x < CTAS && threadIdx.x != q)
            push(at_rank(saddr(from) + q * SLICE, threadIdx.x), saddr(tile) + threadIdx.x * SLICE, SLICE, at_rank(saddr(sums_full), threadIdx.x));
        __syncwarp();
        // nothing cuts this short: the others send their sums whatever happens, and these must have landed
        if (warp < EPI_WARPS && !bar_wait(saddr(sums_full), 0, nullptr) && lane == 0) fail();
        __syncwarp();
        // here: every CTA has what was sent to it (the wait is at the end, before the CTA leaves)
        asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
    }

    const bool turned = P == APPLY ? p.out && p.transposed : i != j;   // the rows are stored as columns (too)
    uint16_t* turn = reinterpret_cast<uint16_t*>(smem + T16_OFFSET);
#pragma unroll
    for (uint32_t k = 0; k < MAX_ROWS; ++k) {
        const uint32_t n = warp + EPI_WARPS * k, r = i * 128 + first + n;
        if (warp >= EPI_WARPS) break;
        const uint32_t word = lane ^ ((first + n) & 7);
        float4 sums[CTAS];
#pragma unroll
        for (uint32_t o = 0; o < CTAS; ++o) sums[o] = o == q ? tile[(first + n) * 32 + word] : from[(o * rows + n) * 32 + word];
        float4 v = sums[0];
#pragma unroll
        for (uint32_t o = 1; o < CTAS; ++o) v = make_float4(v.x + sums[o].x, v.y + sums[o].y, v.z + sums[o].z, v.w + sums[o].w);
        store_four<P>(p, m, r, c, v, held[k], rest[k], turned ? reinterpret_cast<uint32_t*>(turn + n * T16_PITCH + 4 * lane) : nullptr);
    }
    __syncthreads();
    if (turned) store_turned<P>(p, m, i * 128 + first, j * 128, rows, turn);
    if (CTAS > 1) asm volatile("barrier.cluster.wait;" ::: "memory");   // its sums have been sent and received
}

// S <= 256, APPLY with its own b A + c A A: one 128 x 128 tile a CTA.  All of A (as two row blocks) and the
// tile's columns of X are loaded at once; b A + c A A of the tile's rows takes their place in A, what its
// rounding to f16 leaves the other row block's (a second term of the last product).  A launch
// of POLY costs 6 us at these sizes, working its rows out again in every CTA 3 us.  256 x 1000: 8 us, 14 us with
// cold caches; one chain of load, MMA, rounding, MMA and store, on 16 SMs.
constexpr uint32_t FUSED_SMEM = 1024 /* alignment slack */ + (8 + 4) * HALF_STAGE + 256;
static_assert(T16_OFFSET + 128 * T16_PITCH * 2 <= 8 * HALF_STAGE, "the tile fits A's place");

__global__ void __launch_bounds__(THREADS, 1) ortho_fused_kernel(const __grid_constant__ GemmParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;                           // [4 blocks of 64 k][2 blocks of 128 rows]
    uint8_t* sX = sA + 8 * HALF_STAGE;            // [4 blocks of 64 k], 128 columns
    uint64_t* a_full = reinterpret_cast<uint64_t*>(sX + 4 * HALF_STAGE);   // [4]
    uint64_t* x_full = a_full + 4;
    uint64_t* done = x_full + 1;                  // [2]       the MMAs of b A + c A A; of the tile
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 2);
    volatile uint32_t* abort_flag = tmem_slot + 1;

    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        for (uint32_t k = 0; k < 4; ++k) bar_init(saddr(a_full + k), 1);
        bar_init(saddr(x_full), 1);
        bar_init(saddr(done), 1);
        bar_init(saddr(done + 1), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tmem_slot)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (warp == TMA_WARP && lane == 0) {
        prefetch_map(&p.tmA);
        prefetch_map(&p.tmB);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t d_poly = *tmem_slot, d_tile = d_poly + 256;
    launch_next();
    wait_previous();

    uint32_t m, i, j;
    tile_of<APPLY>(p, blockIdx.x, m, i, j);
    const uint32_t kblocks = (p.S + BK - 1) / BK, wide = p.S > 128 ? 256 : 128;    // 256: both row blocks of A
    constexpr uint32_t ROWS = 128 / EPI_WARPS;
    const uint32_t c = j * 128 + 4 * lane;
    uint2 held[ROWS], rest[ROWS];
    fetch_fours<APPLY>(p, m, i * 128, c, held, rest);
    auto wait = [&](uint64_t* bar) {
        if (!bar_wait(saddr(bar), 0, abort_flag) && lane == 0) {
            *abort_flag = 1;
            atomicAdd(p.err, 1u);
        }
        __syncwarp();
    };
    if (warp == TMA_WARP) {
        if (lane == 0) {
            for (uint32_t k = 0; k < kblocks; ++k) {
                bar_expect_tx(saddr(a_full + k), wide / 128 * HALF_STAGE);
                for (uint32_t h = 0; h < wide / 128; ++h)
                    tma_load_3d(saddr(sA + (2 * k + h) * HALF_STAGE), &p.tmA, (int32_t)(k * BK), (int32_t)(h * 128), (int32_t)m, saddr(a_full + k));
            }
            bar_expect_tx(saddr(x_full), kblocks * HALF_STAGE);
            for (uint32_t k = 0; k < kblocks; ++k)
                for (uint32_t h = 0; h < 2; ++h)
                    tma_load_3d(saddr(sX + k * HALF_STAGE + h * (HALF_STAGE / 2)), &p.tmB, (int32_t)(j * 128 + 64 * h), (int32_t)(k * BK), (int32_t)m, saddr(x_full));
        }
        __syncwarp();
        // every load has landed before the CTA can leave, and before A's place is used again
        for (uint32_t k = 0; k < kblocks; ++k) (void)bar_wait(saddr(a_full + k), 0, nullptr);
        (void)bar_wait(saddr(x_full), 0, nullptr);
    } else if (warp == MMA_WARP) {
        for (uint32_t k = 0; k < kblocks; ++k) {
            wait(a_full + k);
            tc_fence_after();
            if (lane == 0)
                for (uint32_t n = 0; n < 4; ++n)
                    umma(d_poly, desc_k(saddr(sA + (2 * k + i) * HALF_STAGE)) + STEP_K * n, desc_k(saddr(sA + 2 * k * HALF_STAGE)) + STEP_K * n,
                         idesc(128, wide), (k | n) != 0);
        }
        if (lane == 0) umma_commit(saddr(done));
        __syncwarp();
    }
    if (warp < EPI_WARPS) {                       // a lane a row; a warp every other 32 columns
        wait(done);
        tc_fence_after();
        const uint32_t row = 32 * (warp % 4) + lane;
        for (uint32_t g = warp / 4; g < 2 * kblocks; g += 2) {
            float v[32];
            tmem_ld32(d_poly + ((32 * (warp % 4)) << 16) + 32 * g, v);
#pragma unroll
            for (uint32_t w = 0; w < 4; ++w) {
                uint4& word = slab_word(sA + (2 * (g / 2) + i) * HALF_STAGE, row, 4 * (g % 2) + w);
                const uint32_t old[4] = {word.x, word.y, word.z, word.w};
                uint32_t to[4], below[4];
#pragma unroll
                for (uint32_t e = 0; e < 4; ++e) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&old[e]));
                    two_terms(p.c * v[8 * w + 2 * e] + p.b * f.x, p.c * v[8 * w + 2 * e + 1] + p.b * f.y, to[e], below[e]);
                }
                word = make_uint4(to[0], to[1], to[2], to[3]);
                slab_word(sA + (2 * (g / 2) + 1 - i) * HALF_STAGE, row, 4 * (g % 2) + w) = make_uint4(below[0], below[1], below[2], below[3]);
            }
        }
        fence_async();
        tc_fence_before();
    }
    __syncthreads();
    if (warp == MMA_WARP) {
        wait(x_full);
        tc_fence_after();
        if (lane == 0) {
            for (uint32_t k = 0; k < 4 * kblocks; ++k)
                for (uint32_t n = 0; n < 2; ++n)
                    umma(d_tile, desc_k(saddr(sA + (2 * (k / 4) + (n ? 1 - i : i)) * HALF_STAGE)) + STEP_K * (k % 4),
                         desc_mn(saddr(sX + k / 4 * HALF_STAGE)) + STEP_MN * (k % 4), idesc(128, 128) | IDESC_B_MN, (k | n) != 0);
            umma_commit(saddr(done + 1));
        }
        __syncwarp();
    }
    // all: the MMAs, which were issued whatever had been given up, are done, and A's place is free
    if (!bar_wait(saddr(done + 1), 0, nullptr) && lane == 0) atomicAdd(p.err, 1u);
    __syncwarp();
    tc_fence_after();
    float4* tile = reinterpret_cast<float4*>(smem);
    if (warp < EPI_WARPS) {
        const uint32_t row = 32 * (warp % 4) + lane;
#pragma unroll
        for (uint32_t g = 0; g < 2; ++g) {
            float v[32];
            tmem_ld32(d_tile + ((32 * (warp % 4)) << 16) + 64 * (warp / 4) + 32 * g, v);
#pragma unroll
            for (uint32_t w = 0; w < 8; ++w)
                tile[row * 32 + ((16 * (warp / 4) + 8 * g + w) ^ (row & 7))] = make_float4(v[4 * w], v[4 * w + 1], v[4 * w + 2], v[4 * w + 3]);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(d_poly), "r"(512) : "memory");
    const bool turned = p.out && p.transposed;
    uint16_t* turn = reinterpret_cast<uint16_t*>(smem + T16_OFFSET);
    if (warp < EPI_WARPS) {
#pragma unroll
        for (uint32_t k = 0; k < ROWS; ++k) {
            const uint32_t n = warp + EPI_WARPS * k;
            store_four<APPLY>(p, m, i * 128 + n, c, tile[n * 32 + (lane ^ (n & 7))], held[k], rest[k],
                              turned ? reinterpret_cast<uint32_t*>(turn + n * T16_PITCH + 4 * lane) : nullptr);
        }
    }
    __syncthreads();
    if (turned) store_turned<APPLY>(p, m, i * 128, j * 128, 128, turn);
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
    uint32_t* counters;          // the pair form's, zeroed here; or null
    uint32_t n_counters;
    __half* hi;
    __half* lo;
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

// Chunk i of 8 columns of a matrix: row r, columns c .., of the momentum (MOM) and of x (bf16 where B16, else f32),
// where it is wanted.  One of a thread's at a time, and many CTAs: 4096 x 4096 in bf16, one step, takes 204 us so,
// 209 with four under way in half as many CTAs.
template <bool B16, bool MOM>
__device__ __forceinline__ void chunk(const UpdateParams& p, const char* x, const char* mom, bool want_x, uint32_t i, uint32_t& r,
                                      uint32_t& c, float (&u)[8], float (&v)[8]) {
    const uint32_t per_row = p.cols / 8;
    r = i / per_row;
    c = 8 * (i - r * per_row);
    Raw8 xs{}, moms{};
    if (want_x) xs = raw8(x + r * p.x_pitch + (uint64_t)c * (B16 ? 2 : 4), B16 ? DTT_BF16 : DTT_F32);
    if (MOM) moms = raw8(mom + r * p.mom_pitch + (uint64_t)c * 4, DTT_F32);
    expand8(xs, B16 ? DTT_BF16 : DTT_F32, u);
    if (MOM) expand8(moms, DTT_F32, v);
}

__device__ __forceinline__ void zero_counters(const UpdateParams& p) {
    if (p.counters && blockIdx.x == 0 && blockIdx.y == 0)
        for (uint32_t i = threadIdx.x; i < p.n_counters; i += 256) p.counters[i] = 0;
}

// The momentum's update, and a part of |u|^2 from each of `parts` CTAs a matrix, which stride over its
// chunks: 16-byte aligned.
template <bool B16, bool MOM>
__global__ void __launch_bounds__(256, START_CTAS) ortho_update_kernel(const __grid_constant__ UpdateParams p) {
    __shared__ float slot[8];
    const uint32_t m = blockIdx.y, total = p.rows * (p.cols / 8), step = p.parts * 256;
    const char* x = p.x + (uint64_t)m * p.x_stride;
    char* mom = MOM ? p.mom + (uint64_t)m * p.mom_stride : nullptr;
    float sum = 0.0f;
    launch_next();
    zero_counters(p);
    for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < total; i += step) {
        float u[8], v[8];
        uint32_t r, c;
        chunk<B16, MOM>(p, x, mom, true, i, r, c, u, v);
        if (MOM) {
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k) {
                v[k] = p.mu * v[k] + u[k];
                u[k] = p.nesterov ? u[k] + p.mu * v[k] : v[k];
            }
            float4* to = reinterpret_cast<float4*>(mom + r * p.mom_pitch + (uint64_t)c * 4);
            to[0] = make_float4(v[0], v[1], v[2], v[3]);
            to[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) sum += u[k] * u[k];
    }
    sum = cta_sum(sum, slot);
    if (threadIdx.x == 0) p.sums[(uint64_t)m * p.parts + blockIdx.x] = sum;
}

// The same for any alignment, an element a lane: a warp has 256 columns of a row under way.
__global__ void __launch_bounds__(256, START_CTAS / 2) ortho_update_elements_kernel(const __grid_constant__ UpdateParams p) {
    __shared__ float slot[8];
    constexpr uint32_t N = 8;
    const uint32_t m = blockIdx.y, lane = threadIdx.x % 32, pieces = (p.cols + 32 * N - 1) / (32 * N), total = p.rows * pieces;   // 2^24 at most
    const char* x = p.x + (uint64_t)m * p.x_stride;
    char* mom = p.mom ? p.mom + (uint64_t)m * p.mom_stride : nullptr;
    float sum = 0.0f;
    launch_next();
    zero_counters(p);
    for (uint32_t i = blockIdx.x * 8 + threadIdx.x / 32; i < total; i += p.parts * 8) {
        const uint32_t r = i / pieces, c = 32 * N * (i - r * pieces) + lane;
        float u[N], v[N];
        const char *xs[N], *moms[N];
        uint32_t cs[N];
#pragma unroll
        for (uint32_t n = 0; n < N; ++n) {
            cs[n] = min(c + 32 * n, p.cols - 1);
            xs[n] = x + r * p.x_pitch;
            moms[n] = mom + r * p.mom_pitch;
        }
        gather(xs, p.x_dt, cs, u);
        if (mom) gather(moms, DTT_F32, cs, v);
#pragma unroll
        for (uint32_t n = 0; n < N; ++n) {
            if (c + 32 * n >= p.cols) break;
            if (mom) {
                v[n] = p.mu * v[n] + u[n];
                u[n] = p.nesterov ? u[n] + p.mu * v[n] : v[n];
                store1(mom + r * p.mom_pitch, DTT_F32, cs[n], v[n]);
            }
            sum += u[n] * u[n];
        }
    }
    sum = cta_sum(sum, slot);
    if (threadIdx.x == 0) p.sums[(uint64_t)m * p.parts + blockIdx.x] = sum;
}

// 1 / (|u| + eps) of matrix m, from its parts; 0 where that overflows (u is then 0 in f16 as well).
__device__ __forceinline__ float inverse_norm(const UpdateParams& p, uint32_t m, float (&slot)[8]) {
    float sum = 0.0f;
    launch_next();
    wait_previous();
#pragma unroll 4
    for (uint32_t i = threadIdx.x; i < p.parts; i += 256) sum += p.sums[(uint64_t)m * p.parts + i];
    const float inv = 1.0f / (sqrtf(cta_sum(sum, slot)) + p.eps);
    return isinf(inv) ? 0.0f : inv;
}

// u again (the momentum is updated by now) and X = u / (|u| + eps), in its two halves: rows
// <= cols, 16-byte aligned.  4096 x 4096 in bf16: 16 us behind the update (10 us), 33 MB read from L2 and 67
// written.
template <bool B16, bool MOM>
__global__ void __launch_bounds__(256, START_CTAS) ortho_start_kernel(const __grid_constant__ UpdateParams p) {
    __shared__ float slot[8];
    const uint32_t m = blockIdx.y, total = p.rows * (p.cols / 8), step = gridDim.x * 256;
    const char* x = p.x + (uint64_t)m * p.x_stride;
    const char* mom = MOM ? p.mom + (uint64_t)m * p.mom_stride : nullptr;
    __half* hi = p.hi + (uint64_t)m * p.S * p.l_pitch;
    __half* lo = p.lo + (uint64_t)m * p.S * p.l_pitch;
    const float inv = inverse_norm(p, m, slot);
    for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < total; i += step) {
        float u[8], v[8];
        uint32_t r, c;
        chunk<B16, MOM>(p, x, mom, !MOM || p.nesterov, i, r, c, u, v);
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) {
            if (MOM) u[k] = p.nesterov ? u[k] + p.mu * v[k] : v[k];
            u[k] *= inv;
        }
        uint4 a, b;
        part(u[0], u[1], a.x, b.x);
        part(u[2], u[3], a.y, b.y);
        part(u[4], u[5], a.z, b.z);
        part(u[6], u[7], a.w, b.w);
        *reinterpret_cast<uint4*>(hi + r * p.l_pitch + c) = a;
        *reinterpret_cast<uint4*>(lo + r * p.l_pitch + c) = b;
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
    constexpr uint32_t N = kStartTile / 4;             // elements a thread: rows warp + 8 (n / 2), columns lane + 32 (n % 2)
    float u[N], v[N];
    const char *xs[N], *moms[N];
    uint32_t cs[N];
    wait_previous();
#pragma unroll
    for (uint32_t n = 0; n < N; ++n) {
        const uint32_t r = min(r0 + warp + 8 * (n / 2), p.rows - 1);
        cs[n] = min(c0 + lane + 32 * (n % 2), p.cols - 1);
        xs[n] = x + r * p.x_pitch;
        moms[n] = mom + r * p.mom_pitch;
    }
    if (!mom || p.nesterov) gather(xs, p.x_dt, cs, u);
    if (mom) {
        gather(moms, DTT_F32, cs, v);
#pragma unroll
        for (uint32_t n = 0; n < N; ++n) u[n] = p.nesterov ? u[n] + p.mu * v[n] : v[n];
    }
    const float inv = inverse_norm(p, m, slot);
    __half* hi = p.hi + (uint64_t)m * p.S * p.l_pitch;
    __half* lo = p.lo + (uint64_t)m * p.S * p.l_pitch;
    if (TALL) {
#pragma unroll
        for (uint32_t k = 0; k < kStartTile / 8; ++k)
#pragma unroll
            for (uint32_t h = 0; h < 2; ++h) tile[warp + 8 * k][lane + 32 * h] = u[2 * k + h];
        __syncthreads();
    }
#pragma unroll
    for (uint32_t k = 0; k < kStartTile / 8; ++k)
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
            const uint32_t a = warp + 8 * k, b = lane + 32 * h;      // TALL: column a, row b of the tile
            const uint32_t r = r0 + (TALL ? b : a), c = c0 + (TALL ? a : b);
            if (r < p.rows && c < p.cols) {
                const float v = (TALL ? tile[b][a] : u[2 * k + h]) * inv;
                const uint64_t at = TALL ? c * p.l_pitch + r : r * p.l_pitch + c;
                uint32_t a, b;
                part(v, 0.0f, a, b);
                reinterpret_cast<uint16_t*>(hi)[at] = (uint16_t)a;
                reinterpret_cast<uint16_t*>(lo)[at] = (uint16_t)b;
            }
        }
}

// ---- resident form -----------------------------------------------------------------------------
constexpr uint32_t RES_THREADS = 256;
constexpr uint32_t RES_BLOCKS = 4;                   // blocks of 64 columns a CTA, at most
constexpr uint32_t RES_CTAS = 16;                    // of a cluster, at most
constexpr uint32_t BLOCK_BYTES = 128 * 64 * 2;       // 128 rows by 64 columns of f16
// hi; two blocks of A (later b A + c A A); the CTA's own f32 sums; and the sums of its rows from all CTAs
constexpr uint32_t RES_SUMS = 128 * 128 * 4;
constexpr uint32_t RES_SMEM = 1024 /* alignment slack */ + (RES_BLOCKS + 2) * BLOCK_BYTES + 2 * RES_SUMS + 128;
struct ResidentParams {
    UpdateParams u;
    Result out;                  // of matrix 0
    uint64_t out_stride;
    uint32_t blocks;             // of a CTA
    uint32_t vec;                // the update and the momentum: rows of 16-byte words, whole chunks of 8 columns
    uint32_t steps;
    uint32_t* err;
    float coeffs[DTT_ORTHO_MAX_STEPS][3];
};

// 16 words of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
          "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]) : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ float load_peer1(uint32_t cluster_addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
    return v;
}

// S <= 128: one cluster of CTAS a matrix, from the update to the result: hi stays in shared memory, lo in
// TMEM.  CTA q holds columns 64 blocks q .. of X; a block of 64 columns by 128 rows serves as it lies
// as the K-contiguous operand of A = X X^T and as the N-contiguous one of (b A + c A A) X.  Only A
// crosses CTAs: each sends its f32 sums of rows 128 / CTAS o .. to CTA o, which adds them in the CTAs'
// order and sends the rows of A, in f16, to all; every CTA then works out b A + c A A for itself, in A's
// place.  The two exchanges (bulk copies; stores by the threads took twice as long) are their own
// hand-shake: a CTA's sums of the next step leave after it has used b A + c A A, its rows of A after
// it has read the sums, and nobody goes on without all of either.  One launch, and nothing but the
// update and the result in memory: a product's 5 us as a launch of its own are mostly set-up here.  128 x 4096
// takes 58 us for five steps, 128 x 128 25: the exchanges' and MMAs' latencies one after the other (tensor pipe
// 12 % of an SM's time).
template <uint32_t CTAS>
__global__ void __launch_bounds__(RES_THREADS, 1) ortho_resident_kernel(const __grid_constant__ ResidentParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* hi = smem;
    uint8_t* gram = hi + RES_BLOCKS * BLOCK_BYTES;
    // rows of 32 words of four columns, words swizzled by the row: the CTA's own [128], and
    // [CTAS sources][128 / CTAS]
    float4* own = reinterpret_cast<float4*>(gram + 2 * BLOCK_BYTES);
    float4* sums = own + RES_SUMS / 16;
    uint8_t* poly_rest = reinterpret_cast<uint8_t*>(own);   // two blocks, once the sums have been sent
    uint64_t* done = reinterpret_cast<uint64_t*>(sums + RES_SUMS / 16);
    uint64_t* sums_full = done + 1;
    uint64_t* gram_full = done + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 3);
    float* norm_part = reinterpret_cast<float*>(tmem_slot + 1);
    __shared__ float slot[8];

    const uint32_t t = threadIdx.x, warp = t / 32, lane = t % 32, q = CTAS > 1 ? cluster_rank() : 0, m = blockIdx.x / CTAS;
    const uint32_t S = p.u.S, L = p.out.L, width = p.blocks * 64, l0 = q * width;
    const bool tall = p.out.transposed;
    if (t == 0) {
        bar_init(saddr(done), 1);
        bar_init(saddr(sums_full), 1);
        bar_init(saddr(gram_full), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tmem_slot)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }

    launch_next();
    wait_previous();
    // the update (and the momentum) in f32 over the two arrays of sums, 16-byte words swizzled by the
    // row; zeros beyond S and L.  Loads go out together before any is stored.
    const char* x = p.u.x + (uint64_t)m * p.u.x_stride;
    char* mom = p.u.mom ? p.u.mom + (uint64_t)m * p.u.mom_stride : nullptr;
    auto staged = [&](uint32_t s, uint32_t l) -> float4& {
        return own[l / 64 * (128 * 16) + s * 16 + ((l % 64 / 4) ^ ((s ^ s / 8) & 15))];
    };
    float sum = 0.0f;
    if (p.vec) {                                      // 16-byte aligned: 8 columns of the update a thread
        constexpr uint32_t N = 4;
        const uint32_t per_row = (tall ? 128 : width) / 8;
        for (uint32_t e0 = t; e0 < 16 * width; e0 += N * RES_THREADS) {     // 16 width: a multiple of N RES_THREADS
            float u[N][8], v[N][8];
            Raw8 xs[N], moms[N];
            uint32_t inside = 0;
#pragma unroll
            for (uint32_t n = 0; n < N; ++n) {
                const uint32_t e = e0 + n * RES_THREADS, r = e / per_row, c = 8 * (e - r * per_row);
                const uint32_t gr = tall ? l0 + r : r, gc = tall ? c : l0 + c;
                const bool in = gr < p.u.rows && gc < p.u.cols;
                const uint64_t fr = in ? gr : 0, fc = in ? gc : 0;
                inside |= (uint32_t)in << n;
                xs[n] = raw8(x + fr * p.u.x_pitch + fc * (p.u.x_dt == DTT_BF16 ? 2 : 4), p.u.x_dt);
                if (mom) moms[n] = raw8(mom + fr * p.u.mom_pitch + fc * 4, DTT_F32);
            }
#pragma unroll
            for (uint32_t n = 0; n < N; ++n) {
                expand8(xs[n], p.u.x_dt, u[n]);
                if (mom) expand8(moms[n], DTT_F32, v[n]);
#pragma unroll
                for (uint32_t k = 0; k < 8; ++k)
                    if (!(inside >> n & 1)) u[n][k] = v[n][k] = 0.0f;
            }
#pragma unroll
            for (uint32_t n = 0; n < N; ++n) {
                const uint32_t e = e0 + n * RES_THREADS, r = e / per_row, c = 8 * (e - r * per_row);
                const uint32_t gr = tall ? l0 + r : r, gc = tall ? c : l0 + c;
                if (mom) {
#pragma unroll
                    for (uint32_t k = 0; k < 8; ++k) {
                        v[n][k] = p.u.mu * v[n][k] + u[n][k];
                        u[n][k] = p.u.nesterov ? u[n][k] + p.u.mu * v[n][k] : v[n][k];
                    }
                    if (gr < p.u.rows && gc < p.u.cols) store8<true>(mom + gr * p.u.mom_pitch, DTT_F32, gc, p.u.cols, v[n]);
                }
#pragma unroll
                for (uint32_t k = 0; k < 8; ++k) sum += u[n][k] * u[n][k];
                if (tall) {
#pragma unroll
                    for (uint32_t k = 0; k < 8; ++k) reinterpret_cast<float*>(&staged(c + k, r))[r % 4] = u[n][k];
                } else {
                    staged(r, c) = make_float4(u[n][0], u[n][1], u[n][2], u[n][3]);
                    staged(r, c + 4) = make_float4(u[n][4], u[n][5], u[n][6], u[n][7]);
                }
            }
        }
    } else {                                          // an element a lane: 32 columns of a row of the update a warp
        constexpr uint32_t N = 16;
        const uint32_t per_row = (tall ? 128 : width) / 32, total = 4 * width;     // a multiple of 8 N / 4
        for (uint32_t e0 = warp; e0 < total; e0 += N * (RES_THREADS / 32)) {
            float u[N], v[N];
            const char *xs[N], *moms[N];
            uint32_t cs[N], inside = 0;
#pragma unroll
            for (uint32_t n = 0; n < N; ++n) {
                const uint32_t e = e0 + n * (RES_THREADS / 32), r = e / per_row, c = 32 * (e - r * per_row) + lane;
                const uint32_t gr = tall ? l0 + r : r, gc = tall ? c : l0 + c;
                const bool in = e < total && gr < p.u.rows && gc < p.u.cols;
                inside |= (uint32_t)in << n;
                cs[n] = in ? gc : 0;
                xs[n] = x + (in ? gr : 0) * p.u.x_pitch;
                moms[n] = mom + (in ? gr : 0) * p.u.mom_pitch;
                v[n] = 0.0f;
            }
            gather(xs, p.u.x_dt, cs, u);
            if (mom) gather(moms, DTT_F32, cs, v);
#pragma unroll
            for (uint32_t n = 0; n < N; ++n)
                if (!(inside >> n & 1)) u[n] = v[n] = 0.0f;
#pragma unroll
            for (uint32_t n = 0; n < N; ++n) {
                const uint32_t e = e0 + n * (RES_THREADS / 32), r = e / per_row, c = 32 * (e - r * per_row) + lane;
                const uint32_t gr = tall ? l0 + r : r, gc = tall ? c : l0 + c, s = tall ? c : r, l = tall ? r : c;
                if (e >= total) break;
                if (mom) {
                    v[n] = p.u.mu * v[n] + u[n];
                    u[n] = p.u.nesterov ? u[n] + p.u.mu * v[n] : v[n];
                    if (gr < p.u.rows && gc < p.u.cols) store1(mom + gr * p.u.mom_pitch, DTT_F32, gc, v[n]);
                }
                sum += u[n] * u[n];
                reinterpret_cast<float*>(&staged(s, l))[l % 4] = u[n];
            }
        }
    }
    sum = cta_sum(sum, slot);
    if (CTAS > 1) {
        if (t == 0) *norm_part = sum;
        cluster_sync_all();
        sum = 0.0f;
#pragma unroll
        for (uint32_t o = 0; o < CTAS; ++o) sum += load_peer1(at_rank(saddr(norm_part), o));
    }
    float inv = 1.0f / (sqrtf(sum) + p.u.eps);
    if (isinf(inv)) inv = 0.0f;                       // u is then 0 in f16 as well
    const uint32_t row = 32 * (warp % 4) + lane, half = warp / 4;
    uint32_t phase = 0;
    // A thread that has given up a wait waits no more, and starts nothing that others count on, so that they give
    // up in their turn; thread 0, which starts the MMAs and arms the barriers of what comes in, waits in
    // the end for what it started last.
    bool ok = true;
    volatile uint32_t not_cut_short = 0;
    uint32_t started = 0, armed = 0;                  // products, of thread 0; steps whose sums and rows of A it awaits
    auto await = [&](uint64_t* bar, uint32_t parity) {
        if (ok && !bar_wait(saddr(bar), parity, &not_cut_short)) {
            ok = false;
            atomicAdd(p.err, 1u);
        }
        __syncwarp();
    };
    // what the threads wrote is there for the MMAs that `issue` starts; all threads wait for these
    auto product = [&](auto issue) {
        fence_async();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (t == 0 && ok) {
            issue();
            umma_commit(saddr(done));
            ++started;
        }
        __syncwarp();
        await(done, phase);
        phase ^= 1;
        tc_fence_after();
    };
    tc_fence_before();
    __syncthreads();                                  // the update is staged, the allocation's address there
    tc_fence_after();
    const uint32_t tmem = *tmem_slot, d_square = tmem, d_apply = tmem + 128;
    const uint32_t lanes = (32u * (warp % 4)) << 16, lo = tmem + 384 + lanes + 16 * half;   // 32 words a block
    for (uint32_t n = 0; n < p.blocks; ++n) {         // X = inv u: 32 columns of a row a thread, as ever after
        uint32_t rest[16];
#pragma unroll
        for (uint32_t w = 0; w < 4; ++w) {
            const float4 u = staged(row, 64 * n + 32 * half + 8 * w), v = staged(row, 64 * n + 32 * half + 8 * w + 4);
            uint4 h;
            part(u.x * inv, u.y * inv, h.x, rest[4 * w]);
            part(u.z * inv, u.w * inv, h.y, rest[4 * w + 1]);
            part(v.x * inv, v.y * inv, h.z, rest[4 * w + 2]);
            part(v.z * inv, v.w * inv, h.w, rest[4 * w + 3]);
            slab_word(hi + n * BLOCK_BYTES, row, 4 * half + w) = h;
        }
        tmem_st16(lo + 32 * n, rest);
    }
    if (CTAS > 1) cluster_sync_all();                 // the update has been read: sums may come in its place

    for (uint32_t k = 0; k < p.steps; ++k) {
        const float a = p.coeffs[k][0], b = p.coeffs[k][1], c = p.coeffs[k][2];
        product([&] {
            for (uint32_t n = 0; n < 4 * p.blocks; ++n) {
                const uint64_t d = desc_k(saddr(hi + n / 4 * BLOCK_BYTES)) + STEP_K * (n % 4);
                umma(d_square, d, d, idesc(128, 128), n != 0);
            }
        });
        if (CTAS == 1) {
#pragma unroll
            for (uint32_t g = 0; g < 2; ++g) {        // columns 64 half + 32 g ..
                float v[32];
                tmem_ld32(d_square + lanes + 64 * half + 32 * g, v);
#pragma unroll
                for (uint32_t w = 0; w < 4; ++w)
                    slab_word(gram + half * BLOCK_BYTES, row, 4 * g + w) =
                        make_uint4(pack_f16(v[8 * w], v[8 * w + 1]), pack_f16(v[8 * w + 2], v[8 * w + 3]),
                                   pack_f16(v[8 * w + 4], v[8 * w + 5]), pack_f16(v[8 * w + 6], v[8 * w + 7]));
            }
        } else {
            constexpr uint32_t ROWS = 128 / CTAS, SLICE = ROWS * 512, A_SLICE = ROWS * 128;
#pragma unroll
            for (uint32_t g = 0; g < 2; ++g) {
                float v[32];
                tmem_ld32(d_square + lanes + 64 * half + 32 * g, v);
#pragma unroll
                for (uint32_t w = 0; w < 8; ++w)
                    own[row * 32 + ((16 * half + 8 * g + w) ^ (row & 7))] = make_float4(v[4 * w], v[4 * w + 1], v[4 * w + 2], v[4 * w + 3]);
            }
            fence_async();
            __syncthreads();
            if (t == 0 && ok) {
                bar_expect_tx(saddr(sums_full), (CTAS - 1) * SLICE);
                bar_expect_tx(saddr(gram_full), (CTAS - 1) * 2 * A_SLICE);
                ++armed;
            }
            if (t < CTAS && t != q && ok)
                push(at_rank(saddr(sums) + q * SLICE, t), saddr(own) + t * SLICE, SLICE, at_rank(saddr(sums_full), t));
            await(sums_full, k & 1);
            // the CTA's rows of A, a word of four columns at a time; to be sent from the place of its own
            // slice, which nobody sends it
            constexpr uint32_t EACH = ROWS * 32 / RES_THREADS;
            uint8_t* made = reinterpret_cast<uint8_t*>(sums) + q * SLICE;
#pragma unroll
            for (uint32_t n = 0; n < EACH; ++n) {
                const uint32_t word = n * RES_THREADS + t, r = q * ROWS + word / 32, w = word % 32, at = w ^ (r & 7);
                float4 from[CTAS];
#pragma unroll
                for (uint32_t o = 0; o < CTAS; ++o) from[o] = o == q ? own[r * 32 + at] : sums[(o * ROWS + word / 32) * 32 + at];
                float4 v = from[0];
#pragma unroll
                for (uint32_t o = 1; o < CTAS; ++o) v = make_float4(v.x + from[o].x, v.y + from[o].y, v.z + from[o].z, v.w + from[o].w);
                const uint2 a16 = make_uint2(pack_f16(v.x, v.y), pack_f16(v.z, v.w));
                const uint32_t in_block = r * 128 + ((w % 16 / 2 ^ (r & 7)) << 4) + w % 2 * 8;
                *reinterpret_cast<uint2*>(gram + w / 16 * BLOCK_BYTES + in_block) = a16;
                *reinterpret_cast<uint2*>(made + w / 16 * A_SLICE + in_block - q * A_SLICE) = a16;
            }
            fence_async();
            __syncthreads();
            if (t < 2 * CTAS && t / 2 != q && ok)
                push(at_rank(saddr(gram) + t % 2 * BLOCK_BYTES + q * A_SLICE, t / 2), saddr(made) + t % 2 * A_SLICE, A_SLICE,
                     at_rank(saddr(gram_full), t / 2));
            await(gram_full, k & 1);
        }
        product([&] {
            for (uint32_t n = 0; n < 8; ++n) {
                const uint64_t d = desc_k(saddr(gram + n / 4 * BLOCK_BYTES)) + STEP_K * (n % 4);
                umma(d_square, d, d, idesc(128, 128), n != 0);
            }
        });
#pragma unroll
        for (uint32_t g = 0; g < 2; ++g) {
            float v[32];
            tmem_ld32(d_square + lanes + 64 * half + 32 * g, v);
#pragma unroll
            for (uint32_t w = 0; w < 4; ++w) {
                uint4& word = slab_word(gram + half * BLOCK_BYTES, row, 4 * g + w);
                const uint32_t from[4] = {word.x, word.y, word.z, word.w};
                uint32_t to[4], rest[4];
#pragma unroll
                for (uint32_t e = 0; e < 4; ++e) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&from[e]));
                    two_terms(c * v[8 * w + 2 * e] + b * f.x, c * v[8 * w + 2 * e + 1] + b * f.y, to[e], rest[e]);
                }
                word = make_uint4(to[0], to[1], to[2], to[3]);
                slab_word(poly_rest + half * BLOCK_BYTES, row, 4 * g + w) = make_uint4(rest[0], rest[1], rest[2], rest[3]);
            }
        }
        // b A + c A A in two f16 terms: the second costs a few MMAs here and takes a third off the error
        product([&] {
            for (uint32_t n = 0; n < 16; ++n)
                umma(d_apply, desc_k(saddr((n < 8 ? gram : poly_rest) + n % 8 / 4 * BLOCK_BYTES)) + STEP_K * (n % 4),
                     desc_of(saddr(hi), BLOCK_BYTES, 1024) + STEP_MN * (n % 8), idesc(128, width) | IDESC_B_MN, n != 0);
        });
        const bool last = k + 1 == p.steps;
        for (uint32_t n = 0; n < p.blocks; ++n) {
            float v[32];
            uint32_t rest[16];
            tmem_ld32(d_apply + lanes + 64 * n + 32 * half, v);
            tmem_ld16(lo + 32 * n, rest);
#pragma unroll
            for (uint32_t w = 0; w < 4; ++w) {
                uint4& word = slab_word(hi + n * BLOCK_BYTES, row, 4 * half + w);
                uint32_t h[4] = {word.x, word.y, word.z, word.w};
#pragma unroll
                for (uint32_t e = 0; e < 4; ++e) {
                    const float2 from = join(h[e], rest[4 * w + e]);
                    v[8 * w + 2 * e] += a * from.x;
                    v[8 * w + 2 * e + 1] += a * from.y;
                    part(v[8 * w + 2 * e], v[8 * w + 2 * e + 1], h[e], rest[4 * w + e]);
                }
                word = make_uint4(h[0], h[1], h[2], h[3]);
            }
            if (!last) tmem_st16(lo + 32 * n, rest);
            if (last) {
                Result out = p.out;
                out.out += (uint64_t)m * p.out_stride;
                store_result(out, row, l0 + 64 * n + 32 * half, hi + n * BLOCK_BYTES, row, half, v);
            }
        }
    }
    if (t == 0 && !ok) {
        if (started) (void)bar_wait(saddr(done), (started - 1) & 1, nullptr);
        if (armed) (void)bar_wait(saddr(sums_full), (armed - 1) & 1, nullptr);
        if (armed) (void)bar_wait(saddr(gram_full), (armed - 1) & 1, nullptr);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    if (CTAS > 1) cluster_sync_all();                 // no CTA leaves while a peer may still send to it
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
    uint64_t hi[2], lo, gram, poly, sums, counters, bytes;   // byte offsets in the workspace
    uint64_t n_counters, parts;
    uint32_t splits;             // of A, where all products run in one launch
};

// Time of one of A's tiles as `splits` parts, where all products run in one launch: 0.275 us a k block, and each
// part's sums through L2, ~1 us apart and 3 us in all besides.
double gram_us(uint64_t L, uint32_t splits) {
    const uint64_t kblocks = (L + BK - 1) / BK;
    return 0.3 + 0.275 * (double)((kblocks + splits - 1) / splits) + (splits > 1 ? 3.0 + splits : 0.0);
}

// How many parts: few tiles of long rows then occupy more of the SMs' pairs.  Measured, by one part and by these: 512 x
// 8192, four of them 428 us and 335, 2048 x 8192 606 and 544, 700 x 4000, four, 291 and 271; 1024 x 1024
// would lose by two, 181 and 190.
uint32_t splits_of(uint64_t S, uint64_t L, uint32_t batch) {
    const uint64_t n = (S + 255) / 256, tiles = n * (n + 1) / 2 * batch, kblocks = (L + BK - 1) / BK;
    uint32_t best = 1;
    for (uint32_t splits = 2; splits <= 4 && tiles * splits <= kSms / 2 && kblocks >= 8 * splits; ++splits)
        if (gram_us(L, splits) < gram_us(L, best)) best = splits;
    const uint64_t each = (kblocks + best - 1) / best;
    return (uint32_t)((kblocks + each - 1) / each);
}

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
    l.hi[0] = take(d.batch * l.S * l.l_pitch * 2);
    l.hi[1] = take(d.batch * l.S * l.l_pitch * 2);
    l.lo = take(d.batch * l.S * l.l_pitch * 2);
    l.gram = take(d.batch * l.S * l.s_pitch * 2);
    l.poly = take(d.batch * l.S * l.s_pitch * 2);
    l.sums = take((uint64_t)d.batch * kMaxParts * 4);
    const uint64_t n = (l.S + 255) / 256, tiles = d.batch * n * (n + 1) / 2;
    l.n_counters = d.batch * 3 * n + tiles;
    l.counters = take(l.n_counters * 4);
    l.splits = l.S > 256 ? splits_of(l.S, l.L, d.batch) : 1;
    l.parts = take(tiles * (l.splits - 1) * 65536 * 4);
    l.bytes = at;
    return l;
}

int check_desc(const char* who, const dtt_ortho_desc* d) {
    if (!d) return fail(DTT_EINVAL, "%s: null desc", who);
    if (d->x_dtype != DTT_BF16 && d->x_dtype != DTT_F32) return fail(DTT_EINVAL, "%s: x is bf16 or f32", who);
    if (d->rows == 0 || d->cols == 0 || d->rows > 65536 || d->cols > 65536)
        return fail(DTT_EINVAL, "%s: rows and cols must be 1 .. 65536", who);
    if (d->batch == 0 || d->batch > 65535) return fail(DTT_EINVAL, "%s: batch must be 1 .. 65535", who);
    if (((d->rows + 127) / 128) * ((d->cols + 127) / 128) * d->batch >= (1ull << 28))
        return fail(DTT_EINVAL, "%s: 2^28 tiles of 128 x 128 or more", who);
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

// Clusters that can be resident at once: pairs, and splits of 1, 2, 4 and 8 CTAs.
struct Fit {
    uint32_t pairs, splits[4];
};

template <class... Params>
uint32_t clusters_of(void (*kernel)(Params...), uint32_t ctas) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ctas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        n = 0;
    }
    return (uint32_t)std::max(n, 1);
}

// A property of the device: asked once per device.
Fit fit_of(int device, uint32_t sms) {
    static std::mutex mu;
    static Fit known[64];
    std::lock_guard<std::mutex> lock(mu);
    Fit local{};
    Fit& f = device < 64 ? known[device] : local;
    if (!f.pairs) {
        f.pairs = clusters_of(ortho_pair_kernel, 2);
        f.splits[0] = sms;
        f.splits[1] = clusters_of(ortho_split_kernel<APPLY, 2>, 2);
        f.splits[2] = clusters_of(ortho_split_kernel<APPLY, 4>, 4);
        f.splits[3] = clusters_of(ortho_split_kernel<APPLY, 8>, 8);
    }
    return f;
}

// How one product runs: by CTA pairs on tiles of 256 x tn, or split over clusters on tiles of 128 x 128.
struct Form {
    bool pair;
    uint32_t tn, ctas;           // pair: columns of a tile; split: CTAs of a cluster
    double us;                   // estimated
};

uint32_t ceil_div(uint64_t a, uint64_t b) { return (uint32_t)((a + b - 1) / b); }

uint32_t tiles_of(bool square, uint32_t tile_m, uint32_t tile_n, uint64_t rows, uint64_t cols) {
    const uint32_t tm = ceil_div(rows, tile_m);
    return square ? tm * (tm + 1) / 2 : tm * ceil_div(cols, tile_n);
}

// The form whose estimated time is least: clusters of 1 instead of the best number take 179 us for 1024 x 1024
// and not 127, 234 for 700 x 4000 and not 164.  Measured: a k block of 64 costs a pair 0.275 us at 256 columns,
// 0.21 us at 128, and its set-up and last epilogue 8 us; a split CTA takes 0.36 us a k block (what one SM
// can load) and 4.6 us besides in every round of tiles, 0.6 us more where a cluster adds up its sums, 0.5
// more in one of eight.
Form form_of(bool square, uint64_t rows, uint64_t cols, uint64_t K, uint32_t batch, const Fit& fit) {
    const uint32_t kblocks = ceil_div(K, BK);
    Form best{};
    double least = 1e30;
    for (uint32_t tn = 256; tn >= (square ? 256u : 128u); tn /= 2) {
        const double rounds = ceil_div((uint64_t)tiles_of(square, 256, tn, rows, cols) * batch, fit.pairs);
        const double t = 8.0 + rounds * (0.3 + kblocks * (tn == 256 ? 0.275 : 0.21));
        if (t < least) {
            least = t;
            best = {true, tn, 0, t};
        }
    }
    for (uint32_t n = 0; n < 4 && (1u << n) <= kblocks; ++n) {
        const uint32_t ctas = 1u << n;
        const double rounds = ceil_div((uint64_t)tiles_of(square, 128, 128, rows, cols) * batch, fit.splits[n]);
        const double t = 0.8 + rounds * (4.6 + 0.6 * (ctas > 1) + 0.5 * (ctas > 4) + 0.36 * ceil_div(kblocks, ctas));
        if (t < least) {
            least = t;
            best = {false, 128, ctas, t};
        }
    }
    return best;
}

// The same for a whole step in the one launch of CTA pairs: a tile of each product after the other, or all tiles
// over all pairs, a tile of the last product no less than its epilogue's 3 us, and 5 us a product from the last
// tile's sums to the next one's first.  Measured, five steps, this against a launch a product: 4096 x 4096
// 915 us and 990, 3000 x 3000 456 and 576, four of 2048 x 2048 540 and 640, 2048 x 8192 544 and 610; the rule
// leaves alone 1024 x 4096, 228 and 178, and four of 300 x 8192, 287 and 267.
double flow_us(uint64_t S, uint64_t L, uint32_t batch, uint32_t splits, const Fit& fit) {
    const double square = (double)tiles_of(true, 256, 256, S, S) * batch, oblong = (double)tiles_of(false, 256, 256, S, L) * batch;
    const double poly = 0.3 + 0.275 * ceil_div(S, BK), apply = std::max(poly, 3.0);
    const double all = (square * (gram_us(L, 1) + poly) + oblong * apply) / fit.pairs;
    const double chain = gram_us(L, splits) + poly + apply * std::max(1.0, oblong / fit.pairs);
    return 16.0 + std::max(1.1 * all, 1.3 * chain);
}

// The same for POLY and APPLY in one (S <= 256): 9 us a round of tiles, measured.  Two launches instead: 100 us
// for 1000 x 256 and not 86, 109 for 256 x 4096 and not 95.
double fused_us(uint64_t S, uint64_t L, uint32_t batch, uint32_t sms) {
    return 0.8 + 9.0 * ceil_div((uint64_t)tiles_of(false, 128, 128, S, L) * batch, sms);
}

// CTAs of a cluster that hold S x L in shared memory: as few as can (A crosses them all); 0: none can.  Taken
// wherever one can: 128 x 4096 58 us against 89 with a launch a product, 32 of them 285 and 364, 256
// of 128 x 512 188 and 430.  (At 64 rows, with more clusters of 16 than run at once, it is level: 64 of 64 x 4096
// take 546 and 532.)
uint32_t resident_ctas(uint64_t S, uint64_t L) {
    uint32_t ctas = 1;
    while (ctas < RES_CTAS && ceil_div(L, 64) > ctas * RES_BLOCKS) ctas *= 2;
    return S <= 128 && ceil_div(L, 64) <= ctas * RES_BLOCKS ? ctas : 0;
}

template <Product P>
cudaError_t launch_split(GemmParams& p, const Form& f, cudaStream_t stream) {
    p.tiles_m = ceil_div(p.S, 128);
    p.tiles = tiles_of(P != APPLY, 128, 128, p.S, p.L);
    auto kernel = f.ctas == 1 ? ortho_split_kernel<P, 1> : f.ctas == 2 ? ortho_split_kernel<P, 2>
                : f.ctas == 4 ? ortho_split_kernel<P, 4> : ortho_split_kernel<P, 8>;
    return launch(kernel, p.tiles * p.batch * f.ctas, THREADS, SMEM_BYTES, f.ctas, true, stream, p);
}

// Tiles of a step's products first .. last, of all matrices.
uint32_t pair_tiles_of(const PairParams& p) {
    uint32_t tiles = 0;
    for (uint32_t q = p.first; q <= p.last; ++q)
        tiles += p.batch * (q == APPLY ? p.n * p.across : p.n * (p.n + 1) / 2 * (q == GRAM ? p.splits : 1));
    return tiles;
}

// One product after the launch before it; or, with counters, everything: a cooperative launch then, since
// its clusters wait for one another.
cudaError_t launch_pair(const PairParams& p, uint32_t pairs, cudaStream_t stream) {
    const uint32_t grid = 2 * (uint32_t)std::min<uint64_t>((uint64_t)pair_tiles_of(p) * p.steps, pairs);
    if (!p.counters) return launch(ortho_pair_kernel, grid, THREADS, SMEM_BYTES, 0, true, stream, p);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeCooperative;
    attr.val.cooperative = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, ortho_pair_kernel, p);
}

template <Product P>
cudaError_t prepare_splits() {
    cudaError_t e = cudaSuccess;
    for (auto kernel : {ortho_split_kernel<P, 1>, ortho_split_kernel<P, 2>, ortho_split_kernel<P, 4>, ortho_split_kernel<P, 8>}) {
        if (e == cudaSuccess) e = prepare_kernel(kernel);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
    }
    return e;
}

using UpdateKernel = void (*)(UpdateParams);
UpdateKernel update_kernel(bool b16, bool mom) {
    return b16 ? mom ? ortho_update_kernel<true, true> : ortho_update_kernel<true, false>
               : mom ? ortho_update_kernel<false, true> : ortho_update_kernel<false, false>;
}
UpdateKernel start_kernel(bool b16, bool mom) {
    return b16 ? mom ? ortho_start_kernel<true, true> : ortho_start_kernel<true, false>
               : mom ? ortho_start_kernel<false, true> : ortho_start_kernel<false, false>;
}

}  // namespace

cudaError_t preload_ortho_kernels() {
    cudaError_t e = prepare_kernel(ortho_pair_kernel);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(ortho_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
    if (e == cudaSuccess) e = prepare_splits<GRAM>();
    if (e == cudaSuccess) e = prepare_splits<POLY>();
    if (e == cudaSuccess) e = prepare_splits<APPLY>();
    for (auto kernel : {ortho_resident_kernel<1>, ortho_resident_kernel<2>, ortho_resident_kernel<4>, ortho_resident_kernel<8>,
                        ortho_resident_kernel<16>}) {
        if (e == cudaSuccess) e = prepare_kernel(kernel);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)RES_SMEM);
    }
    if (e == cudaSuccess) e = cudaFuncSetAttribute(ortho_resident_kernel<16>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) e = prepare_kernel(ortho_fused_kernel);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(ortho_fused_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)FUSED_SMEM);
    for (uint32_t k = 0; k < 4; ++k) {
        if (e == cudaSuccess) e = prepare_kernel(update_kernel(k & 1, k & 2));
        if (e == cudaSuccess) e = prepare_kernel(start_kernel(k & 1, k & 2));
    }
    if (e == cudaSuccess) e = prepare_kernel(ortho_update_elements_kernel);
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
    // boxes of 64 x 128 (columns x rows): K-contiguous operands, and slabs
    CUtensorMap hi_rows[2], lo_rows, gram, poly;
    // boxes of 64 x 64: the N-contiguous operand of the last product, and mirrored blocks
    CUtensorMap hi_cols[2], gram_blocks, poly_blocks;
    bool fused;                  // POLY within APPLY
    bool flow;                   // all products of all steps in one launch of CTA pairs
    uint32_t resident;           // CTAs of a cluster in the resident form; 0: a launch a product
    Fit fit;
    Form form[3];                // of each Product
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
    o->resident = resident_ctas(l.S, l.L);
    o->fit = fit_of(dev, o->sms);
    o->form[GRAM] = form_of(true, l.S, l.S, l.L, d->batch, o->fit);
    o->form[POLY] = form_of(true, l.S, l.S, l.S, d->batch, o->fit);
    o->form[APPLY] = form_of(false, l.S, l.L, l.S, d->batch, o->fit);
    // its second term of b A + c A A is worth some time: without it a flat spectrum's error is 1.6 times bf16's own
    o->fused = l.S <= 256 && fused_us(l.S, l.L, d->batch, o->sms) < 1.3 * (o->form[POLY].us + o->form[APPLY].us);
    o->flow = !o->resident && !o->fused &&
              flow_us(l.S, l.L, d->batch, l.splits, o->fit) < o->form[GRAM].us + o->form[POLY].us + o->form[APPLY].us;
    bool ok = make_map(&o->gram, o->ws + l.gram, l.S, l.S, d->batch, l.s_pitch, 128) &&
              make_map(&o->poly, o->ws + l.poly, l.S, l.S, d->batch, l.s_pitch, 128) &&
              make_map(&o->gram_blocks, o->ws + l.gram, l.S, l.S, d->batch, l.s_pitch, 64) &&
              make_map(&o->poly_blocks, o->ws + l.poly, l.S, l.S, d->batch, l.s_pitch, 64) &&
              make_map(&o->lo_rows, o->ws + l.lo, l.L, l.S, d->batch, l.l_pitch, 128);
    for (int i = 0; i < 2 && ok; ++i)
        ok = make_map(&o->hi_rows[i], o->ws + l.hi[i], l.L, l.S, d->batch, l.l_pitch, 128) &&
             make_map(&o->hi_cols[i], o->ws + l.hi[i], l.L, l.S, d->batch, l.l_pitch, 64);
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
        // one matrix after the other, or the rows of one between those of another
        const uint64_t row = d.cols * a.e;
        if (d.batch > 1 && a.stride < (d.rows - 1) * a.pitch + row && (a.stride < row || a.pitch < (d.batch - 1) * a.stride + row))
            return fail(DTT_EINVAL, "%s: %s: the matrices overlap", who, a.name);
    }
    if (reinterpret_cast<uintptr_t>(err) % 4) return fail(DTT_EINVAL, "%s: err is misaligned", who);

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
    up.counters = o->flow ? reinterpret_cast<uint32_t*>(o->ws + l.counters) : nullptr;
    up.n_counters = (uint32_t)l.n_counters;
    up.hi = reinterpret_cast<__half*>(o->ws + l.hi[0]);
    up.lo = reinterpret_cast<__half*>(o->ws + l.lo);
    up.l_pitch = l.l_pitch;
    up.S = (uint32_t)l.S;
    const bool tall = d.rows > d.cols;
    const bool out_vec = reinterpret_cast<uintptr_t>(out) % 16 == 0 && out_pitch % 16 == 0 && (d.batch == 1 || out_stride % 16 == 0);
    bool vec = d.cols % 8 == 0;
    for (const auto& a : args)
        if (a.p != out && a.p) vec = vec && reinterpret_cast<uintptr_t>(a.p) % 16 == 0 && a.pitch % 16 == 0 && a.stride % 16 == 0;
    const uint64_t items = d.rows * (vec ? d.cols / 8 : (d.cols + 255) / 256);
    const bool b16 = d.x_dtype == DTT_BF16;
    const uint64_t each = vec ? 256 : 8;
    up.parts = (uint32_t)std::min<uint64_t>((items + each - 1) / each, std::max((vec ? kMaxParts : kMaxParts / 2) / d.batch, 1u));
    if (o->resident) {
        ResidentParams r{};
        r.u = up;
        r.out = {static_cast<char*>(out), out_pitch, (uint32_t)l.S, (uint32_t)l.L, d.scale, tall, out_vec};
        r.out_stride = out_stride;
        r.blocks = ceil_div(ceil_div(l.L, 64), o->resident);
        r.vec = vec;
        r.steps = d.steps;
        r.err = err;
        std::copy(&d.coeffs[0][0], &d.coeffs[0][0] + 3 * d.steps, &r.coeffs[0][0]);
        auto kernel = o->resident == 1 ? ortho_resident_kernel<1> : o->resident == 2 ? ortho_resident_kernel<2>
                    : o->resident == 4 ? ortho_resident_kernel<4> : o->resident == 8 ? ortho_resident_kernel<8> : ortho_resident_kernel<16>;
        DTT_CUDA_TRY(launch(kernel, d.batch * o->resident, RES_THREADS, RES_SMEM, o->resident, true, stream, r));
        return DTT_OK;
    }
    const dim3 parts(up.parts, d.batch);
    // not overlapped with what ran before (512 x 512: 105 us, overlapped 108)
    DTT_CUDA_TRY(launch(vec ? update_kernel(b16, momentum) : ortho_update_elements_kernel, parts, 256, 0, 0, false, stream, up));
    if (vec && !tall) {
        const uint32_t ctas = (uint32_t)std::min<uint64_t>((items + 255) / 256, std::max(START_CTAS * o->sms / d.batch, 1u));
        DTT_CUDA_TRY(launch(start_kernel(b16, momentum), dim3(ctas, d.batch), 256, 0, 0, true, stream, up));
    } else {
        const dim3 tiles(ceil_div(up.cols, kStartTile), ceil_div(up.rows, kStartTile), d.batch);
        DTT_CUDA_TRY(launch(tall ? ortho_start_tiles_kernel<true> : ortho_start_tiles_kernel<false>, tiles, 256, 0, 0, true, stream, up));
    }

    PairParams pp{};
    pp.splits = 1;
    for (int i = 0; i < 2; ++i) {
        pp.hi_rows[i] = o->hi_rows[i];
        pp.hi_cols[i] = o->hi_cols[i];
    }
    pp.lo_rows = o->lo_rows;
    pp.gram = o->gram;
    pp.poly = o->poly;
    pp.gram_blocks = o->gram_blocks;
    pp.poly_blocks = o->poly_blocks;
    pp.S = (uint32_t)l.S;
    pp.L = (uint32_t)l.L;
    pp.batch = d.batch;
    pp.n = ceil_div(l.S, 256);
    pp.tn = !o->flow && o->form[APPLY].pair ? o->form[APPLY].tn : 256;
    pp.across = ceil_div(l.L, pp.tn);
    pp.out_pitch = out_pitch;
    pp.out_stride = out_stride;
    pp.scale = d.scale;
    pp.transposed = tall;
    pp.out_vec = out_vec;
    pp.err = err;
    if (o->flow) {
        pp.first = GRAM;
        pp.last = APPLY;
        pp.steps = d.steps;
        pp.counters = up.counters;
        pp.splits = l.splits;
        pp.parts = reinterpret_cast<float*>(o->ws + l.parts);
        pp.out = static_cast<char*>(out);
        std::copy(&d.coeffs[0][0], &d.coeffs[0][0] + 3 * d.steps, &pp.coeffs[0][0]);
        DTT_CUDA_TRY(launch_pair(pp, o->fit.pairs, stream));
        return DTT_OK;
    }
    auto pair = [&](Product product, uint32_t k) {
        pp.first = pp.last = product;
        pp.step = k;
        pp.steps = 1;
        pp.out = product == APPLY && k + 1 == d.steps ? static_cast<char*>(out) : nullptr;
        std::copy(&d.coeffs[k][0], &d.coeffs[k][0] + 3, &pp.coeffs[0][0]);
        return launch_pair(pp, o->fit.pairs, stream);
    };

    GemmParams g{};
    g.S = (uint32_t)l.S;
    g.batch = d.batch;
    g.s_pitch = l.s_pitch;
    g.l_pitch = l.l_pitch;
    g.lo = up.lo;
    g.err = err;
    g.scale = d.scale;
    g.transposed = tall;
    g.out_vec = out_vec;
    g.out_pitch = out_pitch;
    g.out_stride = out_stride;
    for (uint32_t k = 0; k < d.steps; ++k) {
        const uint32_t now = k & 1;
        g.a = d.coeffs[k][0];
        g.b = d.coeffs[k][1];
        g.c = d.coeffs[k][2];
        g.L = g.S;
        g.tmA = g.tmB = o->hi_rows[now];
        g.K = (uint32_t)l.L;
        g.out16 = reinterpret_cast<__half*>(o->ws + l.gram);
        DTT_CUDA_TRY(o->form[GRAM].pair ? pair(GRAM, k) : launch_split<GRAM>(g, o->form[GRAM], stream));
        g.tmA = g.tmB = o->gram;
        g.K = g.S;
        g.gram = g.out16;
        g.out16 = reinterpret_cast<__half*>(o->ws + l.poly);
        if (!o->fused) DTT_CUDA_TRY(o->form[POLY].pair ? pair(POLY, k) : launch_split<POLY>(g, o->form[POLY], stream));
        g.tmA = o->fused ? o->gram : o->poly;
        g.tmB = o->hi_cols[now];
        g.L = (uint32_t)l.L;
        g.hi = reinterpret_cast<const __half*>(o->ws + l.hi[now]);
        g.out16 = reinterpret_cast<__half*>(o->ws + l.hi[now ^ 1]);
        g.out = k + 1 == d.steps ? static_cast<char*>(out) : nullptr;
        if (o->fused) {
            g.tiles_m = ceil_div(g.S, 128);
            g.tiles = tiles_of(false, 128, 128, g.S, g.L);
            DTT_CUDA_TRY(launch(ortho_fused_kernel, g.tiles * g.batch, THREADS, FUSED_SMEM, 0, true, stream, g));
        } else {
            DTT_CUDA_TRY(o->form[APPLY].pair ? pair(APPLY, k) : launch_split<APPLY>(g, o->form[APPLY], stream));
        }
    }
    return DTT_OK;
}

// AdamW over all tensors of a list in one pass (dtt_ops.h has the definition).
//
// What a step cannot do without is reading each gradient, weight and state once and writing the last two: 28
// bytes a weight (bf16 gradients; weights and states f32, a bf16 copy), 10 with states in 8 bits and bf16
// weights.  All f32 between the loads and the stores.  A CTA takes a chunk of one tensor; a launch's table of
// tensors travels with its arguments, so that a call needs no device memory, copies nothing, and may be
// captured with whatever pointers it was given.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>
#include <vector>

#include "dtt_ops.h"
#include "internal.h"
#include "rowio.cuh"

namespace dtt {
namespace {

constexpr uint32_t kThreads = 256, kChunk = 8 * kThreads;      // elements of a CTA
constexpr uint32_t kBlock = DTT_ADAMW_BLOCK;                   // elements of a scale: 16 threads' or 4 of each lane's
constexpr float kCodeMax = 448.0f, kScaleLeast = 0x1p-100f;
constexpr float kCodeLeast = 0x1p-9f;                          // e4m3's smallest value above zero
constexpr uint64_t kMostElements = 1ull << 40;
// 8-bit states: where there are many elements a CTA takes several chunks, whose copies go out together and which share
// the search for the tensor and the step's numbers.  32M weights: 88 us with one chunk a CTA, straight from global memory, 60 with
// four, before the largest were settled.  (f32 states: 715 us with one at 151M weights; two or three by way of shared
// memory 766 to 789, reads that run further ahead of the writes cost more than they hide.)
constexpr uint32_t kTurns = 4;
constexpr uint64_t kManyElements = 4ull * kTurns * kChunk * kSms;

struct Tensor {
    char* p;
    const char* g;
    char* m;
    char* v;
    float* ms;
    float* vs;
    uint16_t* copy;             // or null
    uint64_t n;
    float decay;
    uint32_t lead;              // pointers (not the scales') are moved back by so many elements, from where every eighth is 16-byte
                                // aligned (codes: 8-byte); kElements: there is no such place for all of them
    uint32_t number;            // in the caller's list
};
constexpr uint32_t kElements = 8;

// 8-bit states: v is taken times kUnit^2, its root times kUnit, so that where f32's v would be subnormal it is not, and the
// root's instruction, which takes subnormal numbers for 0, needs no step of its own.  Past 2^104 v leaves f32 then, which eight elements' largest
// root tells, and the few of which it does are worked out again.  32M weights (bf16, at random; to nearest; f32, to nearest) 64.5, 50.4 and 110 us;
// with three instructions more at each root 66, 51 and 116; with those few worked out after all others 64, 54 and 117.
constexpr float kUnit = 0x1p12f;

struct Scalars {
    float beta1, beta2, root_beta2;     // root_beta2: its square root, as the next's; 8-bit states: times kUnit, both
    float one_less_beta1, one_less_beta2, root_one_less_beta2;
    float eps;
    float lr, lr_by_c1, root_c2;        // by the host's step: lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
    float root_by;                      // what roots are taken times, its reciprocal: in root_c2
    float log_beta1, log_beta2;         // for the device's step
    const float* lr_dev;                // or null
    const uint32_t* step_dev;           // or null
    const float* grad_scale;            // or null
    uint32_t step, seed;                // seed: mixed once
    uint32_t sixteen;                   // 16 (stochastic_code)
};

template <uint32_t N>
struct Batch {
    Tensor t[N];
    uint32_t first[N + 1];              // CTA that tensor i begins with
    uint32_t count;
    uint32_t turns;                     // chunks that a CTA takes one after the other
    Scalars s;
};
// Arguments end at 32764 bytes.
constexpr uint32_t kFew = 44, kMany = 384;
static_assert(sizeof(Batch<kMany>) <= 32764 && sizeof(Batch<kFew>) <= 4096, "the tables of tensors travel as arguments");

// 32 bits from 32: products with odd numbers (fractional digits of pi and e) carry every bit upwards, shifts bring
// it down again.
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
    x = (x ^ (x >> 16)) * 0x85A308D3u;
    x = (x ^ (x >> 15)) * 0xB7E15163u;
    return x ^ (x >> 16);
}
constexpr uint32_t kGolden = 0x9E3779B9u, kThird = 0x2E1B2139u;

__device__ __forceinline__ uint32_t random_bits(uint64_t i, uint32_t seed) {
    return mix((uint32_t)i * kGolden + seed + (uint32_t)(i >> 32) * kThird);
}

__device__ __forceinline__ float root_of(float v) {
    float r;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float root_of_normal(float v) {         // 0 of a subnormal v
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float reciprocal(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// What a step's formula needs, by the host or by the device's own step and rate.
struct Rates {
    float lr, lr_by_c1, root_c2;
    float g_m, g_v;             // what the gradient enters m and, squared, v with
    uint32_t step;
};
__device__ __forceinline__ Rates rates_of(const Scalars& s) {
    const float gs = s.grad_scale ? *s.grad_scale : 1.0f;
    Rates r{s.lr, s.lr_by_c1, s.root_c2, s.one_less_beta1 * gs, s.root_one_less_beta2 * gs, s.step};
    if (s.lr_dev || s.step_dev) {
        if (s.lr_dev) r.lr = *s.lr_dev;
        if (s.step_dev) r.step = *s.step_dev;
        const float t = (float)r.step;          // 1 - beta^t = -expm1(t log beta): nothing cancels
        r.lr_by_c1 = r.lr / -expm1f(t * s.log_beta1);
        r.root_c2 = rsqrtf(-expm1f(t * s.log_beta2)) * s.root_by;
    }
    return r;
}

// 8-bit states: the root times kUnit of one element, whose code and gradient are these, where v is above 2^104; and of any.
__device__ __forceinline__ float large_root_from(float code, float v_by, float g, const Rates& r) {
    const float o = __fmul_rn(code, v_by) * (1.0f / kUnit), n = __fmul_rn(g, r.g_v) * (1.0f / kUnit);
    return root_of_normal(fmaf(o, o, __fmul_rn(n, n))) * kUnit;
}
__device__ __forceinline__ float root_from(float code, float v_by, float g, const Rates& r) {
    const float old = __fmul_rn(code, v_by), gv = __fmul_rn(g, r.g_v), v = fmaf(old, old, __fmul_rn(gv, gv));
    return isinf(v) ? large_root_from(code, v_by, g, r) : root_of_normal(v);
}

// Eight elements.  m and v: as the old ones or as codes with what their scales make of them: m_by and v_by, one for each four, are beta1
// and beta2, or the scales times beta1 and sqrt(beta2).  root: sqrt(v), with 8-bit states times kUnit; top: their largest, NaN if one
// is.  decay: lr times the tensor's.  again(k): large_root_from for element k, asked for where v, times kUnit's square, has left f32 (past 2^104).
template <bool S8, class Again>
__device__ __forceinline__ void update(float (&p)[8], const float (&g)[8], float (&m)[8], float (&v)[8], float2 (&root)[4], float& top, float2 m_by, float2 v_by,
                                       float decay, const Rates& r, float eps, Again again) {
#pragma unroll
    for (uint32_t k = 0; k < 8; k += 2) {
        const Pair gg = pair(g[k], g[k + 1]), gv = gg * both(r.g_v);
        const Pair mm = fma2(pair(m[k], m[k + 1]), both(k < 4 ? m_by.x : m_by.y), gg * both(r.g_m));
        Pair vv = pair(v[k], v[k + 1]);
        const Pair by = both(k < 4 ? v_by.x : v_by.y);
        if (S8) {
            vv = vv * by;
            vv = fma2(vv, vv, gv * gv);
        } else {
            vv = fma2(vv, by, gv * gv);
        }
        const float2 b = apart(mm), c = apart(vv);
        m[k] = b.x, m[k + 1] = b.y, v[k] = c.x, v[k + 1] = c.y;
        root[k / 2] = S8 ? make_float2(root_of_normal(c.x), root_of_normal(c.y)) : make_float2(root_of(c.x), root_of(c.y));
    }
    const auto largest = [&] {
        const float a = max3_nan(max3_nan(root[0].x, root[0].y, root[1].x), root[1].y, root[2].x);
        return max3_nan(max_nan(a, root[2].y), root[3].x, root[3].y);
    };
    if (S8) {
        top = largest();
        if (!(top < INFINITY)) {
            uint32_t left = 0;
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k) left |= (isinf(k % 2 ? root[k / 2].y : root[k / 2].x) ? 1u : 0u) << k;
#pragma unroll 1
            for (; left; left &= left - 1) {
                const uint32_t at = __ffs(left) - 1;
                const float x = again(at);
#pragma unroll
                for (uint32_t k = 0; k < 8; ++k)
                    if (k == at) (k % 2 ? root[k / 2].y : root[k / 2].x) = x;
            }
            top = largest();
        }
    }
#pragma unroll
    for (uint32_t k = 0; k < 8; k += 2) {
        const float2 d = apart(fma2(pair(root[k / 2].x, root[k / 2].y), both(r.root_c2), both(eps)));
        const Pair pp = pair(p[k], p[k + 1]);
        // p - decay p, not p (1 - decay): what rounding 1 - 1e-6 to f32 is off by, up to 2^-25, is 3 % of the 1e-6, of every weight the same
        // way
        const float2 a = apart(fma2(pair(m[k], m[k + 1]) * pair(reciprocal(d.x), reciprocal(d.y)), both(-r.lr_by_c1), fma2(pp, both(-decay), pp)));
        p[k] = a.x, p[k + 1] = a.y;
    }
}

// ---- codes ---------------------------------------------------------------------------------------
struct Scale {
    float scale, inv;           // top inv is 448 at most
};
// top: times `by`, as what inv is for.
__device__ __forceinline__ Scale scale_from(float top, float by = 1.0f) {
    const float scale = max_nan(top * (1.0f / kCodeMax / by), kScaleLeast);
    float inv = reciprocal(scale) * (1.0f / by);
    if (top * inv > kCodeMax) inv *= 1.0f - 0x1p-22f;
    return {scale, inv};
}

// Up with the probability of what lies below: a random number in the place of the bits that are cut off, the
// noise's 16 bits (at bit 8) in that of the highest of them.  x, 448 at most, times 2^-120 has e4m3's exponents and its
// subnormal values where f32 has its own, so that the code is bits 20 to 26 of the magnitude; it comes back in the
// highest byte, and the sign is shifted out.  The shift by 4 is a product with a number that the compiler does not know: of
// the highest byte of (x << 4) + noise, with nothing else asked for, CUDA 13.0's leaves out the x.
constexpr float kCodeUnit = 0x1p-120f;
__device__ __forceinline__ uint32_t stochastic_code(float x, uint32_t noise, uint32_t sixteen) {
    uint32_t r;
    asm("mad.lo.u32 %0, %1, %2, %3;" : "=r"(r) : "r"(__float_as_uint(x)), "r"(sixteen), "r"(noise));
    return r;
}
__device__ __forceinline__ uint32_t noise_m(uint32_t r) { return __byte_perm(r, 0, 0x4324); }      // r's high 16 bits at bit 8
__device__ __forceinline__ uint32_t noise_v(uint32_t r) { return __byte_perm(r, 0, 0x4104); }      // its low ones
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}

// The same of bf16; what is cut off is cut off when it is packed.
__device__ __forceinline__ uint32_t stochastic_bf16(float x, uint32_t r) { return __float_as_uint(x) + (r * kThird >> 16); }
__device__ __forceinline__ uint32_t pack_cut(uint32_t lo, uint32_t hi) { return __byte_perm(lo, hi, 0x7632); }

// Four elements' codes of m and of their roots, which stay above zero: the next step divides by them.  r: the
// elements' random bits.
template <bool SR>
__device__ __forceinline__ uint32_t moment_codes(const Pair (&m)[2], float inv, const uint32_t* r, uint32_t sixteen) {
    const Pair x[2] = {m[0] * both(inv), m[1] * both(inv)};
    const float2 a = apart(x[0]), b = apart(x[1]);
    if (!SR) return pack_e4m3(a.x, a.y) | pack_e4m3(b.x, b.y) << 16;
    const float2 c = apart(x[0] * both(kCodeUnit)), d = apart(x[1] * both(kCodeUnit));
    const uint32_t codes = top_bytes(stochastic_code(c.x, noise_m(r[0]), sixteen), stochastic_code(c.y, noise_m(r[1]), sixteen),
                                     stochastic_code(d.x, noise_m(r[2]), sixteen), stochastic_code(d.y, noise_m(r[3]), sixteen));
    return codes | (top_bytes(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y)) & 0x80808080u);
}
__device__ __forceinline__ uint32_t stays_above_zero(uint32_t code, float root) {
    asm("{\n\t.reg .pred p;\n\tsetp.gt.f32 p, %1, 0f00000000;\n\t@p max.u32 %0, %0, %2;\n\t}" : "+r"(code) : "f"(root), "r"(1u << 24));
    return code;
}
template <bool SR>
__device__ __forceinline__ uint32_t root_codes(const float2 (&root)[2], float inv, const uint32_t* r, uint32_t sixteen) {
    const Pair x[2] = {pair(root[0].x, root[0].y) * both(inv), pair(root[1].x, root[1].y) * both(inv)};
    if (SR) {
        const float2 c = apart(x[0] * both(kCodeUnit)), d = apart(x[1] * both(kCodeUnit));
        return top_bytes(stays_above_zero(stochastic_code(c.x, noise_v(r[0]), sixteen), root[0].x), stays_above_zero(stochastic_code(c.y, noise_v(r[1]), sixteen), root[0].y),
                         stays_above_zero(stochastic_code(d.x, noise_v(r[2]), sixteen), root[1].x), stays_above_zero(stochastic_code(d.y, noise_v(r[3]), sixteen), root[1].y));
    }
    const float2 a = apart(x[0]), b = apart(x[1]);
    const auto least = [](float x, float root) { return root == 0.0f ? 0.0f : max_nan(x, kCodeLeast); };
    return pack_e4m3(least(a.x, root[0].x), least(a.y, root[0].y)) | pack_e4m3(least(b.x, root[1].x), least(b.y, root[1].y)) << 16;
}
// What becomes of four codes in a block with a NaN, whose scale is one.
__device__ __forceinline__ uint32_t poison(float top) { return isnan(top) ? 0x7F7F7F7Fu : 0u; }

__device__ __forceinline__ void unpack_e4m3(uint32_t pair, float& lo, float& hi) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)pair));
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}" : "=f"(lo), "=f"(hi) : "r"(h));
}
__device__ __forceinline__ void unpack8(uint2 q, float (&v)[8]) {
    unpack_e4m3(q.x & 0xFFFFu, v[0], v[1]);
    unpack_e4m3(q.x >> 16, v[2], v[3]);
    unpack_e4m3(q.y & 0xFFFFu, v[4], v[5]);
    unpack_e4m3(q.y >> 16, v[6], v[7]);
}

// ---- chunks ----------------------------------------------------------------------------------------
template <uint32_t DT>
__device__ __forceinline__ float element(const char* base, uint64_t i) {
    return DT == DTT_BF16 ? __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(base)[i] << 16) : reinterpret_cast<const float*>(base)[i];
}

__device__ __forceinline__ float code_of(const char* codes, uint64_t i) {
    float v, none;
    unpack_e4m3(reinterpret_cast<const uint8_t*>(codes)[i], v, none);
    return v;
}

template <uint32_t P, uint32_t G, bool S8, class T>
__device__ __forceinline__ void load_element(const T& t, uint64_t i, float& p, float& g, float& m, float& v) {
    p = element<P>(t.p, i);
    g = element<G>(t.g, i);
    if (S8) {
        m = code_of(t.m, i);
        v = code_of(t.v, i);
    } else {
        m = element<DTT_F32>(t.m, i);
        v = element<DTT_F32>(t.v, i);
    }
}

// p: its rounded bits in the high half, where it is bf16 and rounded at random.
template <uint32_t P, bool S8, bool SR, class T>
__device__ __forceinline__ void store_element(const T& t, uint64_t i, float p, uint32_t cut, float m, float v, uint32_t code_m, uint32_t code_v) {
    if (S8) {
        reinterpret_cast<uint8_t*>(t.m)[i] = (uint8_t)code_m;
        reinterpret_cast<uint8_t*>(t.v)[i] = (uint8_t)code_v;
    } else {
        reinterpret_cast<float*>(t.m)[i] = m;
        reinterpret_cast<float*>(t.v)[i] = v;
    }
    if (P == DTT_BF16)
        reinterpret_cast<uint16_t*>(t.p)[i] = SR ? (uint16_t)(cut >> 16) : (uint16_t)pack_bf16(p, 0.0f);
    else
        reinterpret_cast<float*>(t.p)[i] = p;
    if (P == DTT_F32 && t.copy) reinterpret_cast<uint16_t*>(t.copy)[i] = (uint16_t)pack_bf16(p, 0.0f);
}

// Where an element's noise is 0 the largest of a block, which is 448 or an ulp below it once its scale is taken off, has
// 448's code or the one below, 7 % less; with any other noise it has 448's.  Which of them is not to depend on how products and
// sums are put together here, so that it is worked out once more by the formula, each product and sum rounded by itself.
// code and scale: the old m's or root's; g: the gradient.
__device__ __forceinline__ uint32_t largest_code(float x) {
    const float by = __fmul_rn(x, 1.0f / kCodeMax), inv = __frcp_rn(by > kScaleLeast ? by : kScaleLeast);
    return __fmul_rn(x, inv) < kCodeMax ? 0x7Du : 0x7Eu;
}
__device__ __forceinline__ uint32_t largest_m(float code, float scale, float g, const Scalars& s) {
    if (s.grad_scale) g = __fmul_rn(g, *s.grad_scale);
    const float m = __fadd_rn(__fmul_rn(s.beta1, __fmul_rn(code, scale)), __fmul_rn(s.one_less_beta1, g));
    return largest_code(fabsf(m)) | (__float_as_uint(m) >> 24 & 0x80u);
}
__device__ __forceinline__ uint32_t largest_root(float code, float scale, float g, const Scalars& s) {
    if (s.grad_scale) g = __fmul_rn(g, *s.grad_scale);
    const float root = __fmul_rn(code, scale);
    return largest_code(__fsqrt_rn(__fadd_rn(__fmul_rn(s.beta2, __fmul_rn(root, root)), __fmul_rn(__fmul_rn(s.one_less_beta2, g), g))));
}
// Whether an element's noise is 0, of m or of the root.
template <uint32_t N>
__device__ __forceinline__ bool any_noise_0(const uint32_t* bits) {
    uint32_t least = ~0u;
#pragma unroll
    for (uint32_t k = 0; k < N; k += 2) {
        least = __vimin3_u32(least, noise_m(bits[k]), noise_m(bits[k + 1]));
        least = __vimin3_u32(least, noise_v(bits[k]), noise_v(bits[k + 1]));
    }
    return least == 0;
}
// Elements i + k step of one block, k < count, of which one's noise is 0, if they are the block's largest.  Codes are in m
// and v already; as they were they are bytes of old_m and old_v, in the block with scales ms and vs.  first: the number
// of element 0.  A scale that is the least one does not make a code of 448.
struct Tops {
    float ms, vs, m, root;      // root: times kUnit
};
__device__ __forceinline__ float code_value(uint2 codes, uint32_t k) {
    float v, none;
    unpack_e4m3((k < 4 ? codes.x : codes.y) >> 8 * (k % 4) & 0xFFu, v, none);
    return v;
}
template <uint32_t G>
__device__ __forceinline__ void settle_largest(const char* gs, char* m, char* v, uint64_t i, uint64_t first, uint32_t step, uint32_t count, uint2 old_m, uint2 old_v,
                                               Tops t, uint32_t seed, const Rates& r, const Scalars& s) {
    const auto scaled = [](float top) { return top * (1.0f / kCodeMax) > kScaleLeast && top < INFINITY; };
#pragma unroll 1
    for (uint32_t k = 0; k < count; ++k, i += step) {
        const uint32_t bits = random_bits(first + i, seed);
        if (bits >= 1u << 16 && (bits & 0xFFFFu)) continue;
        const float g = element<G>(gs, i), cm = code_value(old_m, k), cv = code_value(old_v, k);           // m and root: as update() has them
        if (bits < 1u << 16 && scaled(t.m) && fabsf(fmaf(cm, __fmul_rn(t.ms, s.beta1), __fmul_rn(g, r.g_m))) == t.m)
            reinterpret_cast<uint8_t*>(m)[i] = (uint8_t)largest_m(cm, t.ms, g, s);
        if (!(bits & 0xFFFFu) && scaled(t.root * (1.0f / kUnit)) && root_from(cv, __fmul_rn(t.vs, s.root_beta2), g, r) == t.root)
            reinterpret_cast<uint8_t*>(v)[i] = (uint8_t)largest_root(cv, t.vs, g, s);
    }
}

// bf16 of eight weights rounded at random; NaN, which the sum would turn into something else, is left as it is.
__device__ __forceinline__ void cut_weights(const float (&p)[8], const uint32_t (&r)[8], uint32_t (&cut)[8]) {
    Pair none = both(0.0f);                     // NaN where one of them is infinite or NaN
#pragma unroll
    for (uint32_t k = 0; k < 8; k += 2) none = fma2(pair(p[k], p[k + 1]), both(0.0f), none);
    const float2 n = apart(none);
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) cut[k] = stochastic_bf16(p[k], r[k]);
    if (isnan(n.x + n.y)) {
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k)
            if (isnan(p[k])) cut[k] = 0x7FFF0000u;
    }
}

// Elements i, one by one, of a tensor of which nothing is aligned: a warp's 256 neighbours, a lane every 32nd, so
// that accesses are contiguous over the warp and a block of 128 is four of each lane's.
template <uint32_t P, uint32_t G, bool S8, bool SR>
__device__ __forceinline__ void chunk_by_elements(const Tensor& t, uint64_t at, uint32_t seed, float decay, const Rates& r, const Scalars& s) {
    const uint64_t i0 = at + threadIdx.x / 32 * 256 + threadIdx.x % 32;
    float p[8], g[8], m[8], v[8], ms[2], vs[2];
    float2 root[4];
    uint32_t old_m[2] = {}, old_v[2] = {};
    Tops tops[2];
    if (S8) {
#pragma unroll
        for (uint32_t b = 0; b < 2; ++b) {
            const uint64_t i = min(i0 + 128 * b, t.n - 1);
            ms[b] = t.ms[i / kBlock];
            vs[b] = t.vs[i / kBlock];
        }
    }
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) {
        const uint64_t i = min(i0 + 32 * k, t.n - 1);
        load_element<P, G, S8>(t, i, p[k], g[k], m[k], v[k]);
        if (S8 && SR) {
            old_m[k / 4] |= (uint32_t) reinterpret_cast<const uint8_t*>(t.m)[i] << 8 * (k % 4);
            old_v[k / 4] |= (uint32_t) reinterpret_cast<const uint8_t*>(t.v)[i] << 8 * (k % 4);
        }
    }
    const float2 m_by = S8 ? make_float2(ms[0] * s.beta1, ms[1] * s.beta1) : make_float2(s.beta1, s.beta1);
    const float2 v_by = S8 ? make_float2(vs[0] * s.root_beta2, vs[1] * s.root_beta2) : make_float2(s.beta2, s.beta2);
    float top;
    update<S8>(p, g, m, v, root, top, m_by, v_by, decay, r, s.eps, [&](uint32_t k) {
        const uint64_t i = min(i0 + 32 * k, t.n - 1);
        return large_root_from(code_of(t.v, i), k < 4 ? v_by.x : v_by.y, element<G>(t.g, i), r);
    });
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k)
        if (S8 && i0 + 32 * k >= t.n) m[k] = (k % 2 ? root[k / 2].y : root[k / 2].x) = 0.0f;
    uint32_t bits[8] = {}, cut[8] = {}, code_m[2] = {}, code_v[2] = {};
    if (SR) {
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) bits[k] = random_bits(i0 + 32 * k, seed);
        if (P == DTT_BF16) cut_weights(p, bits, cut);
    }
    if (S8) {
#pragma unroll
        for (uint32_t b = 0; b < 8; b += 4) {
            float tm = max3_nan(max_nan(fabsf(m[b]), fabsf(m[b + 1])), fabsf(m[b + 2]), fabsf(m[b + 3]));
            float tr = max3_nan(max_nan(root[b / 2].x, root[b / 2].y), root[b / 2 + 1].x, root[b / 2 + 1].y);
            // as bits, magnitudes order like integers, with NaN on top
            tm = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(tm) & 0x7FFFFFFFu));
            tr = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(tr) & 0x7FFFFFFFu));
            const Scale sm = scale_from(tm), sr = scale_from(tr, kUnit);
            const uint64_t i = i0 + 32 * b;
            if (threadIdx.x % 32 == 0 && i < t.n) {
                t.ms[i / kBlock] = sm.scale;
                t.vs[i / kBlock] = sr.scale;
            }
            const Pair of_m[2] = {pair(m[b], m[b + 1]), pair(m[b + 2], m[b + 3])};
            const float2 roots[2] = {root[b / 2], root[b / 2 + 1]};
            code_m[b / 4] = moment_codes<SR>(of_m, sm.inv, bits + b, s.sixteen) | poison(tm);
            code_v[b / 4] = root_codes<SR>(roots, sr.inv, bits + b, s.sixteen) | poison(tr);
            tops[b / 4] = {ms[b / 4], vs[b / 4], tm, tr};
        }
    }
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) {
        const uint64_t i = i0 + 32 * k;
        if (i < t.n) store_element<P, S8, SR>(t, i, p[k], cut[k], m[k], v[k], code_m[k / 4] >> 8 * (k % 4), code_v[k / 4] >> 8 * (k % 4));
    }
    if (S8 && SR) {
#pragma unroll
        for (uint32_t b = 0; b < 8; b += 4) {
            const uint64_t i = i0 + 32 * b;
            if (i < t.n && any_noise_0<4>(bits + b))
                settle_largest<G>(t.g, t.m, t.v, i, 0, 32, (uint32_t)min((t.n - i + 31) / 32, (uint64_t)4), make_uint2(old_m[b / 4], 0), make_uint2(old_v[b / 4], 0), tops[b / 4], seed, r, s);
        }
    }
}

// A CTA's part of a tensor whose groups are aligned: elements are counted from its start.
struct Part {
    char* p;
    const char* g;
    char* m;
    char* v;
    float* ms;
    float* vs;
    char* copy;
    uint64_t first;             // the start's number in the tensor; before the tensor's first element: wrapped around
    uint32_t head, end;         // the tensor's elements there
};
template <uint32_t P, uint32_t G, bool S8>
__device__ __forceinline__ Part part_of(const Tensor& t, uint64_t start, uint32_t count) {
    Part r;
    r.p = t.p + start * (P == DTT_BF16 ? 2 : 4);
    r.g = t.g + start * (G == DTT_BF16 ? 2 : 4);
    r.m = t.m + start * (S8 ? 1 : 4);
    r.v = t.v + start * (S8 ? 1 : 4);
    r.ms = S8 ? t.ms + start / kBlock : nullptr;
    r.vs = S8 ? t.vs + start / kBlock : nullptr;
    r.copy = P == DTT_F32 && t.copy ? reinterpret_cast<char*>(t.copy + start) : nullptr;
    r.first = start - t.lead;
    r.head = start ? 0 : t.lead;
    r.end = (uint32_t)min((uint64_t)count, t.lead + t.n - start);
    return r;
}

// 8-bit states: a thread's groups come through shared memory, each thread copying its own, all chunks' copies under way
// at once and in nobody's registers; nobody waits but for its own.
template <uint32_t P, uint32_t G>
struct Stage {
    static constexpr uint32_t ge = G == DTT_BF16 ? 16 : 32, pe = P == DTT_BF16 ? 16 : 32;      // bytes of a group
    static constexpr uint32_t p = kThreads * ge, m = p + kThreads * pe, v = m + kThreads * 8, bytes = v + kThreads * 8;
};
__device__ __forceinline__ void copy16(uint32_t to, const char* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t to, const char* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
}
template <uint32_t P, uint32_t G>
__device__ __forceinline__ void start_copies(const Part& a, uint32_t o, uint32_t stage) {
    using S = Stage<P, G>;
    const uint32_t t = threadIdx.x;
    if (o + 8 <= a.end) {
#pragma unroll
        for (uint32_t k = 0; k < S::ge; k += 16) copy16(stage + k * kThreads + 16 * t, a.g + o * (S::ge / 8) + k);
#pragma unroll
        for (uint32_t k = 0; k < S::pe; k += 16) copy16(stage + S::p + k * kThreads + 16 * t, a.p + o * (S::pe / 8) + k);
        copy8(stage + S::m + 8 * t, a.m + o);
        copy8(stage + S::v + 8 * t, a.v + o);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}
__device__ __forceinline__ void copy1(uint32_t to, const char* from) {
    asm volatile("st.shared.u8 [%0], %1;" ::"r"(to), "r"((uint32_t)*reinterpret_cast<const uint8_t*>(from)) : "memory");
}
__device__ __forceinline__ uint4 shared16(uint32_t at) {
    uint4 q;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(at) : "memory");
    return q;
}
__device__ __forceinline__ uint2 shared8(uint32_t at) {
    uint2 q;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(q.x), "=r"(q.y) : "r"(at) : "memory");
    return q;
}

template <uint32_t DT>
__device__ __forceinline__ Raw8 group_of(const char* base, uint32_t o) {
    return raw8(base + (uint64_t)o * (DT == DTT_BF16 ? 2 : 4), DT);
}
// What nobody reads before the next step leaves L2 first: 151M weights with f32 states 703 us, with plain stores 715
// (and with loads marked so too 719).
template <uint32_t DT>
__device__ __forceinline__ void put_group(char* base, uint32_t o, const float (&v)[8]) {
    char* at = base + (uint64_t)o * (DT == DTT_BF16 ? 2 : 4);
    if (DT == DTT_BF16) {
        __stcs(reinterpret_cast<uint4*>(at), make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])));
    } else {
        __stcs(reinterpret_cast<float4*>(at), make_float4(v[0], v[1], v[2], v[3]));
        __stcs(reinterpret_cast<float4*>(at + 16), make_float4(v[4], v[5], v[6], v[7]));
    }
}
template <uint32_t DT>
__device__ __forceinline__ void shared_group(uint32_t at, float (&v)[8]) {
    Raw8 q{};
    q.a = shared16(at + 16 * threadIdx.x);
    if (DT == DTT_F32) q.b = shared16(at + 16 * kThreads + 16 * threadIdx.x);
    expand8(q, DT, v);
}

// Eight neighbouring elements a thread, from element o of the part, a block of 128 sixteen lanes.  Pointers are those of
// the element `lead` places before the tensor's first, so that every eighth from there is aligned; the groups at its
// ends that it does not fill go element by element.
template <uint32_t P, uint32_t G, bool S8, bool SR>
__device__ __forceinline__ bool group(const Part& a, uint32_t o, uint32_t stage, float ms, float vs, uint32_t seed, float decay, const Rates& r, const Scalars& s) {
    float p[8], g[8], m[8], v[8];
    float2 root[4];
    const bool whole = o >= a.head && o + 8 <= a.end;
    const auto mine = [&](uint32_t k) { return o + k >= a.head && o + k < a.end; };
    const uint64_t first = a.first + o;
    if (whole) {
        if (S8) {
            using S = Stage<P, G>;
            shared_group<G>(stage, g);
            shared_group<P>(stage + S::p, p);
            unpack8(shared8(stage + S::m + 8 * threadIdx.x), m);
            unpack8(shared8(stage + S::v + 8 * threadIdx.x), v);
        } else {
            const Raw8 gs = group_of<G>(a.g, o), ps = group_of<P>(a.p, o), x = group_of<DTT_F32>(a.m, o), y = group_of<DTT_F32>(a.v, o);
            expand8(gs, G, g);
            expand8(ps, P, p);
            expand8(x, DTT_F32, m);
            expand8(y, DTT_F32, v);
        }
    } else {
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) {
            p[k] = g[k] = m[k] = v[k] = 0.0f;
            if (mine(k)) load_element<P, G, S8>(a, o + k, p[k], g[k], m[k], v[k]);
            if (S8 && SR && mine(k)) {
                copy1(stage + Stage<P, G>::m + 8 * threadIdx.x + k, a.m + o + k);
                copy1(stage + Stage<P, G>::v + 8 * threadIdx.x + k, a.v + o + k);
            }
        }
    }
    const float m_by = S8 ? ms * s.beta1 : s.beta1, v_by = S8 ? vs * s.root_beta2 : s.beta2;
    float tr;
    update<S8>(p, g, m, v, root, tr, make_float2(m_by, m_by), make_float2(v_by, v_by), decay, r, s.eps,
               [&](uint32_t k) { return large_root_from(code_of(a.v, o + k), v_by, element<G>(a.g, o + k), r); });
    uint32_t bits[8] = {}, cut[8] = {};
    if (SR) {
        const uint32_t key = (uint32_t)first * kGolden + seed + (uint32_t)(first >> 32) * kThird;
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) bits[k] = mix(key + k * kGolden);
        if (!S8 && (uint32_t)first > 0xFFFFFFF8u) {      // 2^32 elements end in this group, or the tensor begins there
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k) bits[k] = random_bits(first + k, seed);
        }
        if (P == DTT_BF16) cut_weights(p, bits, cut);
    }
    bool settle = false;
    uint2 cm{}, cv{};
    if (S8) {
        // elements that are not the tensor's have m and root 0
        float tm = max3_nan(max3_nan(fabsf(m[0]), fabsf(m[1]), fabsf(m[2])), fabsf(m[3]), fabsf(m[4]));
        tm = max3_nan(max_nan(tm, fabsf(m[5])), fabsf(m[6]), fabsf(m[7]));
        // both over the block's lanes: even lanes go on with m's, odd ones with the roots'
        const bool odd = threadIdx.x % 2;
        float top = max_nan(odd ? tr : tm, __shfl_xor_sync(0xFFFFFFFFu, odd ? tm : tr, 1));
#pragma unroll
        for (uint32_t d = 2; d < kBlock / 8; d *= 2) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        const float other = __shfl_xor_sync(0xFFFFFFFFu, top, 1);
        tm = odd ? other : top;
        tr = odd ? top : other;
        const Scale sm = scale_from(tm), sr = scale_from(tr, kUnit);
        if (threadIdx.x % (kBlock / 8) == 0 && o < a.end) {
            a.ms[o / kBlock] = sm.scale;
            a.vs[o / kBlock] = sr.scale;
        }
        const Pair m0[2] = {pair(m[0], m[1]), pair(m[2], m[3])}, m1[2] = {pair(m[4], m[5]), pair(m[6], m[7])};
        const float2 r0[2] = {root[0], root[1]}, r1[2] = {root[2], root[3]};
        cm = make_uint2(moment_codes<SR>(m0, sm.inv, bits, s.sixteen) | poison(tm), moment_codes<SR>(m1, sm.inv, bits + 4, s.sixteen) | poison(tm));
        cv = make_uint2(root_codes<SR>(r0, sr.inv, bits, s.sixteen) | poison(tr), root_codes<SR>(r1, sr.inv, bits + 4, s.sixteen) | poison(tr));
        settle = SR && any_noise_0<8>(bits) && o < a.end;
        if (settle)                             // in the place of g, which has been taken from there
            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(stage + 16 * threadIdx.x), "f"(ms), "f"(vs), "f"(tm), "f"(tr) : "memory");
    }
    if (whole) {
        if (S8) {
            *reinterpret_cast<uint2*>(a.m + o) = cm;
            *reinterpret_cast<uint2*>(a.v + o) = cv;
        } else {
            put_group<DTT_F32>(a.m, o, m);
            put_group<DTT_F32>(a.v, o, v);
        }
        if (P == DTT_BF16 && SR)
            *reinterpret_cast<uint4*>(a.p + (uint64_t)o * 2) = make_uint4(pack_cut(cut[0], cut[1]), pack_cut(cut[2], cut[3]), pack_cut(cut[4], cut[5]), pack_cut(cut[6], cut[7]));
        else
            put_group<P>(a.p, o, p);
        if (P == DTT_F32 && a.copy) put_group<DTT_BF16>(a.copy, o, p);
        return settle;
    }
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k)
        if (mine(k))
            store_element<P, S8, SR>(a, o + k, p[k], cut[k], m[k], v[k], (k < 4 ? cm.x : cm.y) >> 8 * (k % 4), (k < 4 ? cv.x : cv.y) >> 8 * (k % 4));
    return settle;
}

// The chunks one after the other, once a thread's own copies for each have landed.  Bit i of what comes back: chunk i is
// left to settle.
template <uint32_t TURN, uint32_t P, uint32_t G, bool SR>
__device__ __forceinline__ uint32_t take_turns(const Part& a, uint32_t stage, const float (&ms)[kTurns], const float (&vs)[kTurns], uint32_t seed, float decay,
                                           const Rates& r, const Scalars& s) {
    if constexpr (TURN < kTurns) {
        if (TURN * kChunk >= a.end) return 0;
        asm volatile("cp.async.wait_group %0;" ::"n"(kTurns - 1 - TURN) : "memory");
        const bool settle = group<P, G, true, SR>(a, TURN * kChunk + 8 * threadIdx.x, stage + TURN * Stage<P, G>::bytes, ms[TURN], vs[TURN], seed, decay, r, s);
        return take_turns<TURN + 1, P, G, SR>(a, stage, ms, vs, seed, decay, r, s) | (settle ? 1u << TURN : 0u);
    }
    return 0;
}

template <uint32_t P, uint32_t G, bool S8, bool SR, uint32_t N>
__global__ void __launch_bounds__(kThreads, 4) adamw_kernel(const __grid_constant__ Batch<N> b) {
    launch_next();
    uint32_t lo = 0, hi = b.count;                  // first[lo] <= blockIdx.x < first[hi]
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) / 2;
        if (b.first[mid] <= blockIdx.x) lo = mid;
        else hi = mid;
    }
    const Tensor& t = b.t[lo];
    wait_previous();
    const Rates r = rates_of(b.s);
    const float decay = r.lr * t.decay;
    uint32_t seed = 0;
    if (SR) seed = mix(mix(b.s.seed + r.step) + t.number);
    const uint64_t start = (uint64_t)(blockIdx.x - b.first[lo]) * b.turns * kChunk;
    if (t.lead < kElements) {
        const Part a = part_of<P, G, S8>(t, start, b.turns * kChunk);
        if (S8) {
            extern __shared__ __align__(16) uint8_t stages[];
            const uint32_t stage = saddr(stages);
            float ms[kTurns], vs[kTurns];
#pragma unroll
            for (uint32_t turn = 0; turn < kTurns; ++turn) {        // those past the part's end copy nothing
                const uint32_t o = turn * kChunk + 8 * threadIdx.x;
                ms[turn] = vs[turn] = 0.0f;
                if (o < a.end) {
                    ms[turn] = a.ms[o / kBlock];
                    vs[turn] = a.vs[o / kBlock];
                }
                start_copies<P, G>(a, o, stage + turn * Stage<P, G>::bytes);
            }
            const uint32_t settle = take_turns<0, P, G, SR>(a, stage, ms, vs, seed, decay, r, b.s);
            // Only now, with nothing of the chunks in registers: one thread in 1000 has something to do here.  32M weights
            // take 65.5 us, settled among the chunks' work 10 more, and 5 less if nothing asked for a noise of 0.
            if (SR && settle) {
#pragma unroll 1
                for (uint32_t turn = 0; turn < kTurns; ++turn) {
                    if (!(settle >> turn & 1)) continue;
                    using S = Stage<P, G>;
                    const uint32_t o = turn * kChunk + 8 * threadIdx.x, at = stage + turn * S::bytes;
                    const uint4 t = shared16(at + 16 * threadIdx.x);
                    const Tops tops{__uint_as_float(t.x), __uint_as_float(t.y), __uint_as_float(t.z), __uint_as_float(t.w)};
                    settle_largest<G>(a.g, a.m, a.v, o, a.first, 1, min(a.end - o, 8u), shared8(at + S::m + 8 * threadIdx.x), shared8(at + S::v + 8 * threadIdx.x), tops, seed, r, b.s);
                }
            }
        } else {
            group<P, G, S8, SR>(a, 8 * threadIdx.x, 0, 0.0f, 0.0f, seed, decay, r, b.s);
        }
    } else {
        const uint64_t end = min(start + b.turns * kChunk, t.n);
        for (uint64_t at = start; at < end; at += kChunk) chunk_by_elements<P, G, S8, SR>(t, at, seed, decay, r, b.s);
    }
}

__global__ void adamw_advance_kernel(uint32_t* step) {
    launch_next();
    wait_previous();
    *step += 1;
}

template <uint32_t N>
struct Kernels {
    using F = void (*)(const Batch<N>);
    template <uint32_t P, uint32_t G>
    static F of(bool s8, bool sr) {
        if (s8) return sr ? adamw_kernel<P, G, true, true, N> : adamw_kernel<P, G, true, false, N>;
        if constexpr (P == DTT_BF16)
            if (sr) return adamw_kernel<P, G, false, true, N>;
        return adamw_kernel<P, G, false, false, N>;
    }
    static F of(const dtt_adamw_desc& d) {
        const bool s8 = d.state_dtype == DTT_E4M3, sr = d.stochastic != 0;
        if (d.param_dtype == DTT_BF16) return d.grad_dtype == DTT_BF16 ? of<DTT_BF16, DTT_BF16>(s8, sr) : of<DTT_BF16, DTT_F32>(s8, sr);
        return d.grad_dtype == DTT_BF16 ? of<DTT_F32, DTT_BF16>(s8, sr) : of<DTT_F32, DTT_F32>(s8, sr);
    }
};

uint32_t elem_bytes(uint32_t dt) { return dt == DTT_BF16 ? 2 : dt == DTT_F32 ? 4 : 1; }

bool misaligned(const void* p, uint32_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

// Shared memory of a chunk.
uint32_t stage_bytes(const dtt_adamw_desc& d) {
    const bool p2 = d.param_dtype == DTT_BF16, g2 = d.grad_dtype == DTT_BF16;
    if (d.state_dtype != DTT_E4M3) return 0;
    return p2 ? (g2 ? Stage<DTT_BF16, DTT_BF16>::bytes : Stage<DTT_BF16, DTT_F32>::bytes) : g2 ? Stage<DTT_F32, DTT_BF16>::bytes : Stage<DTT_F32, DTT_F32>::bytes;
}

// By groups where all of a tensor's pointers are aligned at the same element, with 8-bit states the first, where its
// blocks begin.
Tensor tensor_of(const dtt_adamw_desc& d, const dtt_adamw_tensor& t, const void* grad, uint32_t number) {
    Tensor r{static_cast<char*>(t.param), static_cast<const char*>(grad), static_cast<char*>(t.m), static_cast<char*>(t.v), t.m_scales, t.v_scales,
             static_cast<uint16_t*>(t.copy), t.n, t.weight_decay, kElements, number};
    const uint32_t pe = elem_bytes(d.param_dtype), ge = elem_bytes(d.grad_dtype), se = elem_bytes(d.state_dtype);
    const auto off = [](const void* p, uint32_t size, uint32_t lead) { return (reinterpret_cast<uintptr_t>(p) - lead * size) % std::min(16u, 8 * size) != 0; };
    for (uint32_t lead = 0; lead < (d.state_dtype == DTT_E4M3 ? 1 : kElements); ++lead) {
        if (off(r.p, pe, lead) || off(r.g, ge, lead) || off(r.m, se, lead) || off(r.v, se, lead) || (r.copy && off(r.copy, 2, lead))) continue;
        r.lead = lead;
        r.p -= lead * pe;
        r.g -= lead * ge;
        r.m -= lead * se;
        r.v -= lead * se;
        if (r.copy) r.copy -= lead;
        break;
    }
    return r;
}

}  // namespace

cudaError_t preload_adamw_kernels() {
    cudaError_t e = prepare_kernel(adamw_advance_kernel);
    for (uint32_t k = 0; k < 16 && e == cudaSuccess; ++k) {
        dtt_adamw_desc d{};
        d.param_dtype = k & 1 ? DTT_BF16 : DTT_F32;
        d.grad_dtype = k & 2 ? DTT_BF16 : DTT_F32;
        d.state_dtype = k & 4 ? (uint32_t)DTT_E4M3 : (uint32_t)DTT_F32;
        d.stochastic = k >> 3;
        const int smem = (int)(kTurns * stage_bytes(d));
        e = prepare_kernel(Kernels<kFew>::of(d));
        if (e == cudaSuccess) e = prepare_kernel(Kernels<kMany>::of(d));
        if (e == cudaSuccess) e = cudaFuncSetAttribute(Kernels<kFew>::of(d), cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(Kernels<kMany>::of(d), cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    }
    return e;
}

}  // namespace dtt

using namespace dtt;

struct dtt_adamw {
    dtt_adamw_desc d;
    std::vector<dtt_adamw_tensor> tensors;          // without the empty ones
    std::vector<uint32_t> number;                   // of each in the caller's list
    uint64_t elements = 0;                          // of all
};

namespace {

template <uint32_t N>
int run_batches(const dtt_adamw& o, const void* const* grads, const Scalars& s, cudaStream_t stream) {
    const char* who = "dtt_adamw_run";
    const auto kernel = Kernels<N>::of(o.d);
    const uint32_t turns = o.d.state_dtype == DTT_E4M3 && o.elements >= kManyElements ? kTurns : 1;
    for (size_t i = 0; i < o.tensors.size();) {
        Batch<N> b;
        uint32_t ctas = 0, k = 0;
        b.s = s;
        for (; k < N && i < o.tensors.size(); ++k, ++i) {
            const dtt_adamw_tensor& t = o.tensors[i];
            b.t[k] = tensor_of(o.d, t, grads ? grads[o.number[i]] : t.grad, o.number[i]);
            const uint64_t each = (uint64_t)turns * kChunk, need = (t.n + b.t[k].lead % kElements + each - 1) / each;
            if (ctas + need > 0x7FFFFFFFull) break;
            b.first[k] = ctas;
            ctas += (uint32_t)need;
        }
        b.first[k] = ctas;
        b.count = k;
        b.turns = turns;
        const cudaError_t e = launch(kernel, ctas, kThreads, turns * stage_bytes(o.d), 0, true, stream, b);
        if (e != cudaSuccess) return fail(DTT_ECUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    }
    return DTT_OK;
}

// Whether a buffer that is written overlaps another one; of: the tensor of the one that begins later.
bool overlap(const dtt_adamw_desc& d, const dtt_adamw_tensor* tensors, uint32_t count, uint32_t* of) {
    struct Span {
        uintptr_t from, to;
        uint32_t tensor;
        bool written;
    };
    std::vector<Span> spans;
    for (uint32_t i = 0; i < count; ++i) {
        const dtt_adamw_tensor& t = tensors[i];
        const uint64_t se = elem_bytes(d.state_dtype), blocks = (t.n + kBlock - 1) / kBlock;
        const auto add = [&](const void* p, uint64_t bytes, bool written) {
            const uintptr_t at = reinterpret_cast<uintptr_t>(p);
            if (p && bytes) spans.push_back({at, at + bytes, i, written});
        };
        add(t.param, t.n * elem_bytes(d.param_dtype), true);
        add(t.m, t.n * se, true);
        add(t.v, t.n * se, true);
        add(t.m_scales, blocks * 4, true);
        add(t.v_scales, blocks * 4, true);
        add(t.copy, t.n * 2, true);
        add(t.grad, t.n * elem_bytes(d.grad_dtype), false);
    }
    std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.from < b.from; });
    uintptr_t any = 0, written = 0;             // where those up to here end
    for (const Span& x : spans) {
        *of = x.tensor;
        if (x.from < (x.written ? any : written)) return true;
        any = std::max(any, x.to);
        if (x.written) written = std::max(written, x.to);
    }
    return false;
}

}  // namespace

extern "C" int dtt_adamw_create(const dtt_adamw_desc* d, const dtt_adamw_tensor* tensors, uint32_t count, dtt_adamw** out) {
    const char* who = "dtt_adamw_create";
    if (!out) return fail(DTT_EINVAL, "%s: null out", who);
    *out = nullptr;
    if (!d) return fail(DTT_EINVAL, "%s: null desc", who);
    for (uint32_t t : {d->param_dtype, d->grad_dtype})
        if (t != DTT_BF16 && t != DTT_F32) return fail(DTT_EINVAL, "%s: weights and gradients are bf16 or f32", who);
    if (d->state_dtype != DTT_F32 && d->state_dtype != DTT_E4M3) return fail(DTT_EINVAL, "%s: states are f32 or e4m3", who);
    if (d->stochastic > 1) return fail(DTT_EINVAL, "%s: stochastic is 0 or 1", who);
    for (double b : {d->beta1, d->beta2})
        if (!(b >= 0.0 && b < 1.0)) return fail(DTT_EINVAL, "%s: each beta must be in [0, 1)", who);
    if (!(d->eps >= 0x1p-100f) || !std::isfinite(d->eps)) return fail(DTT_EINVAL, "%s: eps must be finite and 2^-100 at least", who);
    if (count && !tensors) return fail(DTT_EINVAL, "%s: null tensors", who);
    const bool s8 = d->state_dtype == DTT_E4M3;
    const uint32_t pe = elem_bytes(d->param_dtype), ge = elem_bytes(d->grad_dtype), se = elem_bytes(d->state_dtype);
    for (uint32_t i = 0; i < count; ++i) {
        const dtt_adamw_tensor& t = tensors[i];
        if (!std::isfinite(t.weight_decay)) return fail(DTT_EINVAL, "%s: tensor %u: the decay must be finite", who, i);
        if (t.n >= kMostElements) return fail(DTT_EINVAL, "%s: tensor %u: 2^40 elements or more", who, i);
        if (t.n == 0) continue;
        if (!t.param || !t.grad || !t.m || !t.v) return fail(DTT_EINVAL, "%s: tensor %u: a null pointer", who, i);
        if (s8 ? !t.m_scales || !t.v_scales : t.m_scales || t.v_scales)
            return fail(DTT_EINVAL, "%s: tensor %u: scales go with 8-bit states, and with these alone", who, i);
        if (t.copy && d->param_dtype != DTT_F32) return fail(DTT_EINVAL, "%s: tensor %u: a copy goes with f32 weights alone", who, i);
        if (misaligned(t.param, pe) || misaligned(t.grad, ge) || misaligned(t.m, se) || misaligned(t.v, se) ||
            misaligned(t.m_scales, 4) || misaligned(t.v_scales, 4) || misaligned(t.copy, 2))
            return fail(DTT_EINVAL, "%s: tensor %u: a pointer is not aligned to its elements", who, i);
    }
    uint32_t of = 0;
    try {
        if (overlap(*d, tensors, count, &of)) return fail(DTT_EINVAL, "%s: tensor %u: a buffer overlaps another one", who, of);
    } catch (const std::bad_alloc&) {
        return fail(DTT_ENOMEM, "%s: out of host memory", who);
    }
    int rc = preload_once();
    if (rc) return rc;
    dtt_adamw* o = new (std::nothrow) dtt_adamw;
    if (!o) return fail(DTT_ENOMEM, "%s: out of host memory", who);
    try {
        o->d = *d;
        for (uint32_t i = 0; i < count; ++i)
            if (tensors[i].n) {
                o->tensors.push_back(tensors[i]);
                o->number.push_back(i);
                o->elements += tensors[i].n;
            }
    } catch (const std::bad_alloc&) {
        delete o;
        return fail(DTT_ENOMEM, "%s: out of host memory", who);
    }
    *out = o;
    return DTT_OK;
}

extern "C" int dtt_adamw_run(dtt_adamw* o, const void* const* grads, float lr, uint32_t step, const float* lr_dev,
                             uint32_t* step_dev, const float* grad_scale, cudaStream_t stream) {
    const char* who = "dtt_adamw_run";
    if (!o) return fail(DTT_EINVAL, "%s: null handle", who);
    if (!lr_dev && !std::isfinite(lr)) return fail(DTT_EINVAL, "%s: lr must be finite", who);
    if (!step_dev && step == 0) return fail(DTT_EINVAL, "%s: steps count from 1", who);
    if (misaligned(lr_dev, 4) || misaligned(step_dev, 4) || misaligned(grad_scale, 4))
        return fail(DTT_EINVAL, "%s: a pointer is not aligned to its element", who);
    if (grads)
        for (size_t i = 0; i < o->tensors.size(); ++i) {
            const void* g = grads[o->number[i]];
            if (!g || misaligned(g, elem_bytes(o->d.grad_dtype)))
                return fail(DTT_EINVAL, "%s: gradient %u is missing or not aligned to its elements", who, o->number[i]);
        }
    const dtt_adamw_desc& d = o->d;
    Scalars s{};
    s.beta1 = (float)d.beta1;
    s.beta2 = (float)d.beta2;
    const float unit = d.state_dtype == DTT_E4M3 ? kUnit : 1.0f;
    s.root_beta2 = (float)std::sqrt(d.beta2) * unit;
    s.one_less_beta1 = (float)(1.0 - d.beta1);
    s.one_less_beta2 = (float)(1.0 - d.beta2);
    s.root_one_less_beta2 = (float)std::sqrt(1.0 - d.beta2) * unit;
    s.root_by = 1.0f / unit;
    s.sixteen = 16;
    s.eps = d.eps;
    s.lr = lr;
    if (!step_dev) {
        s.lr_by_c1 = (float)((double)lr / (1.0 - std::pow(d.beta1, (double)step)));
        s.root_c2 = (float)(1.0 / std::sqrt(1.0 - std::pow(d.beta2, (double)step))) * s.root_by;
    }
    s.log_beta1 = d.beta1 > 0.0 ? (float)std::log(d.beta1) : -1e30f;
    s.log_beta2 = d.beta2 > 0.0 ? (float)std::log(d.beta2) : -1e30f;
    s.lr_dev = lr_dev;
    s.step_dev = step_dev;
    s.grad_scale = grad_scale;
    s.step = step;
    s.seed = mix(d.seed);
    if (step_dev) {
        const cudaError_t e = launch(adamw_advance_kernel, 1, 1, 0, 0, true, stream, step_dev);
        if (e != cudaSuccess) return fail(DTT_ECUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    }
    return o->tensors.size() <= kFew ? run_batches<kFew>(*o, grads, s, stream) : run_batches<kMany>(*o, grads, s, stream);
}

extern "C" void dtt_adamw_destroy(dtt_adamw* o) { delete o; }

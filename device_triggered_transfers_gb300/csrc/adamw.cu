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
};
constexpr uint32_t kElements = 8;

struct Scalars {
    float beta1, beta2, one_less_beta1, one_less_beta2, eps;
    float lr, lr_by_c1, root_c2;        // by the host's step: lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
    float log_beta1, log_beta2;         // for the device's step
    const float* lr_dev;                // or null
    const uint32_t* step_dev;           // or null
    const float* grad_scale;            // or null
    uint32_t step, seed;                // seed: mixed once
};

template <uint32_t N>
struct Batch {
    Tensor t[N];
    uint32_t first[N + 1];              // chunk that tensor i begins with
    uint32_t count, number;             // number: of t[0] in the whole list
    Scalars s;
};
// Arguments end at 32764 bytes.
constexpr uint32_t kFew = 48, kMany = 384;
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
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// What a step's formula needs, by the host or by the device's own step and rate.
struct Rates {
    float lr, lr_by_c1, root_c2, gs;
    uint32_t step;
};
__device__ __forceinline__ Rates rates_of(const Scalars& s) {
    Rates r{s.lr, s.lr_by_c1, s.root_c2, s.grad_scale ? *s.grad_scale : 1.0f, s.step};
    if (s.lr_dev || s.step_dev) {
        if (s.lr_dev) r.lr = *s.lr_dev;
        if (s.step_dev) r.step = *s.step_dev;
        const float t = (float)r.step;          // 1 - beta^t = -expm1(t log beta): nothing cancels
        r.lr_by_c1 = r.lr / -expm1f(t * s.log_beta1);
        r.root_c2 = rsqrtf(-expm1f(t * s.log_beta2));
    }
    return r;
}

// Up with the probability of what lies below: a random number in the place of the bits that are cut off, the
// noise's 16 bits (at bit 4) in that of the highest of them.  x 2^-120 has e4m3's exponents and its subnormal values
// where f32 has its own, so that the code is bits 20 to 26 of the magnitude; it comes back in the highest byte,
// without the sign.  A NaN becomes 448's code, as what is past it.  The sum comes before the shift: of the highest byte of
// (x << 4) + noise, with nothing else asked for, CUDA 13.0's compiler leaves out the x.
__device__ __forceinline__ uint32_t stochastic_code(float x, uint32_t noise) {
    return (__float_as_uint(fminf(fabsf(x), kCodeMax) * 0x1p-120f) + noise) << 4;
}
__device__ __forceinline__ uint32_t noise_m(uint32_t r) { return r >> 12 & 0xFFFF0u; }      // r's high 16 bits at bit 4
__device__ __forceinline__ uint32_t noise_v(uint32_t r) { return r << 4 & 0xFFFF0u; }       // its low ones

__device__ __forceinline__ float stochastic_bf16(float x, uint32_t noise16) {
    return isnan(x) ? x : __uint_as_float(__float_as_uint(x) + noise16);       // what is cut off is cut off when it is packed
}
__device__ __forceinline__ uint32_t pack_cut(float lo, float hi) { return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632); }

// One element.  root: sqrt(v), where states are codes.
template <bool S8>
__device__ __forceinline__ void update(float& p, float g, float& m, float& v, float& root, float keep, const Rates& r, const Scalars& s) {
    g *= r.gs;
    m = fmaf(s.beta1, m, s.one_less_beta1 * g);
    v = fmaf(s.beta2, v, (s.one_less_beta2 * g) * g);
    root = root_of(v);
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(fmaf(root, r.root_c2, s.eps)));
    p = fmaf(p, keep, -r.lr_by_c1 * (m * inv));
}

struct Scale {
    float scale, inv;
};
__device__ __forceinline__ Scale scale_from(float top) {
    const float scale = max_nan(top * (1.0f / kCodeMax), kScaleLeast);
    return {scale, 1.0f / scale};
}

// The codes of N elements' m and of their roots, which stay above zero: the next step divides by them.  noise: the
// elements' random bits.  16 bits hold two codes; poisoned: 0x7F7F where the block has a NaN, else 0.
template <bool SR>
__device__ __forceinline__ uint32_t moment_codes(float a, float b, float inv, uint32_t ra, uint32_t rb, uint32_t poisoned) {
    a *= inv;
    b *= inv;
    if (!SR) return pack_e4m3(a, b);
    const uint32_t codes = __byte_perm(stochastic_code(a, noise_m(ra)), stochastic_code(b, noise_m(rb)), 0x0073);
    const uint32_t signs = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0073) & 0x8080u;
    return (codes & 0xFFFFu) | signs | poisoned;
}
template <bool SR>
__device__ __forceinline__ uint32_t root_codes(float a, float b, float inv, uint32_t ra, uint32_t rb, uint32_t poisoned) {
    if (!SR)
        return pack_e4m3(a == 0.0f ? 0.0f : max_nan(a * inv, kCodeLeast), b == 0.0f ? 0.0f : max_nan(b * inv, kCodeLeast));
    // a root is zero or normal: twice its bits are then 2^24 at least, the place of the smallest code
    const uint32_t least_a = min(__float_as_uint(a) << 1, 1u << 24), least_b = min(__float_as_uint(b) << 1, 1u << 24);
    const uint32_t code_a = max(stochastic_code(a * inv, noise_v(ra)), least_a), code_b = max(stochastic_code(b * inv, noise_v(rb)), least_b);
    return (__byte_perm(code_a, code_b, 0x0073) & 0xFFFFu) | poisoned;
}
__device__ __forceinline__ uint32_t poisoned(float top) { return isnan(top) ? 0x7F7Fu : 0u; }

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

template <uint32_t DT>
__device__ __forceinline__ float element(const char* base, uint64_t i) {
    return DT == DTT_BF16 ? __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(base)[i] << 16) : reinterpret_cast<const float*>(base)[i];
}

// Elements i, one by one, of a tensor of which nothing is aligned: a warp's 256 neighbours, a lane every 32nd, so
// that accesses are contiguous over the warp and a block of 128 is four of each lane's.
template <uint32_t P, uint32_t G, bool S8, bool SR>
__device__ __forceinline__ void chunk_by_elements(const Tensor& t, uint64_t at, uint32_t seed, const Rates& r, const Scalars& s) {
    const uint64_t i0 = at + threadIdx.x / 32 * 256 + threadIdx.x % 32;
    const float keep = 1.0f - r.lr * t.decay;
    float p[8], g[8], m[8], v[8], root[8];
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) {
        const uint64_t i = min(i0 + 32 * k, t.n - 1);
        p[k] = element<P>(t.p, i);
        g[k] = element<G>(t.g, i);
        if (S8) {
            float none;
            unpack_e4m3(reinterpret_cast<const uint8_t*>(t.m)[i], m[k], none);
            unpack_e4m3(reinterpret_cast<const uint8_t*>(t.v)[i], v[k], none);
            m[k] *= t.ms[i / kBlock];
            v[k] *= t.vs[i / kBlock];
            v[k] *= v[k];
        } else {
            m[k] = element<DTT_F32>(t.m, i);
            v[k] = element<DTT_F32>(t.v, i);
        }
    }
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) {
        update<S8>(p[k], g[k], m[k], v[k], root[k], keep, r, s);
        if (i0 + 32 * k >= t.n) m[k] = root[k] = 0.0f;
    }
    uint32_t noise[8] = {}, code_m[4], code_v[4];
    if (SR) {
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) noise[k] = random_bits(i0 + 32 * k, seed);
    }
    if (S8) {
#pragma unroll
        for (uint32_t b = 0; b < 8; b += 4) {
            float tm = 0.0f, tr = 0.0f;
#pragma unroll
            for (uint32_t k = b; k < b + 4; ++k) {
                tm = max_nan(tm, fabsf(m[k]));
                tr = max_nan(tr, root[k]);
            }
            tm = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(tm)));
            tr = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(tr) & 0x7FFFFFFFu));
            const Scale sm = scale_from(tm), sr = scale_from(tr);
            const uint64_t i = i0 + 32 * b;
            if (threadIdx.x % 32 == 0 && i < t.n) {
                t.ms[i / kBlock] = sm.scale;
                t.vs[i / kBlock] = sr.scale;
            }
#pragma unroll
            for (uint32_t k = b; k < b + 4; k += 2) {
                code_m[k / 2] = moment_codes<SR>(m[k], m[k + 1], sm.inv, noise[k], noise[k + 1], poisoned(tm));
                code_v[k / 2] = root_codes<SR>(root[k], root[k + 1], sr.inv, noise[k], noise[k + 1], poisoned(tr));
            }
        }
    }
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) {
        const uint64_t i = i0 + 32 * k;
        if (i >= t.n) break;
        if (S8) {
            reinterpret_cast<uint8_t*>(t.m)[i] = (uint8_t)(code_m[k / 2] >> 8 * (k % 2));
            reinterpret_cast<uint8_t*>(t.v)[i] = (uint8_t)(code_v[k / 2] >> 8 * (k % 2));
        } else {
            reinterpret_cast<float*>(t.m)[i] = m[k];
            reinterpret_cast<float*>(t.v)[i] = v[k];
        }
        if (P == DTT_BF16)
            reinterpret_cast<uint16_t*>(t.p)[i] = SR ? (uint16_t)pack_cut(stochastic_bf16(p[k], noise[k] * kThird >> 16), 0.0f) : (uint16_t)pack_bf16(p[k], 0.0f);
        else
            reinterpret_cast<float*>(t.p)[i] = p[k];
        if (P == DTT_F32 && t.copy) t.copy[i] = (uint16_t)pack_bf16(p[k], 0.0f);
    }
}

// 8 neighbouring elements from `at`, of which [lo, hi) are the tensor's.
template <uint32_t DT>
__device__ __forceinline__ Raw8 raw_group(const char* base, uint64_t at) {
    return raw8(base + at * (DT == DTT_BF16 ? 2 : 4), DT);
}
template <uint32_t DT>
__device__ __forceinline__ void store_group(char* base, uint64_t at, const float (&v)[8]) {
    store8<true>(base + at * (DT == DTT_BF16 ? 2 : 4), DT, 0, 8, v);
}

// Eight neighbouring elements a thread, a block of 128 sixteen lanes.  Pointers are those of the element `lead` places before
// the first, so that every eighth from there is aligned; the groups at the tensor's ends that it does not fill go
// element by element.
template <uint32_t P, uint32_t G, bool S8, bool SR>
__device__ __forceinline__ void chunk_by_groups(const Tensor& t, uint64_t at, uint32_t seed, const Rates& r, const Scalars& s) {
    const uint64_t i = at + 8 * threadIdx.x, from = t.lead, to = t.lead + t.n;
    const bool whole = i >= from && i + 8 <= to;
    const float keep = 1.0f - r.lr * t.decay;
    float p[8], g[8], m[8], v[8], root[8];
    if (whole) {
        const Raw8 gs = raw_group<G>(t.g, i), ps = raw_group<P>(t.p, i);
        if (S8) {
            const uint2 cm = *reinterpret_cast<const uint2*>(t.m + i), cv = *reinterpret_cast<const uint2*>(t.v + i);
            const float sm = t.ms[i / kBlock], sv = t.vs[i / kBlock];
            unpack8(cm, m);
            unpack8(cv, v);
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k) {
                m[k] *= sm;
                v[k] *= sv;
                v[k] *= v[k];
            }
        } else {
            const Raw8 a = raw_group<DTT_F32>(t.m, i), b = raw_group<DTT_F32>(t.v, i);
            expand8(a, DTT_F32, m);
            expand8(b, DTT_F32, v);
        }
        expand8(gs, G, g);
        expand8(ps, P, p);
    } else {
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) {
            p[k] = g[k] = m[k] = v[k] = 0.0f;
            if (i + k < from || i + k >= to) continue;
            p[k] = element<P>(t.p, i + k);
            g[k] = element<G>(t.g, i + k);
            if (S8) {
                float none;
                unpack_e4m3(reinterpret_cast<const uint8_t*>(t.m)[i + k], m[k], none);
                unpack_e4m3(reinterpret_cast<const uint8_t*>(t.v)[i + k], v[k], none);
                m[k] *= t.ms[i / kBlock];
                v[k] *= t.vs[i / kBlock];
                v[k] *= v[k];
            } else {
                m[k] = element<DTT_F32>(t.m, i + k);
                v[k] = element<DTT_F32>(t.v, i + k);
            }
        }
    }
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) update<S8>(p[k], g[k], m[k], v[k], root[k], keep, r, s);
    uint32_t noise[8] = {};
    if (SR) {
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) noise[k] = random_bits(i + k - from, seed);
    }
    uint2 cm{}, cv{};
    if (S8) {
        float tm = 0.0f, tr = 0.0f;             // elements that are not the tensor's have m and root 0
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) {
            tm = max_nan(tm, fabsf(m[k]));
            tr = max_nan(tr, root[k]);
        }
#pragma unroll
        for (uint32_t d = 1; d < kBlock / 8; d *= 2) {
            tm = max_nan(tm, __shfl_xor_sync(0xFFFFFFFFu, tm, d));
            tr = max_nan(tr, __shfl_xor_sync(0xFFFFFFFFu, tr, d));
        }
        const Scale sm = scale_from(tm), sr = scale_from(tr);
        if (threadIdx.x % (kBlock / 8) == 0 && i < to) {
            t.ms[i / kBlock] = sm.scale;
            t.vs[i / kBlock] = sr.scale;
        }
        uint32_t c[4], d[4];
#pragma unroll
        for (uint32_t k = 0; k < 8; k += 2) {
            c[k / 2] = moment_codes<SR>(m[k], m[k + 1], sm.inv, noise[k], noise[k + 1], poisoned(tm));
            d[k / 2] = root_codes<SR>(root[k], root[k + 1], sr.inv, noise[k], noise[k + 1], poisoned(tr));
        }
        cm = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
        cv = make_uint2(d[0] | d[1] << 16, d[2] | d[3] << 16);
    }
    float q[8];
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) q[k] = P == DTT_BF16 && SR ? stochastic_bf16(p[k], noise[k] * kThird >> 16) : p[k];
    if (whole) {
        if (S8) {
            *reinterpret_cast<uint2*>(t.m + i) = cm;
            *reinterpret_cast<uint2*>(t.v + i) = cv;
        } else {
            store_group<DTT_F32>(t.m, i, m);
            store_group<DTT_F32>(t.v, i, v);
        }
        if (P == DTT_BF16 && SR)
            *reinterpret_cast<uint4*>(t.p + 2 * i) = make_uint4(pack_cut(q[0], q[1]), pack_cut(q[2], q[3]), pack_cut(q[4], q[5]), pack_cut(q[6], q[7]));
        else
            store_group<P>(t.p, i, p);
        if (P == DTT_F32 && t.copy) store_group<DTT_BF16>(reinterpret_cast<char*>(t.copy), i, p);
        return;
    }
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) {
        if (i + k < from || i + k >= to) continue;
        if (S8) {
            reinterpret_cast<uint8_t*>(t.m)[i + k] = (uint8_t)((k < 4 ? cm.x : cm.y) >> 8 * (k % 4));
            reinterpret_cast<uint8_t*>(t.v)[i + k] = (uint8_t)((k < 4 ? cv.x : cv.y) >> 8 * (k % 4));
        } else {
            reinterpret_cast<float*>(t.m)[i + k] = m[k];
            reinterpret_cast<float*>(t.v)[i + k] = v[k];
        }
        if (P == DTT_BF16)
            reinterpret_cast<uint16_t*>(t.p)[i + k] = SR ? (uint16_t)pack_cut(q[k], 0.0f) : (uint16_t)pack_bf16(p[k], 0.0f);
        else
            reinterpret_cast<float*>(t.p)[i + k] = p[k];
        if (P == DTT_F32 && t.copy) t.copy[i + k] = (uint16_t)pack_bf16(p[k], 0.0f);
    }
}

template <uint32_t P, uint32_t G, bool S8, bool SR, uint32_t N>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Batch<N> b) {
    launch_next();
    uint32_t lo = 0, hi = b.count;                  // first[lo] <= blockIdx.x < first[hi]
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) / 2;
        if (b.first[mid] <= blockIdx.x) lo = mid;
        else hi = mid;
    }
    const Tensor& t = b.t[lo];
    const uint64_t at = (uint64_t)(blockIdx.x - b.first[lo]) * kChunk;
    wait_previous();
    const Rates r = rates_of(b.s);
    uint32_t seed = 0;
    if (SR) seed = mix(mix(b.s.seed + r.step) + b.number + lo);
    if (t.lead < kElements) chunk_by_groups<P, G, S8, SR>(t, at, seed, r, b.s);
    else chunk_by_elements<P, G, S8, SR>(t, at, seed, r, b.s);
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

// By groups where all of a tensor's pointers are aligned at the same element, with 8-bit states the first, where its
// blocks begin.
Tensor tensor_of(const dtt_adamw_desc& d, const dtt_adamw_tensor& t, const void* grad) {
    Tensor r{static_cast<char*>(t.param), static_cast<const char*>(grad), static_cast<char*>(t.m), static_cast<char*>(t.v), t.m_scales, t.v_scales,
             static_cast<uint16_t*>(t.copy), t.n, t.weight_decay, kElements};
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
        e = prepare_kernel(Kernels<kFew>::of(d));
        if (e == cudaSuccess) e = prepare_kernel(Kernels<kMany>::of(d));
    }
    return e;
}

}  // namespace dtt

using namespace dtt;

struct dtt_adamw {
    dtt_adamw_desc d;
    std::vector<dtt_adamw_tensor> tensors;          // without the empty ones
    std::vector<uint32_t> number;                   // of each in the caller's list
};

namespace {

template <uint32_t N>
int run_batches(const dtt_adamw& o, const void* const* grads, const Scalars& s, cudaStream_t stream) {
    const char* who = "dtt_adamw_run";
    const auto kernel = Kernels<N>::of(o.d);
    for (size_t i = 0; i < o.tensors.size();) {
        Batch<N> b;
        uint32_t chunks = 0, k = 0;
        b.s = s;
        b.number = o.number[i];
        for (; k < N && i < o.tensors.size(); ++k, ++i) {
            // an empty tensor between two of a launch would shift the numbers after it
            if (o.number[i] != b.number + k) break;
            const dtt_adamw_tensor& t = o.tensors[i];
            b.t[k] = tensor_of(o.d, t, grads ? grads[o.number[i]] : t.grad);
            const uint64_t need = (t.n + b.t[k].lead % kElements + kChunk - 1) / kChunk;
            if (chunks + need > 0x7FFFFFFFull) break;
            b.first[k] = chunks;
            chunks += (uint32_t)need;
        }
        b.first[k] = chunks;
        b.count = k;
        const cudaError_t e = launch(kernel, chunks, kThreads, 0, 0, true, stream, b);
        if (e != cudaSuccess) return fail(DTT_ECUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    }
    return DTT_OK;
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
    s.one_less_beta1 = (float)(1.0 - d.beta1);
    s.one_less_beta2 = (float)(1.0 - d.beta2);
    s.eps = d.eps;
    s.lr = lr;
    if (!step_dev) {
        s.lr_by_c1 = (float)((double)lr / (1.0 - std::pow(d.beta1, (double)step)));
        s.root_c2 = (float)(1.0 / std::sqrt(1.0 - std::pow(d.beta2, (double)step)));
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

// Device helpers shared by the operators' kernels (norm.cu, ortho.cu): elements of rows as f32, and
// the mbarrier basics.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "dtt_ops.h"

namespace dtt {

// SMs of the GPU that the workspaces' sizes and the rules on sizes are made for, both asked for without a device.
// Launches go by the device's own count; on another count the results hold and the rules are less apt.
constexpr uint32_t kSms = 152;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {      // 16 bits
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// The larger of two, NaN if either is: a NaN in a row must reach its scale.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// Columns c .. c + 7 of a row, zeros from `cols` on.  VEC: the row is 16-byte aligned, so a whole
// chunk is one or two 16-byte loads.
template <bool VEC>
__device__ __forceinline__ void load8(const char* row, uint32_t dt, uint32_t c, uint32_t cols, float (&v)[8]) {
    if (VEC && c + 8 <= cols) {
        if (dt == DTT_BF16) {
            const uint4 q = *reinterpret_cast<const uint4*>(row + (uint64_t)c * 2);
            v[0] = bf16_lo(q.x); v[1] = bf16_hi(q.x); v[2] = bf16_lo(q.y); v[3] = bf16_hi(q.y);
            v[4] = bf16_lo(q.z); v[5] = bf16_hi(q.z); v[6] = bf16_lo(q.w); v[7] = bf16_hi(q.w);
        } else {
            const float4 a = *reinterpret_cast<const float4*>(row + (uint64_t)c * 4);
            const float4 b = *reinterpret_cast<const float4*>(row + (uint64_t)c * 4 + 16);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        }
        return;
    }
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) {
        v[k] = 0.0f;
        if (c + k < cols) {
            if (dt == DTT_BF16)
                v[k] = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[c + k] << 16);
            else
                v[k] = reinterpret_cast<const float*>(row)[c + k];
        }
    }
}

template <bool VEC>
__device__ __forceinline__ void store8(char* row, uint32_t dt, uint32_t c, uint32_t cols, const float (&v)[8]) {
    if (VEC && c + 8 <= cols) {
        if (dt == DTT_BF16) {
            *reinterpret_cast<uint4*>(row + (uint64_t)c * 2) =
                make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
        } else if (dt == DTT_F32) {
            *reinterpret_cast<float4*>(row + (uint64_t)c * 4) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(row + (uint64_t)c * 4 + 16) = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *reinterpret_cast<uint2*>(row + c) =
                make_uint2(pack_e4m3(v[0], v[1]) | pack_e4m3(v[2], v[3]) << 16,
                           pack_e4m3(v[4], v[5]) | pack_e4m3(v[6], v[7]) << 16);
        }
        return;
    }
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k)
        if (c + k < cols) {
            if (dt == DTT_BF16)
                reinterpret_cast<uint16_t*>(row)[c + k] = (uint16_t)pack_bf16(v[k], 0.0f);
            else if (dt == DTT_F32)
                reinterpret_cast<float*>(row)[c + k] = v[k];
            else
                reinterpret_cast<uint8_t*>(row)[c + k] = (uint8_t)pack_e4m3(v[k], 0.0f);
        }
}

__device__ __forceinline__ float load1(const char* row, uint32_t dt, uint32_t c) {
    return dt == DTT_BF16 ? __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[c] << 16)
                          : reinterpret_cast<const float*>(row)[c];
}

__device__ __forceinline__ void store1(char* row, uint32_t dt, uint32_t c, float v) {
    if (dt == DTT_BF16)
        reinterpret_cast<uint16_t*>(row)[c] = (uint16_t)pack_bf16(v, 0.0f);
    else if (dt == DTT_F32)
        reinterpret_cast<float*>(row)[c] = v;
    else
        reinterpret_cast<uint8_t*>(row)[c] = (uint8_t)pack_e4m3(v, 0.0f);
}

__device__ __forceinline__ uint32_t saddr(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// 8 columns of bf16 or f32, as loaded and as f32.  Apart, because a load behind a branch of its own waits
// for the one before it only where that one's values are looked at in between.
struct Raw8 {
    uint4 a, b;                 // b: f32 alone
};
__device__ __forceinline__ Raw8 raw8(const char* at, uint32_t dt) {
    Raw8 q{};
    q.a = *reinterpret_cast<const uint4*>(at);
    if (dt != DTT_BF16) q.b = *reinterpret_cast<const uint4*>(at + 16);
    return q;
}
__device__ __forceinline__ void expand8(const Raw8& q, uint32_t dt, float (&v)[8]) {
    if (dt == DTT_BF16) {
        v[0] = bf16_lo(q.a.x); v[1] = bf16_hi(q.a.x); v[2] = bf16_lo(q.a.y); v[3] = bf16_hi(q.a.y);
        v[4] = bf16_lo(q.a.z); v[5] = bf16_hi(q.a.z); v[6] = bf16_lo(q.a.w); v[7] = bf16_hi(q.a.w);
    } else {
        v[0] = __uint_as_float(q.a.x); v[1] = __uint_as_float(q.a.y); v[2] = __uint_as_float(q.a.z); v[3] = __uint_as_float(q.a.w);
        v[4] = __uint_as_float(q.b.x); v[5] = __uint_as_float(q.b.y); v[6] = __uint_as_float(q.b.z); v[7] = __uint_as_float(q.b.w);
    }
}

// N elements at rows[n], column c[n], as f32.  The loads go out together: they are unconditional and the
// type is decided once, since a load behind a branch of its own waits for the one before it.
template <uint32_t N>
__device__ __forceinline__ void gather(const char* const (&rows)[N], uint32_t dt, const uint32_t (&c)[N], float (&v)[N]) {
    if (dt == DTT_BF16) {
        uint16_t raw[N];
#pragma unroll
        for (uint32_t n = 0; n < N; ++n) raw[n] = reinterpret_cast<const uint16_t*>(rows[n])[c[n]];
#pragma unroll
        for (uint32_t n = 0; n < N; ++n) v[n] = __uint_as_float((uint32_t)raw[n] << 16);
    } else {
#pragma unroll
        for (uint32_t n = 0; n < N; ++n) v[n] = reinterpret_cast<const float*>(rows[n])[c[n]];
    }
}

// The launch after this one may begin (it waits for this one's results itself), and: everything the
// launch before wrote is there, and it reads nothing any more.
__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launched so that its set-up overlaps the end of the kernel before it (for which it waits with
// wait_previous), unless `overlap` says otherwise.  cluster: CTAs of a cluster, 0 where the kernel itself
// says.
template <class... Params, class... Args>
cudaError_t launch(void (*kernel)(Params...), dim3 grid, dim3 threads, uint32_t smem, uint32_t cluster, bool overlap, cudaStream_t stream,
                   const Args&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = threads;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = overlap;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

}  // namespace dtt

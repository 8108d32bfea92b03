// ssm_common.cuh -- loads and stores of states and rows shared by the scan kernels.
#pragma once

#include "layer_common.cuh"

namespace lar {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// SPL (4 or 8) elements st apart, fp32 or bf16, vector loads where they fit.
template <int SPL>
__device__ __forceinline__ void load_row(const void* base, int64_t off, int64_t st, int dt, float* f) {
#pragma unroll
    for (int i = 0; i < SPL; i += 4) ld_in4(base, off + i * st, st, dt, f + i);
}

// A log2(e): the decay of a step s is 2^(s a2).
template <int SPL>
__device__ __forceinline__ void load_a2(const SsmParams& p, int d, int n0, float* a2) {
    load_row<SPL>(p.A, d * p.as[0] + n0 * p.as[1], p.as[1], LAR_F32, a2);
#pragma unroll
    for (int i = 0; i < SPL; ++i) a2[i] *= kLog2e;
}

// SPL states of channel d from n0 on; the pool's rows are 16-byte aligned.
template <int SPL>
__device__ __forceinline__ void load_states(const SsmParams& p, int64_t slot, int d, int n0, float* h) {
    if (slot < 0) {
#pragma unroll
        for (int i = 0; i < SPL; ++i) h[i] = 0.f;
        return;
    }
    const int64_t off = slot * p.ps[0] + d * p.ps[1] + n0;
    if (p.pool_dt == LAR_F32) {
#pragma unroll
        for (int i = 0; i < SPL; i += 4) {
            const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p.pool) + off + i);
            h[i] = v.x; h[i + 1] = v.y; h[i + 2] = v.z; h[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < SPL; i += 4) {
            const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const unsigned short*>(p.pool) + off + i);
            h[i] = __uint_as_float(v.x << 16);
            h[i + 1] = __uint_as_float(v.x & 0xffff0000u);
            h[i + 2] = __uint_as_float(v.y << 16);
            h[i + 3] = __uint_as_float(v.y & 0xffff0000u);
        }
    }
}

// Rounded to nearest even, once, into a bf16 pool.
template <int SPL>
__device__ __forceinline__ void store_states(const SsmParams& p, int64_t slot, int d, int n0, const float* h) {
    if (slot < 0) return;
    const int64_t off = slot * p.ps[0] + d * p.ps[1] + n0;
    if (p.pool_dt == LAR_F32) {
#pragma unroll
        for (int i = 0; i < SPL; i += 4)
            st_state(reinterpret_cast<float4*>(static_cast<float*>(p.pool) + off + i),
                     make_float4(h[i], h[i + 1], h[i + 2], h[i + 3]));
    } else if constexpr (SPL == 8) {
        st_state(reinterpret_cast<uint4*>(static_cast<unsigned short*>(p.pool) + off), pack8(h));
    } else {
        st_state(reinterpret_cast<uint2*>(static_cast<unsigned short*>(p.pool) + off),
                 make_uint2(pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3])));
    }
}

}  // namespace lar

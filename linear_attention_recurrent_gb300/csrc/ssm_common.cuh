// ssm_common.cuh -- loads and stores of states and rows shared by the scan kernels.
#pragma once

#include "layer_common.cuh"

namespace lar {

// log(1 + e^v) = max(v, 0) + log1p(u), u = e^-|v| in (0, 1].  log1p(u) / u is
// a polynomial of degree 8, fitted to the relative error (Chebyshev nodes,
// Lawson's weights): off by 2e-7 at most in fp32 arithmetic, for small u too,
// where 1 + u would lose it.  Small steps matter: most are near 0.001.
__device__ __forceinline__ float softplus1(float v) {
    const float u = exp2_f(-fabsf(v) * kLog2e);
    float q = fmaf(0.005232624243944883f, u, -0.029504956677556038f);
    q = fmaf(q, u, 0.07822549343109131f);
    q = fmaf(q, u, -0.1366320699453354f);
    q = fmaf(q, u, 0.1910598874092102f);
    q = fmaf(q, u, -0.2484297752380371f);
    q = fmaf(q, u, 0.3331909477710724f);
    q = fmaf(q, u, -0.4999949336051941f);
    q = fmaf(q, u, 0.9999999403953552f);
    return fmaf(q, u, fmaxf(v, 0.f));
}

// SPL (a multiple of 4) elements st apart, fp32 or bf16, vector loads where they fit.
template <int SPL>
__device__ __forceinline__ void load_row(const void* base, int64_t off, int64_t st, int dt, float* f) {
#pragma unroll
    for (int i = 0; i < SPL; i += 4) ld_in4(base, off + i * st, st, dt, f + i);
}

// A log2(e): the decay of a step s is 2^(s a2).  A finite rate stays finite (the least number
// is a usual one for "forget"): a step of 0 times it is 0, and any step of 1e-36 or more
// forgets with the largest a2 as with 1.44 times it.
template <int SPL>
__device__ __forceinline__ void load_a2(const SsmParams& p, int d, int n0, float* a2) {
    load_row<SPL>(p.A, d * p.as[0] + n0 * p.as[1], p.as[1], LAR_F32, a2);
#pragma unroll
    for (int i = 0; i < SPL; ++i) {
        const float a = a2[i], most = 3.402823466e38f;
        a2[i] = a * kLog2e;
        if (fabsf(a) <= most) a2[i] = fminf(fmaxf(a2[i], -most), most);
    }
}

// 16 bytes of channel d's states from n0 on, as they lie in the pool; zero
// without a slot.
__device__ __forceinline__ uint4 load_raw(const SsmParams& p, int64_t slot, int d, int n0) {
    if (slot < 0) return make_uint4(0u, 0u, 0u, 0u);
    const int64_t off = slot * p.ps[0] + d * p.ps[1] + n0;
    return *reinterpret_cast<const uint4*>(static_cast<const char*>(p.pool) + off * (p.pool_dt == LAR_F32 ? 4 : 2));
}

// 16 bytes of states from or to p, rounded to nearest even, once, where they are bf16
template <int SPL>
__device__ __forceinline__ void store_raw(void* p, const float* h) {
    if constexpr (SPL == 4) st_state(static_cast<float4*>(p), make_float4(h[0], h[1], h[2], h[3]));
    else st_state(static_cast<uint4*>(p), pack8(h));
}

// 4 fp32 or 8 bf16 of them
template <int SPL>
__device__ __forceinline__ void raw_states(const uint4 u, float* h) {
    if constexpr (SPL == 8) {
        unpack8(u, h);
    } else {
        h[0] = __uint_as_float(u.x);
        h[1] = __uint_as_float(u.y);
        h[2] = __uint_as_float(u.z);
        h[3] = __uint_as_float(u.w);
    }
}

// SPL (a multiple of 4) states of channel d from n0 on; the pool's rows are 16-byte aligned.
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
    } else if constexpr (SPL % 8 == 0) {
#pragma unroll
        for (int i = 0; i < SPL; i += 8)
            st_state(reinterpret_cast<uint4*>(static_cast<unsigned short*>(p.pool) + off + i), pack8(h + i));
    } else {
#pragma unroll
        for (int i = 0; i < SPL; i += 4)
            st_state(reinterpret_cast<uint2*>(static_cast<unsigned short*>(p.pool) + off + i),
                     make_uint2(pack_bf16x2(h[i], h[i + 1]), pack_bf16x2(h[i + 2], h[i + 3])));
    }
}

}  // namespace lar

// layer_common.cuh -- device helpers shared by the convolution, scan and
// verification kernels: slot resolution, spans, 8-channel loads and stores.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "decode_kernel.cuh"
#include "layer_params.h"

namespace lar {

// Order after the previous kernel on the stream (launched with programmatic
// serialization); its successor may be scheduled from here on.
__device__ __forceinline__ void stream_order() {
#if LAR_PDL
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
#endif
}

// `cluster`: blocks of a cluster along x (1: none).
template <typename... Kp, typename... Args>
lar_status launch_ordered(void (*kern)(Kp...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t stream,
                          const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int na = 0;
#if LAR_PDL
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na++].val.programmaticStreamSerializationAllowed = 1;
#endif
    if (cluster > 1) {
        attr[na].id = cudaLaunchAttributeClusterDimension;
        attr[na].val.clusterDim.x = static_cast<unsigned>(cluster);
        attr[na].val.clusterDim.y = 1;
        attr[na++].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = na;
    return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? LAR_OK : LAR_ERR_LAUNCH;
}

__device__ __forceinline__ void flag_err(int32_t* word, int32_t bits) {
    if (word && bits) atomicOr(word, bits);
}

// The slot that sequence b starts from; -1: a zero state.
__device__ __forceinline__ int64_t read_slot(const SlotParams& s, int b, int32_t* bits) {
    int64_t slot;
    if (s.nacc) {
        const int64_t n = ld_idx(s.nacc, b * s.na_s, s.na_dt);
        if (n < 1 || n > s.T) {
            *bits |= LAR_DEVERR_ACCEPTED;
            return -1;
        }
        slot = ld_idx(s.tslot, b * s.tsl_s[0] + (n - 1) * s.tsl_s[1], s.tsl_dt);
    } else {
        slot = ld_idx(s.ridx, b * s.ri_s, s.ri_dt);
    }
    if (slot >= s.P) {
        *bits |= LAR_DEVERR_READ_SLOT;
        return -1;
    }
    return slot;
}

// The slot that takes the state of sequence b after its token t (per-token
// slots) or after its last one; -1: none.
__device__ __forceinline__ int64_t write_slot(const SlotParams& s, int b, int t, int32_t* bits) {
    const int64_t slot = s.tslot ? ld_idx(s.tslot, b * s.tsl_s[0] + t * s.tsl_s[1], s.tsl_dt)
                         : s.widx ? ld_idx(s.widx, b * s.wi_s, s.wi_dt)
                                  : ld_idx(s.ridx, b * s.ri_s, s.ri_dt);
    if (slot >= s.P) {
        *bits |= LAR_DEVERR_WRITE_SLOT;
        return -1;
    }
    return slot;
}

// Span n of a packed call.  A reversed span or one that leaves the token arrays
// counts as empty.
__device__ __forceinline__ void span_of(const SlotParams& s, int n, int* begin, int* len, int32_t* bits) {
    const int64_t a = ld_idx(s.cu, n * s.cu_s, s.cu_dt), e = ld_idx(s.cu, (n + 1) * s.cu_s, s.cu_dt);
    const bool ok = a >= 0 && a <= e && e <= s.ntok;
    if (!ok) *bits |= LAR_DEVERR_SEQLEN;
    *begin = ok ? static_cast<int>(a) : 0;
    *len = ok ? static_cast<int>(e - a) : 0;
}

// Cluster of blocks: this block's place in it, its size, a barrier over it, and
// the address that `p` of this block's shared memory has in block `rank`.
__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ unsigned cluster_size() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// its two halves
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ unsigned peer_addr(const void* p, unsigned rank) {
    const unsigned local = static_cast<unsigned>(__cvta_generic_to_shared(p));
    unsigned remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
    return remote;
}

__device__ __forceinline__ float ld_peer_f32(const float* p, unsigned rank) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(peer_addr(p, rank)));
    return v;
}

__device__ __forceinline__ void st_peer_f32(float* p, unsigned rank, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(peer_addr(p, rank)), "f"(v) : "memory");
}

__device__ __forceinline__ float4 ld_peer_f32x4(const float* p, unsigned rank) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(peer_addr(p, rank)));
    return v;
}

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 numbers in a register pair: one instruction issued for two products.
using f32x2 = unsigned long long;

__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ void unpack2(f32x2 v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}

__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ f32x2 ex2_2(f32x2 a) {
    float lo, hi;
    unpack2(a, lo, hi);
    return pack2(exp2_f(lo), exp2_f(hi));
}

// 8 neighbouring channels as fp32, 16-byte loads; NC: through the read-only path
// (never for the pool, which the same call writes).
template <bool NC>
__device__ __forceinline__ uint4 ld16(const void* p) {
    return NC ? __ldg(static_cast<const uint4*>(p)) : *static_cast<const uint4*>(p);
}

__device__ __forceinline__ void unpack8(const uint4 u, float* f) {
    const unsigned w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

template <bool NC>
__device__ __forceinline__ void ld8(const void* base, int64_t off, int dt, float* f) {
    if (dt == LAR_BF16) {
        unpack8(ld16<NC>(static_cast<const unsigned short*>(base) + off), f);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4 u = ld16<NC>(static_cast<const float*>(base) + off + 4 * h);
            f[4 * h] = __uint_as_float(u.x);
            f[4 * h + 1] = __uint_as_float(u.y);
            f[4 * h + 2] = __uint_as_float(u.z);
            f[4 * h + 3] = __uint_as_float(u.w);
        }
    }
}

__device__ __forceinline__ uint4 pack8(const float* f) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ void st8(void* base, int64_t off, int dt, const float* f) {
    if (dt == LAR_BF16) {
        *reinterpret_cast<uint4*>(static_cast<unsigned short*>(base) + off) = pack8(f);
    } else {
        float4* d = reinterpret_cast<float4*>(static_cast<float*>(base) + off);
        d[0] = make_float4(f[0], f[1], f[2], f[3]);
        d[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
}

// One element of the pool (a plain load: see ld16).
__device__ __forceinline__ float ld_pool(const void* base, int64_t off, int dt) {
    return dt == LAR_F32 ? static_cast<const float*>(base)[off]
                         : bf16_bits_to_float(static_cast<const unsigned short*>(base)[off]);
}

// 8 neighbouring values, asked for (raw) and widened: two steps, so that many are
// on their way at once
template <typename T, bool NC = true>
struct Eight {
    uint4 u[sizeof(T) / 2];
    __device__ __forceinline__ void load(const void* base, int64_t i) {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(base) + i);
#pragma unroll
        for (int h = 0; h < static_cast<int>(sizeof(T) / 2); ++h) u[h] = NC ? __ldg(src + h) : src[h];
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int h = 0; h < static_cast<int>(sizeof(T) / 2); ++h) u[h] = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void store(void* base, int64_t i) const {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(base) + i);
#pragma unroll
        for (int h = 0; h < static_cast<int>(sizeof(T) / 2); ++h) dst[h] = u[h];
    }
    __device__ __forceinline__ void widen(float* f) const {
        if constexpr (sizeof(T) == 2) {
            unpack8(u[0], f);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                f[4 * h] = __uint_as_float(u[h].x);
                f[4 * h + 1] = __uint_as_float(u[h].y);
                f[4 * h + 2] = __uint_as_float(u[h].z);
                f[4 * h + 3] = __uint_as_float(u[h].w);
            }
        }
    }
};

__device__ __forceinline__ float rcp_f(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// y / (1 + e^-y).  Both SFU steps are good to 2 ulp; where e^-y overflows, the
// reciprocal is 0 and so is the limit.
__device__ __forceinline__ float silu_f(float y) { return y * rcp_f(1.f + exp2_f(-kLog2e * y)); }

}  // namespace lar

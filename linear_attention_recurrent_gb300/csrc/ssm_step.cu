// ssm_step.cu -- the selective state space recurrence for the tokens of one step
// (ssm_decode, ssm_decode_tokens).  Per token and channel d, with N states:
//
//     s = softplus(dt[d] + dt_bias[d])  (or dt[d])
//     h[n] <- exp(s A[d, n]) h[n] + s x[d] B[g, n]
//     out = (sum_n C[g, n] h[n] + D[d] x[d]) silu(z[d])
//
// Bound by the state's way through memory, 2 N words a channel against 4
// activations.
#include "ssm_common.cuh"

namespace lar {

namespace {

constexpr int kThreads = 128;

// SPL states a lane, 16 bytes of the pool; N / SPL lanes a channel.
template <int N, int SPL>
__global__ void __launch_bounds__(kThreads) ssm_step_kernel(const SsmParams p) {
    constexpr int LPC = N / SPL;
    constexpr int CPB = kThreads / LPC;
    const int b = blockIdx.y, lane = threadIdx.x % LPC, d = blockIdx.x * CPB + threadIdx.x / LPC;
    const int n0 = lane * SPL;
    stream_order();
    int32_t bits = 0;
    const int64_t slot = read_slot(p.s, b, &bits);
    const bool live = d < p.D;   // the group's lanes alike
    const int dc = live ? d : p.D - 1;
    float h[SPL], a2[SPL];
    load_states<SPL>(p, slot, dc, n0, h);
    load_a2<SPL>(p, dc, n0, a2);
    const float bias = p.dt_bias ? p.dt_bias[dc * p.dtb_s] : 0.f;
    const float skip = p.skip ? p.skip[dc * p.skip_s] : 0.f;
    const int g = dc / p.per_group;
    for (int t = 0; t < p.s.T; ++t) {
        const float x = ld_in(p.x, b * p.xs[0] + t * p.xs[1] + dc * p.xs[2], p.x_dt);
        float s = ld_in(p.dt, b * p.ds[0] + t * p.ds[1] + dc * p.ds[2], p.dt_dt);
        if (p.softplus) s = softplus_fast(s + bias);
        float Bv[SPL], Cv[SPL];
        load_row<SPL>(p.B, b * p.bs[0] + t * p.bs[1] + g * p.bs[2] + n0 * p.bs[3], p.bs[3], p.B_dt, Bv);
        load_row<SPL>(p.C, b * p.cs[0] + t * p.cs[1] + g * p.cs[2] + n0 * p.cs[3], p.cs[3], p.C_dt, Cv);
        const float sx = s * x;
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < SPL; ++i) {
            h[i] = fmaf(exp2_f(s * a2[i]), h[i], sx * Bv[i]);
            y = fmaf(Cv[i], h[i], y);
        }
#pragma unroll
        for (int off = LPC / 2; off > 0; off >>= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
        if (live && lane == 0) {
            y = fmaf(skip, x, y);
            if (p.z) y *= silu_f(ld_in(p.z, b * p.zs[0] + t * p.zs[1] + dc * p.zs[2], p.z_dt));
            st_out(p.out, b * p.os[0] + t * p.os[1] + dc * p.os[2], p.out_dt, y);
        }
        if (p.s.tslot) {
            const int64_t w = write_slot(p.s, b, t, &bits);
            if (live) store_states<SPL>(p, w, d, n0, h);
        }
    }
    if (!p.s.tslot) {
        const int64_t w = write_slot(p.s, b, 0, &bits);
        if (live) store_states<SPL>(p, w, d, n0, h);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) flag_err(p.s.dev_err, bits);
}

template <int N, int SPL>
lar_status go(const SsmParams& p, cudaStream_t st) {
    constexpr int CPB = kThreads / (N / SPL);
    return launch_ordered(ssm_step_kernel<N, SPL>, dim3((p.D + CPB - 1) / CPB, p.s.n), kThreads, 0, 1, st, p);
}

}  // namespace

lar_status launch_ssm_step(const SsmParams& p, void* stream) {
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool f32 = p.pool_dt == LAR_F32;
    switch (p.N) {
        case 16: return f32 ? go<16, 4>(p, st) : go<16, 8>(p, st);
        case 32: return f32 ? go<32, 4>(p, st) : go<32, 8>(p, st);
        case 64: return f32 ? go<64, 4>(p, st) : go<64, 8>(p, st);
        default: return f32 ? go<128, 4>(p, st) : go<128, 8>(p, st);
    }
}

}  // namespace lar

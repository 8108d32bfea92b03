// ssm_prefill.cu -- the selective scan over packed spans (ssm_prefill).
//
// One block takes a block of channels of one span and walks its tokens, tile by
// tile, with the states in registers: a channel's N states lie SPL to a lane on
// N / SPL neighbouring lanes.  Per tile the block first turns dt and x into the
// step s and s x for every (token, channel) in shared memory, with B and C
// beside them in fp32, then runs the recurrence, then applies the skip and the
// gate to the sums.
#include "ssm_common.cuh"

namespace lar {

namespace {

constexpr int kThreads = 128;

template <int N, int SPL>
struct Geo {
    static constexpr int LPC = N / SPL;              // lanes of a channel
    static constexpr int CH = kThreads / LPC;        // channels of a block
    static constexpr int TT = 32;                    // tokens of a tile
    static constexpr size_t smem = static_cast<size_t>(TT) * (CH * 8 + 2 * N * 4);
};

template <int N, int SPL>
__global__ void __launch_bounds__(kThreads) ssm_prefill_kernel(const SsmParams p) {
    using G = Geo<N, SPL>;
    constexpr int LPC = G::LPC, CH = G::CH, TT = G::TT;
    extern __shared__ __align__(16) unsigned char smem[];
    float2* step = reinterpret_cast<float2*>(smem);             // [TT][CH]: s, s x; then the sum y in .x
    float* Bs = reinterpret_cast<float*>(step + TT * CH);       // [TT][N]
    float* Cs = Bs + TT * N;
    const int tid = threadIdx.x, ch = tid / LPC, lane = tid % LPC, n0 = lane * SPL;
    const int seq = blockIdx.y;
    // channel blocks do not straddle groups: block i of group g
    const int per_g = (p.per_group + CH - 1) / CH;
    const int g = blockIdx.x / per_g, d0 = g * p.per_group + (blockIdx.x % per_g) * CH;
    const int nch = min(CH, (g + 1) * p.per_group - d0);
    stream_order();
    int32_t bits = 0;
    int begin, len;
    span_of(p.s, seq, &begin, &len, &bits);
    const int64_t slot = read_slot(p.s, seq, &bits), dest = write_slot(p.s, seq, 0, &bits);
    if (blockIdx.x == 0 && tid == 0) flag_err(p.s.dev_err, bits);
    const bool live = ch < nch;
    const int d = live ? d0 + ch : d0;
    float h[SPL], a2[SPL];
    load_states<SPL>(p, slot, d, n0, h);
    load_a2<SPL>(p, d, n0, a2);
    for (int t0 = 0; t0 < len; t0 += TT) {
        const int nt = min(TT, len - t0);
        const int64_t tok = begin + t0;
        for (int i = tid; i < nt * CH; i += kThreads) {
            const int t = i / CH, c = i % CH;
            float2 v = make_float2(0.f, 0.f);
            if (c < nch) {
                const int dd = d0 + c;
                const float x = ld_in(p.x, (tok + t) * p.xs[1] + dd * p.xs[2], p.x_dt);
                float s = ld_in(p.dt, (tok + t) * p.ds[1] + dd * p.ds[2], p.dt_dt);
                if (p.softplus) s = softplus_f(s + (p.dt_bias ? p.dt_bias[dd * p.dtb_s] : 0.f));
                v = make_float2(s, s * x);
            }
            step[i] = v;
        }
        for (int i = tid; i < nt * N; i += kThreads) {
            const int t = i / N, n = i % N;
            Bs[i] = ld_in(p.B, (tok + t) * p.bs[1] + g * p.bs[2] + n * p.bs[3], p.B_dt);
            Cs[i] = ld_in(p.C, (tok + t) * p.cs[1] + g * p.cs[2] + n * p.cs[3], p.C_dt);
        }
        __syncthreads();
        for (int t = 0; t < nt; ++t) {
            const float2 v = step[t * CH + ch];
            float y = 0.f;
#pragma unroll
            for (int i = 0; i < SPL; ++i) {
                h[i] = fmaf(exp2_f(v.x * a2[i]), h[i], v.y * Bs[t * N + n0 + i]);
                y = fmaf(Cs[t * N + n0 + i], h[i], y);
            }
#pragma unroll
            for (int off = LPC / 2; off > 0; off >>= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
            if (lane == 0) step[t * CH + ch].x = y;   // its lanes have read s: they met in the sum
        }
        __syncthreads();
        for (int i = tid; i < nt * CH; i += kThreads) {
            const int t = i / CH, c = i % CH;
            if (c >= nch) continue;
            const int dd = d0 + c;
            float y = step[i].x;
            if (p.skip) y = fmaf(p.skip[dd * p.skip_s], ld_in(p.x, (tok + t) * p.xs[1] + dd * p.xs[2], p.x_dt), y);
            if (p.z) y *= silu_f(ld_in(p.z, (tok + t) * p.zs[1] + dd * p.zs[2], p.z_dt));
            st_out(p.out, (tok + t) * p.os[1] + dd * p.os[2], p.out_dt, y);
        }
        __syncthreads();
    }
    if (live) store_states<SPL>(p, dest, d, n0, h);
}

template <int N, int SPL>
lar_status go(const SsmParams& p, cudaStream_t st) {
    using G = Geo<N, SPL>;
    const unsigned blocks = static_cast<unsigned>(p.G) * ((p.per_group + G::CH - 1) / G::CH);
    return launch_ordered(ssm_prefill_kernel<N, SPL>, dim3(blocks, p.s.n), kThreads, G::smem, st, p);
}

}  // namespace

lar_status launch_ssm_prefill(const SsmParams& p, void* stream) {
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (p.N) {
        case 16: return go<16, 4>(p, st);
        case 32: return go<32, 4>(p, st);
        case 64: return go<64, 4>(p, st);
        default: return go<128, 4>(p, st);
    }
}

}  // namespace lar

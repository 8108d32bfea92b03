// ssm_step.cu -- the selective state space recurrence for the tokens of one step
// (ssm_decode, ssm_decode_tokens).  Per token and channel d, with N states:
//
//     s = softplus(dt[d] + dt_bias[d])  (or dt[d])
//     h[n] <- exp(s A[d, n]) h[n] + s x[d] B[g, n]
//     out = (sum_n C[g, n] h[n] + D[d] x[d]) silu(z[d])
//
// Bound by the state's way through memory, 2 N words a channel against 4
// activations.  A lane holds 16 bytes of each of two neighbouring channels; a
// block takes its channels through several sequences, so that A, as large as one
// state, is read once for all of them, and asks for the next sequence's states
// before it works on the current ones.  256 x 4096 x 16, fp32 states: 26 us for 143 MB
// (5.4 TB/s; one sequence a block with single loads: 139 us); 64 sequences of 4 tokens
// with a bf16 state stored after each: 15 us for 50 MB, at 275 instructions a warp and
// token (the scan over spans has 116: there a lane works out one channel's step, here
// both) in 55 % of the issue slots, the tokens one after another.
#include <algorithm>

#include "ssm_common.cuh"

namespace lar {

namespace {

constexpr int kThreads = 128;
constexpr int kMaxSeqs = 16;   // sequences of a block

// two neighbouring channels; `two`: the second exists
__device__ __forceinline__ float2 ld_pair(const void* base, int64_t off, int64_t st, int dt, bool vec, bool two) {
    if (vec) {
        if (dt == LAR_BF16) {
            const unsigned u = __ldg(reinterpret_cast<const unsigned*>(static_cast<const unsigned short*>(base) + off));
            return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
        }
        return __ldg(reinterpret_cast<const float2*>(static_cast<const float*>(base) + off));
    }
    return make_float2(ld_in(base, off, dt), two ? ld_in(base, off + st, dt) : 0.f);
}

// SPL states a lane, 16 bytes of the pool; N / SPL lanes a pair of channels.  Any
// layout and types.
template <int N, int SPL>
__global__ void __launch_bounds__(kThreads, 4) ssm_step_any_kernel(const SsmParams p, int per_block) {
    constexpr int LPC = N / SPL;
    constexpr int CPB = 2 * kThreads / LPC;
    __shared__ int64_t from[kMaxSeqs], to[kMaxSeqs];
    const int b0 = blockIdx.y * per_block, nb = min(per_block, p.s.n - b0);
    const int lane = threadIdx.x % LPC, n0 = lane * SPL;
    const int d0 = blockIdx.x * CPB + threadIdx.x / LPC * 2;
    stream_order();
    int32_t bits = 0;
    if (threadIdx.x < nb) {
        from[threadIdx.x] = read_slot(p.s, b0 + threadIdx.x, &bits);
        if (!p.s.tslot) to[threadIdx.x] = write_slot(p.s, b0 + threadIdx.x, 0, &bits);
        if (blockIdx.x == 0) flag_err(p.s.dev_err, bits);
    }
    // channels past the last one do its work again and store nothing
    const bool one = d0 < p.D, two = d0 + 1 < p.D;
    const int d[2] = {min(d0, p.D - 1), min(d0 + 1, p.D - 1)};
    const int g[2] = {d[0] / p.per_group, d[1] / p.per_group};
    float a2[2][SPL], bias[2], skip[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        load_a2<SPL>(p, d[r], n0, a2[r]);
        bias[r] = p.dt_bias ? p.dt_bias[d[r] * p.dtb_s] : 0.f;
        skip[r] = p.skip ? p.skip[d[r] * p.skip_s] : 0.f;
    }
    __syncthreads();
    uint4 next[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) next[r] = load_raw(p, from[0], d[r], n0);
    for (int i = 0; i < nb; ++i) {
        const int64_t b = b0 + i;
        float h[2][SPL];
#pragma unroll
        for (int r = 0; r < 2; ++r) raw_states<SPL>(next[r], h[r]);
        if (i + 1 < nb) {
#pragma unroll
            for (int r = 0; r < 2; ++r) next[r] = load_raw(p, from[i + 1], d[r], n0);
        }
        for (int t = 0; t < p.s.T; ++t) {
            const float2 x = ld_pair(p.x, b * p.xs[0] + t * p.xs[1] + d[0] * p.xs[2], p.xs[2], p.x_dt, p.vec && two, two);
            float2 s = ld_pair(p.dt, b * p.ds[0] + t * p.ds[1] + d[0] * p.ds[2], p.ds[2], p.dt_dt, p.vec && two, two);
            float2 z = make_float2(0.f, 0.f);
            if (p.z) z = ld_pair(p.z, b * p.zs[0] + t * p.zs[1] + d[0] * p.zs[2], p.zs[2], p.z_dt, p.vec && two, two);
            float Bv[SPL], Cv[SPL];
            load_row<SPL>(p.B, b * p.bs[0] + t * p.bs[1] + g[0] * p.bs[2] + n0 * p.bs[3], p.bs[3], p.B_dt, Bv);
            load_row<SPL>(p.C, b * p.cs[0] + t * p.cs[1] + g[0] * p.cs[2] + n0 * p.cs[3], p.cs[3], p.C_dt, Cv);
            if (p.softplus) s = make_float2(softplus1(s.x + bias[0]), softplus1(s.y + bias[1]));
            float y[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float sr = r ? s.y : s.x, xr = r ? x.y : x.x;
                if (r && g[1] != g[0]) {
                    load_row<SPL>(p.B, b * p.bs[0] + t * p.bs[1] + g[1] * p.bs[2] + n0 * p.bs[3], p.bs[3], p.B_dt, Bv);
                    load_row<SPL>(p.C, b * p.cs[0] + t * p.cs[1] + g[1] * p.cs[2] + n0 * p.cs[3], p.cs[3], p.C_dt, Cv);
                }
                float acc[2] = {0.f, 0.f};   // as the pairs below add them: the same bits in any layout
#pragma unroll
                for (int k = 0; k < SPL; ++k) {
                    h[r][k] = fmaf(exp2_f(sr * a2[r][k]), h[r][k], sr * xr * Bv[k]);
                    acc[k % 2] = fmaf(Cv[k], h[r][k], acc[k % 2]);
                }
                y[r] = acc[0] + acc[1];
            }
#pragma unroll
            for (int off = LPC / 2; off > 0; off >>= 1) {
                y[0] += __shfl_xor_sync(0xffffffffu, y[0], off);
                y[1] += __shfl_xor_sync(0xffffffffu, y[1], off);
            }
            if (lane == 0 && one) {
                y[0] = fmaf(skip[0], x.x, y[0]);
                y[1] = fmaf(skip[1], x.y, y[1]);
                if (p.z) {
                    y[0] *= silu_f(z.x);
                    y[1] *= silu_f(z.y);
                }
                const int64_t o = b * p.os[0] + t * p.os[1] + d0 * p.os[2];
                if (p.vec && p.out_dt == LAR_BF16) {
                    *reinterpret_cast<unsigned*>(static_cast<unsigned short*>(p.out) + o) = pack_bf16x2(y[0], y[1]);
                } else {
                    st_out(p.out, o, p.out_dt, y[0]);
                    if (two) st_out(p.out, o + p.os[2], p.out_dt, y[1]);
                }
            }
            if (p.s.tslot) {
                const int64_t w = write_slot(p.s, static_cast<int>(b), t, &bits);
                if (one) store_states<SPL>(p, w, d0, n0, h[0]);
                if (two) store_states<SPL>(p, w, d0 + 1, n0, h[1]);
            }
        }
        if (!p.s.tslot) {
            if (one) store_states<SPL>(p, to[i], d0, n0, h[0]);
            if (two) store_states<SPL>(p, to[i], d0 + 1, n0, h[1]);
        }
    }
    if (p.s.tslot && blockIdx.x == 0 && threadIdx.x == 0) flag_err(p.s.dev_err, bits);
}

// What a lane reads for one token: its pair of channels and its part of the rows B, C.
template <typename X, int SPL>
struct Token {
    static constexpr int W = SPL * sizeof(X) / 4;   // 32-bit words of a part
    unsigned x[sizeof(X) / 2], dt[sizeof(X) / 2], z[sizeof(X) / 2], B[W], C[W];

    template <int K>
    static __device__ __forceinline__ void words(const X* src, unsigned* w) {
        if constexpr (K == 1) {
            w[0] = __ldg(reinterpret_cast<const unsigned*>(src));
        } else if constexpr (K == 2) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
            w[0] = v.x;
            w[1] = v.y;
        } else {
#pragma unroll
            for (int i = 0; i < K; i += 4) {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(src) + i / 4);
                w[i] = v.x;
                w[i + 1] = v.y;
                w[i + 2] = v.z;
                w[i + 3] = v.w;
            }
        }
    }
    template <int K>
    static __device__ __forceinline__ void widen(const unsigned* w, float* f) {
#pragma unroll
        for (int i = 0; i < K; ++i) {
            if constexpr (sizeof(X) == 2) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            } else {
                f[i] = __uint_as_float(w[i]);
            }
        }
    }
};

// The same for x, dt, z, B, C and out of one type X, in 16-byte aligned rows.
// Everything of the next token, and the next sequence's states, is asked for
// before the current one is worked on.  ONE: a single token, one state stored.
// R: blocks that an SM holds at once.
template <int N, int SPL, typename X, bool ONE, int R>
__global__ void __launch_bounds__(kThreads, R) ssm_step_kernel(const SsmParams p, int per_block) {
    constexpr int LPC = N / SPL, H = SPL / 2;
    constexpr int CPB = 2 * kThreads / LPC;
    using Tok = Token<X, SPL>;
    constexpr int PW = sizeof(X) / 2;   // words of a pair of channels
    __shared__ int64_t from[kMaxSeqs], to[ONE ? kMaxSeqs : kMaxSeqs * kMaxTokens];
    const int b0 = blockIdx.y * per_block, nb = min(per_block, p.s.n - b0), T = ONE ? 1 : p.s.T;
    const int lane = threadIdx.x % LPC, n0 = lane * SPL;
    const int d_own = blockIdx.x * CPB + threadIdx.x / LPC * 2;
    const bool live = d_own < p.D;
    const int d = live ? d_own : p.D - 2;   // does the last pair's work again and stores nothing
    stream_order();
    int32_t bits = 0;
    const bool each = !ONE && p.s.tslot;   // a slot for every token
    constexpr int PB = 16 / SPL;           // bytes of a state in the pool
    const auto bytes_of = [&](int64_t slot) { return slot < 0 ? int64_t{-1} : slot * p.ps[0] * PB; };
    const int writes = each ? nb * T : nb;
    for (int i = threadIdx.x; i < writes; i += kThreads)
        to[i] = bytes_of(each ? write_slot(p.s, b0 + i / T, i % T, &bits) : write_slot(p.s, b0 + i, 0, &bits));
    if (threadIdx.x < nb) from[threadIdx.x] = bytes_of(read_slot(p.s, b0 + threadIdx.x, &bits));
    if (blockIdx.x == 0) flag_err(p.s.dev_err, bits);

    const int g = d / p.per_group;
    const X* px = static_cast<const X*>(p.x) + b0 * p.xs[0] + d;
    const X* pd = static_cast<const X*>(p.dt) + b0 * p.ds[0] + d;
    const X* pz = static_cast<const X*>(p.z) + (p.z ? b0 * p.zs[0] + d : 0);
    const X* pB = static_cast<const X*>(p.B) + b0 * p.bs[0] + g * p.bs[2] + n0;
    const X* pC = static_cast<const X*>(p.C) + b0 * p.cs[0] + g * p.cs[2] + n0;
    X* po = static_cast<X*>(p.out) + b0 * p.os[0] + d;
    Tok next;
    const auto ask = [&]() {
        Tok::template words<PW>(px, next.x);
        Tok::template words<PW>(pd, next.dt);
        if (p.z) Tok::template words<PW>(pz, next.z);
        Tok::template words<Tok::W>(pB, next.B);
        Tok::template words<Tok::W>(pC, next.C);
    };
    ask();
    f32x2 a2[2][H];
    float2 bias = make_float2(0.f, 0.f), skip = bias;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        float a[SPL];
        load_a2<SPL>(p, d + r, n0, a);
#pragma unroll
        for (int i = 0; i < H; ++i) a2[r][i] = pack2(a[2 * i], a[2 * i + 1]);
    }
    if (p.dt_bias) bias = make_float2(p.dt_bias[d * p.dtb_s], p.dt_bias[(d + 1) * p.dtb_s]);
    if (p.skip) skip = make_float2(p.skip[d * p.skip_s], p.skip[(d + 1) * p.skip_s]);
    __syncthreads();
    // this lane's states in a slot
    char* const mine = static_cast<char*>(p.pool) + (d * p.ps[1] + n0) * PB;
    const int64_t other = p.ps[1] * PB;   // and the pair's other channel
    uint4 raw[2];
    const auto ask_states = [&](int64_t off) {
        raw[0] = raw[1] = make_uint4(0u, 0u, 0u, 0u);
        if (off >= 0) {
            raw[0] = *reinterpret_cast<const uint4*>(mine + off);
            raw[1] = *reinterpret_cast<const uint4*>(mine + off + other);
        }
    };
    ask_states(from[0]);
    for (int i = 0; i < nb; ++i) {
        f32x2 h[2][H];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float f[SPL];
            raw_states<SPL>(raw[r], f);
#pragma unroll
            for (int k = 0; k < H; ++k) h[r][k] = pack2(f[2 * k], f[2 * k + 1]);
        }
        if (i + 1 < nb) ask_states(from[i + 1]);
        for (int t = 0; t < T; ++t) {
            const Tok cur = next;
            const bool same = t + 1 < T;   // the next token is this sequence's
            if (same) {
                px += p.xs[1];
                pd += p.ds[1];
                pz += p.zs[1];
                pB += p.bs[1];
                pC += p.cs[1];
                ask();
            } else if (i + 1 < nb) {
                px += p.xs[0] - (T - 1) * p.xs[1];
                pd += p.ds[0] - (T - 1) * p.ds[1];
                pz += p.zs[0] - (T - 1) * p.zs[1];
                pB += p.bs[0] - (T - 1) * p.bs[1];
                pC += p.cs[0] - (T - 1) * p.cs[1];
                ask();
            }
            float x[2], s[2], Bv[SPL], Cv[SPL], y[2];
            Tok::template widen<PW>(cur.x, x);
            Tok::template widen<PW>(cur.dt, s);
            Tok::template widen<Tok::W>(cur.B, Bv);
            Tok::template widen<Tok::W>(cur.C, Cv);
            if (p.softplus) {
                s[0] = softplus1(s[0] + bias.x);
                s[1] = softplus1(s[1] + bias.y);
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const f32x2 ss = pack2(s[r], s[r]), xx = pack2(s[r] * x[r], s[r] * x[r]);
                f32x2 acc = 0ull;
#pragma unroll
                for (int k = 0; k < H; ++k) {
                    h[r][k] = fma2(ex2_2(mul2(ss, a2[r][k])), h[r][k], mul2(xx, pack2(Bv[2 * k], Bv[2 * k + 1])));
                    acc = fma2(pack2(Cv[2 * k], Cv[2 * k + 1]), h[r][k], acc);
                }
                float lo, hi;
                unpack2(acc, lo, hi);
                y[r] = lo + hi;
            }
#pragma unroll
            for (int off = LPC / 2; off > 0; off >>= 1) {
                y[0] += __shfl_xor_sync(0xffffffffu, y[0], off);
                y[1] += __shfl_xor_sync(0xffffffffu, y[1], off);
            }
            if (lane == 0 && live) {
                y[0] = fmaf(skip.x, x[0], y[0]);
                y[1] = fmaf(skip.y, x[1], y[1]);
                if (p.z) {
                    float z[2];
                    Tok::template widen<PW>(cur.z, z);
                    y[0] *= silu_f(z[0]);
                    y[1] *= silu_f(z[1]);
                }
                if constexpr (sizeof(X) == 2) *reinterpret_cast<unsigned*>(po) = pack_bf16x2(y[0], y[1]);
                else *reinterpret_cast<float2*>(po) = make_float2(y[0], y[1]);
            }
            po += same ? p.os[1] : p.os[0] - (T - 1) * p.os[1];
            if (live && (each || !same)) {
                const int64_t off = to[each ? i * T + t : i];
                if (off >= 0) {
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float f[SPL];
#pragma unroll
                        for (int k = 0; k < H; ++k) unpack2(h[r][k], f[2 * k], f[2 * k + 1]);
                        store_raw<SPL>(mine + off + r * other, f);
                    }
                }
            }
        }
    }
}

// Sequences of a block: the fewest with which the device holds all blocks at once
// (100 x 3 tokens, 2048 channels, bf16: 10.5 us; in two waves of fewer, 12.7 us).
int seqs_of_block(const SsmParams& p, int64_t columns, int resident) {
    const int64_t held = int64_t{152} * resident;
    return static_cast<int>(std::min<int64_t>(kMaxSeqs, (columns * p.s.n + held - 1) / held));
}

template <int N, int SPL, typename X, int R>
lar_status alike(const SsmParams& p, int64_t columns, cudaStream_t st) {
    const int per = seqs_of_block(p, columns, R);
    const dim3 grid(static_cast<unsigned>(columns), (p.s.n + per - 1) / per);
    return launch_ordered(p.s.T == 1 ? ssm_step_kernel<N, SPL, X, true, R> : ssm_step_kernel<N, SPL, X, false, R>, grid,
                          kThreads, 0, 1, st, p, per);
}

template <int N, int SPL>
lar_status go(const SsmParams& p, cudaStream_t st) {
    constexpr int CPB = 2 * kThreads / (N / SPL);
    const int64_t columns = (p.D + CPB - 1) / CPB;
    const int dt = p.x_dt;
    if (!p.vec || !p.vec_bc || p.dt_dt != dt || p.B_dt != dt || p.C_dt != dt || p.out_dt != dt || (p.z && p.z_dt != dt)) {
        const int per = seqs_of_block(p, columns, 4);
        const dim3 grid(static_cast<unsigned>(columns), (p.s.n + per - 1) / per);
        return launch_ordered(ssm_step_any_kernel<N, SPL>, grid, kThreads, 0, 1, st, p, per);
    }
    if constexpr (SPL == 8) {
        if (dt == LAR_F32) return alike<N, SPL, float, 4>(p, columns, st);
        // With the registers of five blocks the code is slower (17 x 4 tokens, 4096
        // channels: 6.9 us against 6.0), and pays where a block then takes fewer
        // sequences (64 x 4 tokens: 14.9 us against 16.0).
        if (seqs_of_block(p, columns, 5) < seqs_of_block(p, columns, 4))
            return alike<N, SPL, unsigned short, 5>(p, columns, st);
        return alike<N, SPL, unsigned short, 4>(p, columns, st);
    } else {
        return dt == LAR_F32 ? alike<N, SPL, float, 5>(p, columns, st) : alike<N, SPL, unsigned short, 7>(p, columns, st);
    }
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

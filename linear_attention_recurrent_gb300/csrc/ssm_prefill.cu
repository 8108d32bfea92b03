// ssm_prefill.cu -- the selective scan over packed spans (ssm_prefill).
//
// A warp walks the tokens of (a part of) one span for CW channels with the states
// in registers, by itself: a lane holds eight states of each of two channels, N / 8
// neighbouring lanes hold a pair of channels.  Inputs come in by cp.async, eight tokens
// a stage and a stage ahead, into shared memory of the warp's own; B and C are widened
// there once for all channels.  The lanes work out the steps, gates and outputs of
// their channels themselves, so warps never wait for one another.
//
// What bounds it, at N = 16 for a (token, channel): 19 SFU operations (32 a clock on
// an SM: 0.6 clocks), 64 fp32 multiplies and adds (128 a clock: 0.5 clocks), and their
// issue beside everything else: 116 instructions of 32 lanes, four a clock, 0.9
// clocks.  Products are taken in pairs, one instruction for two: their operands lie in
// neighbouring registers anyway.  A lane has eight states of each of two channels, of
// which it owns one: it works out that one's step, gate and output, and gets the other's
// step from the neighbour that owns it; so B and C, which every lane reads from shared
// memory for itself, serve two channels (with 16 states of one channel a lane, N = 64
// and 128 took 1.6 and 2.4 times as long).  64 spans of 256 tokens, 4096 channels:
// 303 us, 1.3 clocks a (token, channel), at 68 % of the issue slots: an instruction on
// pairs (32 of the 116) holds dispatch and its pipe for two cycles, which the counters
// show as what warps wait for.  An earlier form,
// in which blocks prepared the steps of all channels in shared memory and met at three
// barriers a tile, had 154 instructions.
//
// Long spans among others: a block's four warps share the tokens of one column.  Every
// warp but the last first runs its tokens from a zero state and keeps the end state and
// the sum of its steps (the decay over its part is exp(A sum)); the parts before it,
// joined, are the state that each then starts from, with outputs this time.  That is
// 1.7 times the work.  Few rows: the same over the blocks of a cluster, through
// distributed shared memory.  8192 tokens, 2048 channels: 161 us (unsplit 940 us);
// 24 ragged spans of 16384 tokens, 4096 channels: 380 to 400 us (unsplit 720 us).  With the
// first part's outputs made at once from the seed, as 1.4 times the work, the loop
// around both runs cost more than it saved: 167 and 416 us against 158 and 400.
//
// What is split is decided from averages.  One long span among many short ones therefore
// does worse than alone: 8192 tokens x 2048 beside 16 or 60 single tokens, over the four
// warps of a block, 740 and 620 us; beside 64 or more, where spans are not sorted and
// none is split, 1.1 to 1.2 ms.
//
// Types that differ, and rows that 16-byte loads do not fit, are staged by single elements
// through registers: 8192 x 2047 bf16 234 us; 8192 x 2048 with dt alone in fp32 590 us.
#include <algorithm>
#include <type_traits>

#include "ssm_common.cuh"

namespace lar {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kSPL = 8;        // states of a channel on a lane,
constexpr int kH = kSPL / 2;   // and pairs of them
constexpr int kTok = 8;        // tokens of a stage
// Tokens whose steps and gates are worked out together, and blocks an SM: a whole
// stage with the registers of three blocks, or half of one with four, which spans
// over clusters want (8192 x 2048 x 16: 158 us, with three 181 us; 24 ragged spans of
// 16384 x 4096 x 16 within blocks: 401 us with three, 450 us with four).
__host__ __device__ constexpr int tokens_of(bool cluster) { return cluster ? 4 : kTok; }
__host__ __device__ constexpr int blocks_of(bool cluster) { return cluster ? 4 : 3; }
constexpr int kSms = 152;      // of a GB300
constexpr int kFill = 4096;    // warps that keep it busy

// The types of x, dt, z, B, C and out: all bf16 or all fp32, staged as they are, or
// mixed, staged as fp32.
enum Mode { MIXED, BF16, F32 };

template <int MODE>
using Elem = typename std::conditional<MODE == BF16, unsigned short, float>::type;

template <int N, int MODE>
struct Geo {
    using E = Elem<MODE>;
    static constexpr int LPC = N / kSPL;      // lanes of a pair of channels
    static constexpr int CW = 64 / LPC;       // channels of a warp
    // a stage: x, dt, z [kTok][CW], B, C [kTok][N] as they come
    static constexpr int X = kTok * CW, R = kTok * N;
    static constexpr int stage = (3 * X + 2 * R) * static_cast<int>(sizeof(E));
    static constexpr int stages = 2;                            // in work and on its way
    static constexpr int wide = MODE == BF16 ? 2 * R * 4 : 0;   // B, C of the stage in work, in fp32
    static constexpr int warp_bytes = stages * stage + wide;
    static_assert(stage % 16 == 0, "stages start on 16 bytes");
};

template <int BYTES>
__device__ __forceinline__ void cp_async(void* dst, const void* src) {
    const unsigned d = static_cast<unsigned>(__cvta_generic_to_shared(dst));
    if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(d), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(d), "l"(src), "n"(BYTES) : "memory");
}

// nt rows of the first `cols` of COLS elements, by the lanes of a warp
template <int COLS, typename E>
__device__ __forceinline__ void copy_rows(E* dst, const E* src, int64_t row, int nt, int cols, int lane) {
    constexpr int B = COLS * sizeof(E) >= 16 ? 16 : static_cast<int>(COLS * sizeof(E));
    constexpr int PER = COLS * static_cast<int>(sizeof(E)) / B, EPC = B / static_cast<int>(sizeof(E));
    constexpr int ALL = PER * kTok;
#pragma unroll
    for (int i0 = 0; i0 < ALL; i0 += 32) {
        const int i = i0 + lane, t = i / PER, k = i % PER * EPC;
        if (i < ALL && t < nt && k < cols) cp_async<B>(dst + t * COLS + k, src + t * row + k);
    }
}

// the same by single elements: fp32 neighbours by 4-byte copies, others by loads and
// stores, which the warp waits for
template <int COLS, typename E>
__device__ __forceinline__ void read_rows(E* dst, const void* src, int64_t off, int64_t row, int64_t st, int dt, int nt,
                                          int cols, int lane) {
    constexpr int ALL = COLS * kTok, PER = (ALL + 31) / 32;
    if (sizeof(E) == 4 && dt == LAR_F32 && st == 1) {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int i = k * 32 + lane, t = i / COLS, c = i % COLS;
            if (i < ALL && t < nt && c < cols) cp_async<4>(dst + i, static_cast<const float*>(src) + off + t * row + c);
        }
        return;
    }
    constexpr int AT = PER < 8 ? PER : 8;   // on their way at once
#pragma unroll
    for (int k0 = 0; k0 < PER; k0 += AT) {
        E v[AT];
#pragma unroll
        for (int k = 0; k < AT; ++k) {
            const int i = (k0 + k) * 32 + lane, t = i / COLS, c = i % COLS;
            v[k] = E(0);
            if (i < ALL && t < nt && c < cols) {
                if constexpr (sizeof(E) == 2) v[k] = __ldg(static_cast<const unsigned short*>(src) + off + t * row + c * st);
                else v[k] = ld_in(src, off + t * row + c * st, dt);
            }
        }
#pragma unroll
        for (int k = 0; k < AT; ++k) {
            const int i = (k0 + k) * 32 + lane;
            if (i < ALL) dst[i] = v[k];
        }
    }
}

template <int N, int MODE, bool VEC>
struct Scan {
    using G = Geo<N, MODE>;
    using E = typename G::E;
    static constexpr int LPC = G::LPC, CW = G::CW, kStages = G::stages;

    const SsmParams& p;
    unsigned char* mem;        // this warp's shared memory
    int lane, sub, ch, n0;     // lane; its place among the pair's lanes; its own channel; its first state
    int g, d0, nch;            // group, first channel, channels
    float bias, skip;          // of its own channel
    f32x2 h[2][kH], a2[2][kH]; // of its own channel and of the pair's other
    float ssum;                // pass without outputs: the sum of the own channel's steps

    __device__ __forceinline__ Scan(const SsmParams& params, unsigned char* m, int column) : p(params), mem(m) {
        lane = threadIdx.x & 31;
        sub = lane % LPC;
        ch = lane / LPC * 2 + (sub & 1);
        n0 = sub * kSPL;
        const int per_g = (p.per_group + CW - 1) / CW;   // warps do not straddle groups
        g = column / per_g;
        d0 = g * p.per_group + (column % per_g) * CW;
        nch = min(CW, (g + 1) * p.per_group - d0);
    }

    // The lane's own channel (j = 0) and the other one; past the last, the last.
    __device__ __forceinline__ int d(int j) const { return d0 + min(ch ^ j, nch - 1); }

    __device__ __forceinline__ void load_weights() {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float a[kSPL];
            load_a2<kSPL>(p, d(j), n0, a);
#pragma unroll
            for (int i = 0; i < kH; ++i) a2[j][i] = pack2(a[2 * i], a[2 * i + 1]);
        }
        bias = p.dt_bias ? p.dt_bias[d(0) * p.dtb_s] : 0.f;
        skip = p.skip ? p.skip[d(0) * p.skip_s] : 0.f;
    }

    __device__ __forceinline__ void load_seed(int64_t slot) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float v[kSPL];
            load_states<kSPL>(p, slot, d(j), n0, v);
#pragma unroll
            for (int i = 0; i < kH; ++i) h[j][i] = pack2(v[2 * i], v[2 * i + 1]);
        }
    }

    __device__ __forceinline__ void store_end(int64_t slot) const {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float v[kSPL];
#pragma unroll
            for (int i = 0; i < kH; ++i) unpack2(h[j][i], v[2 * i], v[2 * i + 1]);
            if ((ch ^ j) < nch) store_states<kSPL>(p, slot, d(j), n0, v);
        }
    }

    __device__ __forceinline__ E* stage(int s) const { return reinterpret_cast<E*>(mem + s * G::stage); }

    // Ask for tokens [tok, tok + nt).
    template <bool OUT>
    __device__ __forceinline__ void fetch(int64_t tok, int nt, int s) const {
        E* r = stage(s);
        if constexpr (VEC) {
            copy_rows<CW>(r, static_cast<const E*>(p.x) + tok * p.xs[1] + d0, p.xs[1], nt, nch, lane);
            copy_rows<CW>(r + G::X, static_cast<const E*>(p.dt) + tok * p.ds[1] + d0, p.ds[1], nt, nch, lane);
            if (OUT && p.z) copy_rows<CW>(r + 2 * G::X, static_cast<const E*>(p.z) + tok * p.zs[1] + d0, p.zs[1], nt, nch, lane);
        } else {
            read_rows<CW>(r, p.x, tok * p.xs[1] + d0 * p.xs[2], p.xs[1], p.xs[2], p.x_dt, nt, nch, lane);
            read_rows<CW>(r + G::X, p.dt, tok * p.ds[1] + d0 * p.ds[2], p.ds[1], p.ds[2], p.dt_dt, nt, nch, lane);
            if (OUT && p.z)
                read_rows<CW>(r + 2 * G::X, p.z, tok * p.zs[1] + d0 * p.zs[2], p.zs[1], p.zs[2], p.z_dt, nt, nch, lane);
        }
        if (MODE != MIXED && (VEC || p.vec_bc)) {
            copy_rows<N>(r + 3 * G::X, static_cast<const E*>(p.B) + tok * p.bs[1] + g * p.bs[2], p.bs[1], nt, N, lane);
            if (OUT) copy_rows<N>(r + 3 * G::X + G::R, static_cast<const E*>(p.C) + tok * p.cs[1] + g * p.cs[2], p.cs[1], nt, N, lane);
        } else {
            read_rows<N>(r + 3 * G::X, p.B, tok * p.bs[1] + g * p.bs[2], p.bs[1], p.bs[3], p.B_dt, nt, N, lane);
            if (OUT) read_rows<N>(r + 3 * G::X + G::R, p.C, tok * p.cs[1] + g * p.cs[2], p.cs[1], p.cs[3], p.C_dt, nt, N, lane);
        }
    }

    static __device__ __forceinline__ float value(E v) {
        if constexpr (MODE == BF16) return bf16_bits_to_float(v);
        else return v;
    }

    // Tokens [begin, end) of the packed arrays; OUT: with outputs, else the end
    // state and the steps' sum alone.
    template <bool OUT, int U>
    __device__ __forceinline__ void run(int64_t begin, int64_t end) {
        const int64_t n = end - begin;
        const auto left = [&](int64_t i) { return static_cast<int>(max(int64_t{0}, min(static_cast<int64_t>(kTok), n - i * kTok))); };
#pragma unroll
        for (int s = 0; s + 1 < kStages; ++s) {
            if (left(s) > 0) fetch<OUT>(begin + s * kTok, left(s), s);
            cp_async_commit();
        }
        int s = 0, sn = kStages - 1;   // stage in work, stage to fill
        for (int64_t i = 0; i * kTok < n; ++i) {
            const int nt = left(i);
            const int64_t tok = begin + i * kTok, ahead = i + kStages - 1;
            if (left(ahead) > 0) fetch<OUT>(begin + ahead * kTok, left(ahead), sn);
            cp_async_commit();
            cp_async_wait<kStages - 1>();
            __syncwarp();
            const E* r = stage(s);
            const float *Bs, *Cs;
            if constexpr (MODE == BF16) {
                float* w = reinterpret_cast<float*>(mem + kStages * G::stage);
                // 8 numbers a lane and turn; C lies behind B in both
#pragma unroll
                for (int k = lane * 8; k < (OUT ? 2 : 1) * G::R; k += 256) {
                    float f[8];
                    unpack8(*reinterpret_cast<const uint4*>(r + 3 * G::X + k), f);
                    *reinterpret_cast<float4*>(w + k) = make_float4(f[0], f[1], f[2], f[3]);
                    *reinterpret_cast<float4*>(w + k + 4) = make_float4(f[4], f[5], f[6], f[7]);
                }
                __syncwarp();
                Bs = w + n0;
                Cs = w + G::R + n0;
            } else {
                Bs = reinterpret_cast<const float*>(r) + 3 * G::X + n0;
                Cs = Bs + G::R;
            }
            if (nt == kTok) {
                for (int t = 0; t < kTok; t += U) tokens<OUT, U>(r, Bs, Cs, tok, t);
            } else {
                for (int t = 0; t < nt; ++t) tokens<OUT, 1>(r, Bs, Cs, tok, t);
            }
            __syncwarp();   // the stage, and B and C, are free
            s = s + 1 == kStages ? 0 : s + 1;
            sn = sn + 1 == kStages ? 0 : sn + 1;
        }
        cp_async_wait<0>();
        __syncwarp();
    }

    // U tokens of the stage from t on
    template <bool OUT, int U>
    __device__ __forceinline__ void tokens(const E* r, const float* Bs, const float* Cs, int64_t tok, int t) {
        float st[U], x[U], y[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x[u] = value(r[(t + u) * CW + ch]);
            st[u] = value(r[G::X + (t + u) * CW + ch]);
        }
        if (p.softplus) {
#pragma unroll
            for (int u = 0; u < U; ++u) st[u] = softplus1(st[u] + bias);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // s and s x of the own channel; the other's come from the neighbour that owns it
            const float s0 = st[u], x0 = st[u] * x[u];
            const float s1 = __shfl_xor_sync(0xffffffffu, s0, 1), x1 = __shfl_xor_sync(0xffffffffu, x0, 1);
            const f32x2 ss[2] = {pack2(s0, s0), pack2(s1, s1)}, xx[2] = {pack2(x0, x0), pack2(x1, x1)};
            f32x2 acc[2] = {0ull, 0ull};
#pragma unroll
            for (int i = 0; i < kH; i += 2) {
                const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(Bs + (t + u) * N + 2 * i);
                ulonglong2 c = b;
                if (OUT) c = *reinterpret_cast<const ulonglong2*>(Cs + (t + u) * N + 2 * i);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    h[j][i] = fma2(ex2_2(mul2(ss[j], a2[j][i])), h[j][i], mul2(xx[j], b.x));
                    h[j][i + 1] = fma2(ex2_2(mul2(ss[j], a2[j][i + 1])), h[j][i + 1], mul2(xx[j], b.y));
                    if (OUT) {
                        acc[j] = i == 0 ? mul2(c.x, h[j][i]) : fma2(c.x, h[j][i], acc[j]);
                        acc[j] = fma2(c.y, h[j][i + 1], acc[j]);
                    }
                }
            }
            if (OUT) {
                float lo, hi, lo1, hi1;
                unpack2(acc[0], lo, hi);
                unpack2(acc[1], lo1, hi1);
                y[u] = lo + hi + __shfl_xor_sync(0xffffffffu, lo1 + hi1, 1);
            } else {
                ssum += st[u];
            }
        }
        if constexpr (OUT) finish<U>(r, tok, t, x, y);
    }

    // The sums over the pair's lanes, the skip, the gate and the stores
    template <int U>
    __device__ __forceinline__ void finish(const E* r, int64_t tok, int t, const float* x, float* y) const {
#pragma unroll
        for (int off = 2; off < LPC; off <<= 1) {
#pragma unroll
            for (int u = 0; u < U; ++u) y[u] += __shfl_xor_sync(0xffffffffu, y[u], off);
        }
        if (sub > 1 || ch >= nch) return;
        if (p.skip) {
#pragma unroll
            for (int u = 0; u < U; ++u) y[u] = fmaf(skip, x[u], y[u]);
        }
        if (p.z) {
#pragma unroll
            for (int u = 0; u < U; ++u) y[u] *= silu_f(value(r[2 * G::X + (t + u) * CW + ch]));
        }
        const int64_t o = (tok + t) * p.os[1] + (d0 + ch) * p.os[2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if constexpr (MODE == BF16) static_cast<__nv_bfloat16*>(p.out)[o + u * p.os[1]] = __float2bfloat16_rn(y[u]);
            else st_out(p.out, o + u * p.os[1], MODE == F32 ? LAR_F32 : p.out_dt, y[u]);
        }
    }
};

// h <- 2^(s a2) h + e for both channels of a lane, s0 and s1 the sums of their steps.
// Over a long part the factor may be past fp32 on either side where its product with h
// is not: a large h falls far, a small one grows, an empty one stays.  So it is taken in
// four equal factors (a quarter of s is exact), each held within [2^-125, 2^127]: 2^-500
// takes any finite h to 0 and 2^508 the least one, 2^-149, past fp32, and neither makes a
// NaN of an infinite or an empty h.  Each channel by its own numbers alone: beside the last
// channel of an odd count there is a lane whose numbers are whatever shared memory held.
__device__ __forceinline__ void decay_join(f32x2 (*h)[kH], const f32x2 (*a2)[kH], float s0, float s1,
                                           const f32x2 (*e)[kH]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const float quarter = 0.25f * (j ? s1 : s0);
#pragma unroll
        for (int i = 0; i < kH; ++i) {
            float v[2], f[2];
            unpack2(mul2(pack2(quarter, quarter), a2[j][i]), v[0], v[1]);
#pragma unroll
            for (int k = 0; k < 2; ++k) f[k] = exp2_f(fmaxf(fminf(v[k], 127.f), -125.f));   // of a NaN: e is one, too
            const f32x2 ff = pack2(f[0], f[1]);
            h[j][i] = fma2(mul2(mul2(mul2(h[j][i], ff), ff), ff), ff, e[j][i]);
        }
    }
}

// The y-th longest span (equal ones in order); y itself past kSorted spans.  Blocks
// start in this order: the last ones to start are short.
constexpr int kSorted = 64;

__device__ __forceinline__ int longest(const SlotParams& s, int y, int* lens, int* found) {
    if (s.n > kSorted) return y;
    int32_t bits = 0;
    int begin;
    for (int i = threadIdx.x; i < s.n; i += kThreads) span_of(s, i, &begin, &lens[i], &bits);
    __syncthreads();
    for (int i = threadIdx.x; i < s.n; i += kThreads) {
        const int li = lens[i];
        int rank = 0;
        for (int j = 0; j < s.n; ++j) rank += lens[j] > li || (lens[j] == li && j < i);
        if (rank == y) *found = i;
    }
    __syncthreads();
    return *found;
}

// How a launch spreads its work.
struct Spread {
    int columns;    // columns of channels
    int ranks;      // blocks of a cluster that share a column of a span, or 1
    int min_part;   // ranks > 1: least tokens of a part
    int long_len;   // ranks 1: spans of more tokens are split over the warps of a block,
    int long_max;   // and there are at most so many of them
};

// ranks 1: a block takes four columns of a span, a warp each, or, of a long span, one
// column whose tokens its warps share.  ranks > 1: the warps of a whole cluster share
// the tokens of one column.
template <int N, int MODE, bool VEC, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, blocks_of(CLUSTER)) ssm_prefill_kernel(const SsmParams p, const Spread w) {
    extern __shared__ __align__(16) unsigned char smem[];
    // what a warp (and, behind them, the block) leaves: its lanes' states, four by
    // four, and the sums of the steps of the channels that its lanes own
    struct Left {
        float4 h[kSPL / 2][32];
        float s[32];
    };
    constexpr int WB = Geo<N, MODE>::warp_bytes;
    static_assert(WB >= 2 * static_cast<int>(sizeof(Left)) && WB % 16 == 0, "the stages' memory, between the two runs, holds both");
    const auto left = [&](int v) -> Left& { return *reinterpret_cast<Left*>(smem + v * WB); };
    Left& whole = *reinterpret_cast<Left*>(smem + sizeof(Left));
    __shared__ int lens[kSorted], found;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int rank = CLUSTER ? static_cast<int>(blockIdx.x) % w.ranks : 0;
    stream_order();
    int seq, column, parts, part;   // the span, this warp's column and part of the span's tokens
    int begin, len;
    int32_t bits = 0;
    if (CLUSTER) {
        seq = blockIdx.y;
        span_of(p.s, seq, &begin, &len, &bits);
        column = static_cast<int>(blockIdx.x) / w.ranks;
        parts = min(w.ranks * kWarps, max(1, len / w.min_part));
        part = rank * kWarps + warp;
    } else {
        // blocks: a column each of the spans that may be long, four of the others
        const int quads = (w.columns + kWarps - 1) / kWarps;
        const int64_t b = blockIdx.x, longs = static_cast<int64_t>(w.long_max) * w.columns;
        const int y = static_cast<int>(b < longs ? b / w.columns : w.long_max + (b - longs) / quads);
        const int at = static_cast<int>(b < longs ? b % w.columns : (b - longs) % quads);
        seq = longest(p.s, y, lens, &found);
        span_of(p.s, seq, &begin, &len, &bits);
        const bool split = b < longs && len > w.long_len;
        if (!split && at >= quads) return;   // not long after all: others have its columns
        column = split ? at : at * kWarps + warp;
        parts = split ? kWarps : 1;
        part = split ? warp : 0;
        if (column >= w.columns) return;     // split blocks are whole: no barrier misses this warp
    }
    Scan<N, MODE, VEC> sc(p, smem + warp * WB, column);
    const int64_t slot = read_slot(p.s, seq, &bits), dest = write_slot(p.s, seq, 0, &bits);
    if (column == 0 && part == 0 && lane == 0) flag_err(p.s.dev_err, bits);
    // whole stages a part; the last ones may have none
    const int each = ((len + parts - 1) / parts + kTok - 1) / kTok * kTok;
    const int lo = static_cast<int>(min(static_cast<int64_t>(part) * each, static_cast<int64_t>(len)));
    const int hi = min(lo + each, len);
    sc.load_weights();
    if (parts > 1) {   // all warps of the block, of the cluster, agree
        const auto put = [&](Left& to) {
#pragma unroll
            for (int i = 0; i < kSPL / 2; ++i) {
                const f32x2* h = &sc.h[0][0] + 2 * i;
                float4 v;
                unpack2(h[0], v.x, v.y);
                unpack2(h[1], v.z, v.w);
                to.h[i][lane] = v;
            }
            to.s[lane] = sc.ssum;
        };
        const auto take = [&](const float4* v, f32x2* e) {
#pragma unroll
            for (int i = 0; i < kSPL / 2; ++i) {
                e[2 * i] = pack2(v[i].x, v[i].y);
                e[2 * i + 1] = pack2(v[i].z, v[i].w);
            }
        };
        const auto clear = [](f32x2 (*h)[kH]) {
#pragma unroll
            for (int i = 0; i < 2 * kH; ++i) h[i / kH][i % kH] = 0ull;
        };
        clear(sc.h);
        sc.ssum = 0.f;
        if (hi < len) sc.template run<false, tokens_of(CLUSTER)>(begin + lo, begin + hi);   // somebody comes after this warp
        put(left(warp));
        __syncthreads();
        // what the warps before this one in the block come to; the last one, with its
        // own part, what the block does
        f32x2 pre[2][kH];
        float pre_s = 0.f, pre_t = 0.f;   // sums of steps: the own channel's, the other's
        clear(pre);
        for (int v = 0; v < warp; ++v) {
            float4 q[kSPL / 2];
            f32x2 e[2][kH];
#pragma unroll
            for (int i = 0; i < kSPL / 2; ++i) q[i] = left(v).h[i][lane];
            take(q, &e[0][0]);
            const float s0 = left(v).s[lane], s1 = left(v).s[lane ^ 1];
            decay_join(pre, sc.a2, s0, s1, e);
            pre_s += s0;
            pre_t += s1;
        }
        if (CLUSTER) {
            if (warp == kWarps - 1) {
                f32x2 own[2][kH];
#pragma unroll
                for (int i = 0; i < 2 * kH; ++i) {
                    own[i / kH][i % kH] = sc.h[i / kH][i % kH];
                    sc.h[i / kH][i % kH] = pre[i / kH][i % kH];
                }
                decay_join(sc.h, sc.a2, sc.ssum, __shfl_xor_sync(0xffffffffu, sc.ssum, 1), own);
                sc.ssum += pre_s;
                put(whole);
            }
            cluster_sync();
        }
        if (lo < len) {
            sc.load_seed(slot);
            if (CLUSTER) {
                for (int r = 0; r < rank; ++r) {
                    float4 q[kSPL / 2];
                    f32x2 e[2][kH];
#pragma unroll
                    for (int i = 0; i < kSPL / 2; ++i)
                        q[i] = ld_peer_f32x4(reinterpret_cast<const float*>(&whole.h[i][lane]), r);
                    const float s0 = ld_peer_f32(&whole.s[lane], r);
                    const float s1 = ld_peer_f32(&whole.s[lane ^ 1], r);
                    take(q, &e[0][0]);
                    decay_join(sc.h, sc.a2, s0, s1, e);
                }
            }
            // the first warp has none before it: no steps times a rate of -infinity would be NaN
            if (warp > 0) decay_join(sc.h, sc.a2, pre_s, pre_t, pre);
        }
        // all have read their peers, and the seed before any end state is stored
        if (CLUSTER) cluster_sync();
        else __syncthreads();
    } else if (part == 0) {
        sc.load_seed(slot);
    }
    if (lo < len || (len == 0 && part == 0)) {
        sc.template run<true, tokens_of(CLUSTER)>(begin + lo, begin + hi);
        if (hi == len) sc.store_end(dest);
    }
}

template <int N, int MODE, bool VEC>
lar_status go(const SsmParams& p, cudaStream_t st) {
    using G = Geo<N, MODE>;
    Spread w;
    w.columns = p.G * ((p.per_group + G::CW - 1) / G::CW);
    const int64_t rows = static_cast<int64_t>(w.columns) * p.s.n;
    // Clusters where a warp a column leaves the device empty even with every span split
    // over a block: blocks enough to fill it, up to the portable 8 (a span of 8192 x 2048 x
    // 16: 262, 182, 163 us with 2, 4, 8 when chosen; sizes between, as 7 with 188 us, fit the
    // device worse than the next power of two), while the spans have 16 tokens a warp on
    // average.  Parts have 32 at least: a span of average length then leaves half of the
    // blocks without tokens, a longer one does not.
    w.ranks = 1;
    while (w.ranks < 8 && rows * kWarps * w.ranks < kFill && p.s.ntok >= int64_t{128} * w.ranks * p.s.n) w.ranks *= 2;
    w.min_part = 32;
    // Long: more than 1.5 times the tokens of a warp if all that the device holds had
    // the same.  Measured at the ragged spans above: 720 us unsplit, 441, 446 and 401
    // us at 1, 1.25 and 1.5 times, 543 us at twice.  Past kSorted spans none is split.
    const int64_t len = p.s.ntok * w.columns * 3 / (int64_t{2} * kSms * 4 * 3);
    w.long_len = static_cast<int>(std::min<int64_t>(std::max<int64_t>(len, 64), INT32_MAX));
    w.long_max = p.s.n > kSorted ? 0 : static_cast<int>(std::min<int64_t>(p.s.n, p.s.ntok / w.long_len));
    const int smem = kWarps * G::warp_bytes;
    const auto kern = w.ranks > 1 ? ssm_prefill_kernel<N, MODE, VEC, true> : ssm_prefill_kernel<N, MODE, VEC, false>;
    const void* k = reinterpret_cast<const void*>(kern);
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return LAR_ERR_LAUNCH;
    dim3 grid(static_cast<unsigned>(w.columns * w.ranks), p.s.n);
    if (w.ranks == 1) {
        const int64_t quads = (w.columns + kWarps - 1) / kWarps;
        const int64_t blocks = static_cast<int64_t>(w.long_max) * w.columns + (p.s.n - w.long_max) * quads;
        if (blocks > INT32_MAX) return LAR_ERR_SHAPE;
        grid = dim3(static_cast<unsigned>(blocks));
    }
    return launch_ordered(kern, grid, kThreads, smem, w.ranks, st, p, w);
}

template <int N>
lar_status pick(const SsmParams& p, cudaStream_t st) {
    const int dt = p.x_dt;
    const bool alike = p.dt_dt == dt && p.B_dt == dt && p.C_dt == dt && p.out_dt == dt && (!p.z || p.z_dt == dt);
    if (!alike) return go<N, MIXED, false>(p, st);
    const bool vec = p.vec && p.vec_bc;
    if (dt == LAR_BF16) return vec ? go<N, BF16, true>(p, st) : go<N, BF16, false>(p, st);
    return vec ? go<N, F32, true>(p, st) : go<N, F32, false>(p, st);
}

}  // namespace

lar_status launch_ssm_prefill(const SsmParams& p, void* stream) {
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (p.N) {
        case 16: return pick<16>(p, st);
        case 32: return pick<32>(p, st);
        case 64: return pick<64>(p, st);
        default: return pick<128>(p, st);
    }
}

}  // namespace lar

// ssm_prefill.cu -- the selective scan over packed spans (ssm_prefill).
//
// A block of 128 threads walks the tokens of one span for CH channels, tile by
// tile, with the states in registers: a lane holds SPL states of each of CPL
// channels, LPC = N / SPL neighbouring lanes hold a channel.  Per tile
//   1. dt and x of every (token, channel) become the step s and s x in shared
//      memory, B and C lie beside them in fp32;
//   2. the recurrence runs, its sums y go where s was;
//   3. the skip and the gate are applied and the tile is stored.
// The next tile's inputs come in by cp.async meanwhile.
//
// What bounds it: for N = 16 a (token, channel) costs 16 SFU exponentials (32 a
// clock on an SM: 0.5 clocks), 64 fp32 multiplies and adds (0.5 clocks; issued
// in pairs), and what a lane reads of shared memory (128 bytes a clock).  A lane
// with one channel would read 2 N words of B and C for every channel, a clock's
// worth; four channels a lane share them.
//
// Few rows, long spans: the tokens of a span are split over the blocks of a
// cluster.  Every block but the last first runs its tokens from a zero state and
// keeps the end state and the sum of its steps (the decay over the block is
// exp(A sum)); all read the ones before them through distributed shared memory,
// join them to the state they start from, and run their tokens again with
// outputs.  That costs 1.7 times the work, so a span is split only where blocks
// are too few (see launch).
#include "ssm_common.cuh"

namespace lar {

namespace {

constexpr int kThreads = 128;
constexpr int kSms = 152;      // of a GB300
constexpr int kMinSeg = 64;    // least tokens of a block where a span is split

#ifndef LAR_TU
#define LAR_TU 4
#endif
constexpr int kTU = LAR_TU;   // tokens taken together: their loads and exponentials do not wait for one another

template <int N, int SPL, int CPL>
struct Geo {
    static constexpr int LPC = N / SPL;                     // lanes of a channel
    static constexpr int CPW = 32 / LPC * CPL;              // channels of a warp
    static constexpr int CH = kThreads / 32 * CPW;          // channels of a block
    static constexpr int TT = 2048 / CH < 32 ? 2048 / CH : 32;   // tokens of a tile
    static constexpr int E = TT * CH;
    static constexpr int PAIRS = CH / 2;                    // channel pairs: a thread prepares one, for
    static constexpr int TSTEP = kThreads / PAIRS;          // every TSTEP-th token,
    static constexpr int PT = TT / TSTEP;                   // PT of a tile
    static_assert(TT % kTU == 0 && TT % TSTEP == 0, "whole groups of tokens");
    static_assert(CH % 8 == 0 && kThreads % (CH / 2) == 0, "whole 16-byte groups; pairs of channels tile the block");
};

// Where the parts of a block's shared memory lie (bytes).
struct Parts {
    int bs, raw, x, dt, z, b, c, stage, total;
};

template <int N, int SPL, int CPL>
__host__ __device__ inline Parts parts_of(const SsmParams& p) {
    using G = Geo<N, SPL, CPL>;
    Parts q;
    q.bs = G::E * 8;                                        // after s, s x
    q.raw = q.bs + G::TT * N * 8;                           // after B, C
    const auto size = [](int dt, int n) { return n * (dt == LAR_F32 ? 4 : 2); };
    q.x = 0;
    q.dt = q.x + size(p.x_dt, G::E);
    q.z = q.dt + size(p.dt_dt, G::E);
    q.b = q.z + (p.z ? size(p.z_dt, G::E) : 0);
    q.c = q.b + size(p.B_dt, G::TT * N);
    q.stage = q.c + size(p.C_dt, G::TT * N);
    q.total = q.raw + 2 * q.stage;
    return q;
}

// Rows [0, nt) of the first `cols` of COLS elements, `row` elements apart in
// memory and COLS in shared memory, by 16-byte copies.
template <int COLS, int ES>
__device__ __forceinline__ void copy_rows_of(unsigned char* dst, const unsigned char* src, int64_t row, int nt, int cols) {
    constexpr int PER = COLS * ES / 16;   // a power of two
    constexpr int STEP = kThreads / PER > 0 ? kThreads / PER : 1;
    static_assert(PER <= kThreads, "a thread keeps its column");
    const int k = threadIdx.x % PER;
    if (k * 16 >= cols * ES) return;
    int t = threadIdx.x / PER;
    const unsigned char* s = src + t * row * ES + k * 16;
#pragma unroll 4
    for (; t < nt; t += STEP, s += STEP * row * ES) cp_async16(dst + t * COLS * ES + k * 16, s);
}

template <int COLS>
__device__ __forceinline__ void copy_rows(unsigned char* dst, const void* src, int64_t off, int64_t row, int dt, int nt,
                                          int cols) {
    if (dt == LAR_BF16)
        copy_rows_of<COLS, 2>(dst, static_cast<const unsigned char*>(src) + off * 2, row, nt, cols);
    else
        copy_rows_of<COLS, 4>(dst, static_cast<const unsigned char*>(src) + off * 4, row, nt, cols);
}

__device__ __forceinline__ float2 bf2(unsigned u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// PT pairs, `step` elements apart, from a stage
template <int PT>
__device__ __forceinline__ void raw_pairs(const unsigned char* base, int dt, int i, int step, float2* v) {
    if (dt == LAR_BF16) {
#pragma unroll
        for (int k = 0; k < PT; ++k) v[k] = bf2(*reinterpret_cast<const unsigned*>(base + (i + k * step) * 2));
    } else {
#pragma unroll
        for (int k = 0; k < PT; ++k) v[k] = *reinterpret_cast<const float2*>(base + (i + k * step) * 4);
    }
}

// the same from memory, any layout: pair k at off + k row, its second element st on
template <int PT, typename T>
__device__ __forceinline__ void mem_pairs_of(const T* src, int64_t row, int64_t st, int n_tok, int tstep, bool one,
                                             bool two, float2* v) {
#pragma unroll
    for (int k = 0; k < PT; ++k) {
        v[k] = make_float2(0.f, 0.f);
        const T* a = src + k * row;
        if constexpr (sizeof(T) == 2) {
            if (one && k * tstep < n_tok) v[k].x = bf16_bits_to_float(__ldg(a));
            if (two && k * tstep < n_tok) v[k].y = bf16_bits_to_float(__ldg(a + st));
        } else {
            if (one && k * tstep < n_tok) v[k].x = __ldg(a);
            if (two && k * tstep < n_tok) v[k].y = __ldg(a + st);
        }
    }
}

template <int PT>
__device__ __forceinline__ void mem_pairs(const void* base, int dt, int64_t off, int64_t row, int64_t st, int n_tok,
                                          int tstep, bool one, bool two, float2* v) {
    if (dt == LAR_BF16)
        mem_pairs_of<PT>(static_cast<const unsigned short*>(base) + off, row, st, n_tok, tstep, one, two, v);
    else
        mem_pairs_of<PT>(static_cast<const float*>(base) + off, row, st, n_tok, tstep, one, two, v);
}

// Sums of y[token][channel] over the LPC lanes of a channel, scattered over them.
// Steps that halve the channels need no selection: channel j of lane l is channel
// j ^ perm(l) of its group, so that a lane always keeps its first values and sends
// its last ones.  Steps past that halve the tokens, which lanes take in order.
template <int LPC, int CPL>
struct Scatter {
    static constexpr int CK = CPL / (LPC < CPL ? LPC : CPL);                 // channels kept
    static constexpr int LEFT = LPC < CPL ? 1 : LPC / CPL;                   // lanes that share them
    static constexpr int TK = kTU / (LEFT < kTU ? LEFT : kTU);               // tokens kept

    static __device__ __forceinline__ int perm_of(int lane) {
        int m = 0;
#pragma unroll
        for (int bit = 1, half = CPL / 2; bit < LPC && half > 0; bit <<= 1, half >>= 1)
            if (lane & bit) m |= half;
        return m;
    }
    // the first of the TK tokens that a lane ends with
    static __device__ __forceinline__ int first_token(int lane) {
        int t = 0;
#pragma unroll
        for (int bit = CPL, half = kTU / 2; bit < LPC && half > 0; bit <<= 1, half >>= 1)
            if (lane & bit) t += half;
        return t;
    }
    static __device__ __forceinline__ void sum(float (*y)[CPL], int lane) {
        int nt = kTU;
#pragma unroll
        for (int bit = 1, half = CPL / 2; bit < LPC; bit <<= 1, half >>= 1) {
            if (half > 0) {
#pragma unroll
                for (int u = 0; u < kTU; ++u)
#pragma unroll
                    for (int j = 0; j < half; ++j) y[u][j] += __shfl_xor_sync(0xffffffffu, y[u][j + half], bit);
            } else if (nt > 1) {
                nt /= 2;
                const bool up = lane & bit;
#pragma unroll
                for (int u = 0; u < kTU / 2; ++u) {
                    if (u >= nt) continue;
                    const float keep = up ? y[u + nt][0] : y[u][0], send = up ? y[u][0] : y[u + nt][0];
                    y[u][0] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
                }
            } else {
                y[0][0] += __shfl_xor_sync(0xffffffffu, y[0][0], bit);
            }
        }
    }
};

template <int N, int SPL, int CPL>
struct Scan {
    using G = Geo<N, SPL, CPL>;
    using S = Scatter<G::LPC, CPL>;
    static constexpr int LPC = G::LPC, CH = G::CH, TT = G::TT, H = SPL / 2;

    const SsmParams& p;
    const Parts q;
    unsigned char* smem;
    float2* step;              // [TT][CH]: s, s x; the sum y takes the place of s
    float *Bs, *Cs;            // [TT][N]
    int g, d0, nch;            // group, first channel, channels
    int ch0, n0, perm, t_own;  // this lane's channels (in the block) and states; the token of a group it ends with
    f32x2 h[CPL][H], a2[CPL][H];
    float ssum[CPL];           // pass 1: the steps' sum

    __device__ __forceinline__ Scan(const SsmParams& params, unsigned char* sm, int column)
        : p(params), q(parts_of<N, SPL, CPL>(params)), smem(sm) {
        step = reinterpret_cast<float2*>(smem);
        Bs = reinterpret_cast<float*>(smem + q.bs);
        Cs = Bs + TT * N;
        const int per_g = (p.per_group + CH - 1) / CH;   // blocks do not straddle groups
        g = column / per_g;
        d0 = g * p.per_group + (column % per_g) * CH;
        nch = min(CH, (g + 1) * p.per_group - d0);
        const int lane = threadIdx.x % LPC;
        ch0 = threadIdx.x / LPC * CPL;
        n0 = lane * SPL;
        perm = S::perm_of(lane);
        t_own = S::first_token(lane);
    }

    __device__ __forceinline__ int channel(int j) const { return ch0 + (j ^ perm); }

    __device__ __forceinline__ void load_decay() {
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            float a[SPL];
            load_a2<SPL>(p, d0 + min(channel(j), nch - 1), n0, a);
#pragma unroll
            for (int i = 0; i < H; ++i) a2[j][i] = pack2(a[2 * i], a[2 * i + 1]);
        }
    }

    __device__ __forceinline__ void load_seed(int64_t slot) {
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            float v[SPL];
            load_states<SPL>(p, slot, d0 + min(channel(j), nch - 1), n0, v);
#pragma unroll
            for (int i = 0; i < H; ++i) h[j][i] = pack2(v[2 * i], v[2 * i + 1]);
        }
    }

    __device__ __forceinline__ void store_end(int64_t slot) const {
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            float v[SPL];
#pragma unroll
            for (int i = 0; i < H; ++i) unpack2(h[j][i], v[2 * i], v[2 * i + 1]);
            if (channel(j) < nch) store_states<SPL>(p, slot, d0 + channel(j), n0, v);
        }
    }

    // Start the copies of tokens [tok, tok + nt) into a stage.
    template <bool OUT>
    __device__ __forceinline__ void fetch(int64_t tok, int nt, int stage) const {
        unsigned char* r = smem + q.raw + stage * q.stage;
        if (p.vec) {
            copy_rows<CH>(r + q.x, p.x, tok * p.xs[1] + d0, p.xs[1], p.x_dt, nt, nch);
            copy_rows<CH>(r + q.dt, p.dt, tok * p.ds[1] + d0, p.ds[1], p.dt_dt, nt, nch);
            if (OUT && p.z) copy_rows<CH>(r + q.z, p.z, tok * p.zs[1] + d0, p.zs[1], p.z_dt, nt, nch);
        }
        if (p.vec_bc) {
            copy_rows<N>(r + q.b, p.B, tok * p.bs[1] + g * p.bs[2], p.bs[1], p.B_dt, nt, N);
            if (OUT) copy_rows<N>(r + q.c, p.C, tok * p.cs[1] + g * p.cs[2], p.cs[1], p.C_dt, nt, N);
        }
        cp_async_commit();
    }

    // This thread's pairs of x, dt or z: channels c, c + 1 of every TSTEP-th token
    // of the tile from t on.
    __device__ __forceinline__ void pairs(const void* base, int part, const unsigned char* r, int dt, int64_t tok,
                                          const int64_t* st, int t, int c, int nt, float2* v) const {
        if (p.vec)
            raw_pairs<G::PT>(r + part, dt, t * CH + c, G::TSTEP * CH, v);
        else
            mem_pairs<G::PT>(base, dt, (tok + t) * st[1] + (d0 + c) * st[2], G::TSTEP * st[1], st[2], nt - t, G::TSTEP,
                             c < nch, c + 1 < nch, v);
    }

    // Rows of B or C, zero past the tile's last token.
    __device__ __forceinline__ void rows(float* dst, const void* base, int part, const unsigned char* r, int dt,
                                         int64_t off, const int64_t* st, int nt) const {
        constexpr int PT = (TT * N / 2 + kThreads - 1) / kThreads;
        float2 v[PT];
        const int i = 2 * threadIdx.x;
        if (i >= TT * N) return;   // a tile of few values; else they divide evenly
        if (p.vec_bc) {
            raw_pairs<PT>(r + part, dt, i, 2 * kThreads, v);
        } else {
#pragma unroll
            for (int k = 0; k < PT; ++k) {
                const int t = (i + k * 2 * kThreads) / N, n = (i + k * 2 * kThreads) % N;
                if (t < nt)
                    v[k] = make_float2(ld_in(base, off + t * st[1] + n * st[3], dt),
                                       ld_in(base, off + t * st[1] + (n + 1) * st[3], dt));
            }
        }
#pragma unroll
        for (int k = 0; k < PT; ++k) {
            const int e = i + k * 2 * kThreads;
            *reinterpret_cast<float2*>(dst + e) = e < nt * N ? v[k] : make_float2(0.f, 0.f);
        }
    }

    // Tokens [begin, end) of the packed arrays; OUT: with outputs, else the end
    // state and the steps' sum alone.
    template <bool OUT>
    __device__ __forceinline__ void run(int64_t begin, int64_t end) {
        constexpr int PT = G::PT, TSTEP = G::TSTEP;
        const int c = threadIdx.x % G::PAIRS * 2, t0 = threadIdx.x / G::PAIRS;
        const bool one = c < nch, two = c + 1 < nch;
        const float2 bias = make_float2(one && p.dt_bias ? p.dt_bias[(d0 + c) * p.dtb_s] : 0.f,
                                        two && p.dt_bias ? p.dt_bias[(d0 + c + 1) * p.dtb_s] : 0.f);
        const float2 skip = make_float2(one && p.skip ? p.skip[(d0 + c) * p.skip_s] : 0.f,
                                        two && p.skip ? p.skip[(d0 + c + 1) * p.skip_s] : 0.f);
        int stage = 0;
        fetch<OUT>(begin, static_cast<int>(min(static_cast<int64_t>(TT), end - begin)), 0);
        for (int64_t tok = begin; tok < end; tok += TT, stage ^= 1) {
            const int nt = static_cast<int>(min(static_cast<int64_t>(TT), end - tok));
            cp_async_wait<0>();
            __syncthreads();   // the stage is in; the last tile's step and stage are free
            if (tok + TT < end)
                fetch<OUT>(tok + TT, static_cast<int>(min(static_cast<int64_t>(TT), end - tok - TT)), stage ^ 1);
            const unsigned char* r = smem + q.raw + stage * q.stage;
            {
                float2 x[PT], s[PT];
                pairs(p.x, q.x, r, p.x_dt, tok, p.xs, t0, c, nt, x);
                pairs(p.dt, q.dt, r, p.dt_dt, tok, p.ds, t0, c, nt, s);
                if (p.softplus) {
#pragma unroll
                    for (int k = 0; k < PT; ++k)
                        s[k] = softplus2(make_float2(s[k].x + bias.x, s[k].y + bias.y));
                }
#pragma unroll
                for (int k = 0; k < PT; ++k) {   // a step of 0 past the last token and the last channel
                    const bool a = one && t0 + k * TSTEP < nt, b = two && t0 + k * TSTEP < nt;
                    *reinterpret_cast<float4*>(step + (t0 + k * TSTEP) * CH + c) =
                        make_float4(a ? s[k].x : 0.f, a ? s[k].x * x[k].x : 0.f, b ? s[k].y : 0.f,
                                    b ? s[k].y * x[k].y : 0.f);
                }
            }
            rows(Bs, p.B, q.b, r, p.B_dt, tok * p.bs[1] + g * p.bs[2], p.bs, nt);
            if (OUT) rows(Cs, p.C, q.c, r, p.C_dt, tok * p.cs[1] + g * p.cs[2], p.cs, nt);
            __syncthreads();
            for (int t = 0; t < nt; t += kTU) tokens<OUT>(t);
            if (!OUT) continue;
            __syncthreads();
            float2 y[PT];
#pragma unroll
            for (int k = 0; k < PT; ++k) {
                const float4 v = *reinterpret_cast<const float4*>(step + (t0 + k * TSTEP) * CH + c);
                y[k] = make_float2(v.x, v.z);
            }
            if (p.skip) {
                float2 x[PT];
                pairs(p.x, q.x, r, p.x_dt, tok, p.xs, t0, c, nt, x);
#pragma unroll
                for (int k = 0; k < PT; ++k) y[k] = make_float2(fmaf(skip.x, x[k].x, y[k].x), fmaf(skip.y, x[k].y, y[k].y));
            }
            if (p.z) {
                float2 z[PT];
                pairs(p.z, q.z, r, p.z_dt, tok, p.zs, t0, c, nt, z);
#pragma unroll
                for (int k = 0; k < PT; ++k) y[k] = make_float2(y[k].x * silu_f(z[k].x), y[k].y * silu_f(z[k].y));
            }
            const int64_t o = (tok + t0) * p.os[1] + (d0 + c) * p.os[2], row = TSTEP * p.os[1];
            if (p.vec && p.out_dt == LAR_BF16) {
#pragma unroll
                for (int k = 0; k < PT; ++k)
                    if (one && t0 + k * TSTEP < nt)   // channels come by eights
                        *reinterpret_cast<unsigned*>(static_cast<unsigned short*>(p.out) + o + k * row) =
                            pack_bf16x2(y[k].x, y[k].y);
            } else {
#pragma unroll
                for (int k = 0; k < PT; ++k) {
                    if (t0 + k * TSTEP >= nt) continue;
                    if (one) st_out(p.out, o + k * row, p.out_dt, y[k].x);
                    if (two) st_out(p.out, o + k * row + p.os[2], p.out_dt, y[k].y);
                }
            }
        }
        __syncthreads();   // before anything else uses the shared memory
    }

    // kTU tokens of the tile, from t on
    template <bool OUT>
    __device__ __forceinline__ void tokens(int t) {
        float y[kTU][CPL];
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            // every decay of the group before the recurrence needs the first
            f32x2 e[kTU][H];
            float sx[kTU];
#pragma unroll
            for (int u = 0; u < kTU; ++u) {
                const float2 v = step[(t + u) * CH + channel(j)];
                sx[u] = v.y;
                if (!OUT) ssum[j] += v.x;
#pragma unroll
                for (int i = 0; i < H; ++i) e[u][i] = ex2_2(mul2(pack2(v.x, v.x), a2[j][i]));
            }
#pragma unroll
            for (int u = 0; u < kTU; ++u) {
                f32x2 acc = 0ull;
#pragma unroll
                for (int i = 0; i < H; i += 2) {
                    const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(Bs + (t + u) * N + n0 + 2 * i);
                    h[j][i] = fma2(e[u][i], h[j][i], mul2(pack2(sx[u], sx[u]), b.x));
                    h[j][i + 1] = fma2(e[u][i + 1], h[j][i + 1], mul2(pack2(sx[u], sx[u]), b.y));
                    if (OUT) {
                        const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(Cs + (t + u) * N + n0 + 2 * i);
                        acc = i == 0 ? mul2(c.x, h[j][i]) : fma2(c.x, h[j][i], acc);
                        acc = fma2(c.y, h[j][i + 1], acc);
                    }
                }
                if (OUT) {
                    float lo, hi;
                    unpack2(acc, lo, hi);
                    y[u][j] = lo + hi;
                }
            }
        }
        if (OUT) {
            S::sum(y, threadIdx.x % LPC);
            // y goes where s was: the lanes of a channel have read it, they met in the sums
#pragma unroll
            for (int u = 0; u < S::TK; ++u)
#pragma unroll
                for (int j = 0; j < S::CK; ++j) step[(t + t_own + u) * CH + channel(j)].x = y[u][j];
        }
    }
};

// blockIdx.x: (column of channels, rank in the cluster), blockIdx.y: the span.
// min_seg: the least tokens worth a block of their own where a span is split.
template <int N, int SPL, int CPL>
__global__ void __launch_bounds__(kThreads) ssm_prefill_kernel(const SsmParams p, int ranks, int min_seg) {
    using G = Geo<N, SPL, CPL>;
    extern __shared__ __align__(16) unsigned char smem[];
    const int seq = blockIdx.y, rank = static_cast<int>(blockIdx.x) % ranks;
    Scan<N, SPL, CPL> sc(p, smem, static_cast<int>(blockIdx.x) / ranks);
    stream_order();
    int32_t bits = 0;
    int begin, len;
    span_of(p.s, seq, &begin, &len, &bits);
    const int64_t slot = read_slot(p.s, seq, &bits), dest = write_slot(p.s, seq, 0, &bits);
    if (blockIdx.x == 0 && threadIdx.x == 0) flag_err(p.s.dev_err, bits);
    const int parts = min(ranks, max(1, len / min_seg));
    if (parts == 1) {
        if (rank > 0) return;   // the whole cluster agrees
        sc.load_decay();
        sc.load_seed(slot);
        sc.template run<true>(begin, begin + len);
        sc.store_end(dest);
        return;
    }
    // whole tiles a block; the last ones may have none
    const int seg = ((len + parts - 1) / parts + G::TT - 1) / G::TT * G::TT;
    const int lo = min(rank * seg, len), hi = min(lo + seg, len);
    float* hend = reinterpret_cast<float*>(smem);              // [CPL][SPL / 4][threads] of 4: a lane's own order
    float* send = hend + kThreads * CPL * SPL;                 // [CPL][threads]
    sc.load_decay();
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
        sc.ssum[j] = 0.f;
#pragma unroll
        for (int i = 0; i < SPL / 2; ++i) sc.h[j][i] = 0ull;
    }
    const bool tail = hi < len;   // somebody comes after this block
    if (tail) {
        sc.template run<false>(begin + lo, begin + hi);
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
#pragma unroll
            for (int i = 0; i < SPL / 4; ++i) {
                ulonglong2 v;
                v.x = sc.h[j][2 * i];
                v.y = sc.h[j][2 * i + 1];
                *reinterpret_cast<ulonglong2*>(hend + ((j * (SPL / 4) + i) * kThreads + threadIdx.x) * 4) = v;
            }
            send[j * kThreads + threadIdx.x] = sc.ssum[j];
        }
    }
    cluster_sync();
    if (lo < len) {
        sc.load_seed(slot);
        for (int r = 0; r < rank; ++r) {
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                const float s = ld_peer_f32(send + j * kThreads + threadIdx.x, r);
                const f32x2 ss = pack2(s, s);
#pragma unroll
                for (int i = 0; i < SPL / 4; ++i) {
                    const float4 e = ld_peer_f32x4(hend + ((j * (SPL / 4) + i) * kThreads + threadIdx.x) * 4, r);
                    f32x2* h = &sc.h[j][2 * i];
                    h[0] = fma2(ex2_2(mul2(ss, sc.a2[j][2 * i])), h[0], pack2(e.x, e.y));
                    h[1] = fma2(ex2_2(mul2(ss, sc.a2[j][2 * i + 1])), h[1], pack2(e.z, e.w));
                }
            }
        }
    }
    cluster_sync();   // all have read their peers, and the seed before any end state is stored
    if (lo < len) {
        sc.template run<true>(begin + lo, begin + hi);
        if (!tail) sc.store_end(dest);
    }
}

template <int N, int SPL, int CPL>
lar_status go(const SsmParams& p, int ranks, int min_seg, cudaStream_t st) {
    using G = Geo<N, SPL, CPL>;
    auto kern = ssm_prefill_kernel<N, SPL, CPL>;
    size_t smem = static_cast<size_t>(parts_of<N, SPL, CPL>(p).total);
    const size_t joined = static_cast<size_t>(kThreads) * CPL * (SPL + 1) * 4;
    if (smem < joined) smem = joined;
    if (cudaFuncSetAttribute(reinterpret_cast<const void*>(kern), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem)) != cudaSuccess)
        return LAR_ERR_LAUNCH;
    if (ranks > 8 && cudaFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                          cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return LAR_ERR_LAUNCH;
    const unsigned columns = static_cast<unsigned>(p.G) * ((p.per_group + G::CH - 1) / G::CH);
    return launch_ordered(kern, dim3(columns * ranks, p.s.n), kThreads, smem, ranks, st, p, ranks, min_seg);
}

// Blocks of a span: one where the columns of all spans fill the device twice over,
// else as many as fill it four times, at most 16 (the largest cluster).
template <int N, int SPL, int CPL>
lar_status pick(const SsmParams& p, cudaStream_t st) {
    using G = Geo<N, SPL, CPL>;
    const int64_t rows = static_cast<int64_t>(p.G) * ((p.per_group + G::CH - 1) / G::CH) * p.s.n;
    int ranks = 1;
    if (rows < 2 * kSms)
        while (ranks < 16 && rows * ranks < 4 * kSms && p.s.ntok >= 2 * ranks * kMinSeg) ranks *= 2;
    return go<N, SPL, CPL>(p, ranks, kMinSeg, st);
}

}  // namespace

lar_status launch_ssm_prefill(const SsmParams& p, void* stream) {
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (p.N) {
        case 16: return pick<16, 8, 1>(p, st);
        case 32: return pick<32, 8, 1>(p, st);
        case 64: return pick<64, 8, 2>(p, st);
        default: return pick<128, 8, 2>(p, st);
    }
}

}  // namespace lar

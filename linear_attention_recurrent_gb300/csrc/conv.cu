// conv.cu -- the short causal convolution in front of a recurrent layer, with its
// state (the last W - 1 inputs of a sequence) in pool slots:
//
//     y[t, c] = bias[c] + sum_{j < W} w[c, j] x[t - (W - 1) + j, c],  out = y or silu(y)
//
// Inputs before the sequence's first token come from its state; rows of a state
// are the inputs, oldest first, channels innermost.  Bound by memory: 2 W + 5
// operations for every element that is read and written once.  In plain fp32: pairs
// of channels in one instruction (as the scan has them) cost more moves than they
// saved, 112 us against 106 in the prefill.
#include <algorithm>

#include "layer_common.cuh"

namespace lar {

namespace {

constexpr int kThreads = 128;   // of a step's blocks
// Of the prefill's blocks.  16384 x 8192 bf16 on 608 blocks of 128 threads: 105 us; on
// 1216 of 64: 94 us, 5.7 TB/s of 6.7 (the tokens' groups ahead: 3; 4 and 5 are slower).
constexpr int kPre = 64;
constexpr int kTile = 16;    // tokens of a prefill tile, which blocks share out
// Blocks of the prefill on an SM.  bf16: all of a call's blocks are held at once.  The fp32
// ring, 32 KB a block, admits 6, and a call runs in two waves: 16384 x 4096, 161 us for
// the bytes that bf16 moves in 93.
constexpr int kBlocks = 8;
constexpr int kGroup = 4;    // tokens of a group of copies,
constexpr int kAhead = 3;    // groups asked for ahead of the one in work,
constexpr int kRing = kGroup * (kAhead + 1);   // and the tokens that the ring holds

// VEC channels from channel c0: one 16-byte access (8) or one element (1).
template <int VEC, bool NC>
__device__ __forceinline__ void ld_ch(const void* base, int64_t off, int64_t cs, int c0, int dt, float* f) {
    if constexpr (VEC == 8) ld8<NC>(base, off + c0, dt, f);
    else f[0] = NC ? ld_in(base, off + c0 * cs, dt) : ld_pool(base, off + c0 * cs, dt);
}

template <int VEC>
__device__ __forceinline__ void st_ch(void* base, int64_t off, int64_t cs, int c0, int dt, const float* f) {
    if constexpr (VEC == 8) st8(base, off + c0, dt, f);
    else st_out(base, off + c0 * cs, dt, f[0]);
}

// The taps and bias of VEC channels, any layout.
template <int W, int VEC>
struct Taps {
    float w[VEC][W], b[VEC];
    __device__ __forceinline__ void load(const ConvParams& p, int c0) {
        if (VEC == 8 && p.vec_w) {   // [C, W] in one piece: 8 W numbers from c0 W on
            float* f = &w[0][0];
#pragma unroll
            for (int k = 0; k < VEC * W; k += 8) ld8<true>(p.w, static_cast<int64_t>(c0) * W + k, p.w_dt, f + k);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
#pragma unroll
                for (int j = 0; j < W; ++j) w[i][j] = ld_in(p.w, (c0 + i) * p.ws[0] + j * p.ws[1], p.w_dt);
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) b[i] = 0.f;
        if (p.bias) {
            if (VEC == 8 && p.vec_b) {
                ld8<true>(p.bias, c0, p.bias_dt, b);
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) b[i] = ld_in(p.bias, (c0 + i) * p.b_s, p.bias_dt);
            }
        }
    }
    // y of the newest input u after the W - 1 in h, which it joins
    __device__ __forceinline__ void step(float (*h)[VEC], const float* u, float* y, bool silu) const {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            float a = b[i];
#pragma unroll
            for (int j = 0; j + 1 < W; ++j) a = fmaf(w[i][j], h[j][i], a);
            a = fmaf(w[i][W - 1], u[i], a);
            y[i] = silu ? silu_f(a) : a;
#pragma unroll
            for (int j = 0; j + 2 < W; ++j) h[j][i] = h[j + 1][i];
            h[W - 2][i] = u[i];
        }
    }
};

// 8 channels of a window of W inputs.
template <int W>
struct Taps8 : Taps<W, 8> {
    // y of the newest input of the window
    __device__ __forceinline__ void at(const float (*win)[8], float* y, bool silu) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            y[i] = this->b[i];
#pragma unroll
            for (int j = 0; j < W; ++j) y[i] = fmaf(this->w[i][j], win[j][i], y[i]);
        }
        if (silu) {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = silu_f(y[i]);
        }
    }
};

template <int W, int VEC>
__device__ __forceinline__ void load_state(const ConvParams& p, int64_t slot, int c0, float (*h)[VEC]) {
#pragma unroll
    for (int j = 0; j + 1 < W; ++j) {
        if (slot >= 0) {
            ld_ch<VEC, false>(p.pool, slot * p.ps[0] + j * p.ps[1], 1, c0, p.pool_dt, h[j]);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) h[j][i] = 0.f;
        }
    }
}

template <int W, int VEC>
__device__ __forceinline__ void store_state(const ConvParams& p, int64_t slot, int c0, const float (*h)[VEC]) {
    if (slot < 0) return;
#pragma unroll
    for (int j = 0; j + 1 < W; ++j)
        st_ch<VEC>(p.pool, slot * p.ps[0] + j * p.ps[1], 1, c0, p.pool_dt, h[j]);
}

// T tokens of sequence blockIdx.y.  A thread owns its channels from the state's
// load to its stores, so a seed slot may be one of the slots it then writes.
template <int W, int VEC>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(const ConvParams p) {
    const int b = blockIdx.y, c0 = (blockIdx.x * kThreads + threadIdx.x) * VEC;
    stream_order();
    int32_t bits = 0;
    const int64_t slot = read_slot(p.s, b, &bits);
    if (c0 < p.C) {
        Taps<W, VEC> taps;
        taps.load(p, c0);
        float h[W - 1][VEC], next[VEC];
        const auto input = [&](int t, float* u) {
            ld_ch<VEC, true>(p.x, b * p.xs[0] + t * p.xs[1], p.xs[2], c0, p.x_dt, u);
        };
        input(0, next);
        int64_t to = write_slot(p.s, b, 0, &bits);
        load_state<W, VEC>(p, slot, c0, h);
        for (int t = 0; t < p.s.T; ++t) {
            float u[VEC], y[VEC];
            const int64_t dest = to;
#pragma unroll
            for (int i = 0; i < VEC; ++i) u[i] = next[i];
            if (t + 1 < p.s.T) {   // on its way while this token is worked on
                input(t + 1, next);
                if (p.s.tslot) to = write_slot(p.s, b, t + 1, &bits);
            }
            taps.step(h, u, y, p.silu);
            st_ch<VEC>(p.out, b * p.os[0] + t * p.os[1], p.os[2], c0, p.out_dt, y);
            if (p.s.tslot || t + 1 == p.s.T) store_state<W, VEC>(p, dest, c0, h);
        }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) flag_err(p.s.dev_err, bits);
}

// One token of NB sequences, 8 channels a thread: the states and inputs of all of
// them are asked for at once, and the filters, larger than all of them, are read once.
// X: type of x; S: of the pool.  256 x 8192 bf16: 9.3 us (a sequence at a time 14 us);
// 5 us of it is the memory's, the rest the way from slot to state to store.
template <int W, typename X, typename S, int NB>
__global__ void __launch_bounds__(kThreads, NB == 1 ? 6 : 4) conv_token_kernel(const ConvParams p) {
    const int c0 = (blockIdx.x * kThreads + threadIdx.x) * 8, b0 = blockIdx.y * NB;
    stream_order();
    int32_t bits = 0;
    int64_t from[NB], to[NB];
#pragma unroll
    for (int k = 0; k < NB; ++k) {
        from[k] = to[k] = -1;
        if (b0 + k < p.s.n) {
            from[k] = read_slot(p.s, b0 + k, &bits);
            to[k] = write_slot(p.s, b0 + k, 0, &bits);
        }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) flag_err(p.s.dev_err, bits);
    if (c0 >= p.C) return;
    Eight<X> x[NB];
    Eight<S, false> st[NB][W - 1];
#pragma unroll
    for (int k = 0; k < NB; ++k) {
        x[k].load(p.x, min(b0 + k, p.s.n - 1) * p.xs[0] + c0);
#pragma unroll
        for (int j = 0; j + 1 < W; ++j) {
            st[k][j].zero();
            if (from[k] >= 0) st[k][j].load(p.pool, from[k] * p.ps[0] + j * p.ps[1] + c0);
        }
    }
    Taps8<W> taps;
    taps.load(p, c0);
#pragma unroll
    for (int k = 0; k < NB; ++k) {
        if (b0 + k >= p.s.n) break;
        float win[W][8];
#pragma unroll
        for (int j = 0; j + 1 < W; ++j) st[k][j].widen(win[j]);
        x[k].widen(win[W - 1]);
        float y[8];
        taps.at(win, y, p.silu);
        st8(p.out, (b0 + k) * p.os[0] + c0, p.out_dt, y);
        if (to[k] >= 0) {   // rows move up as they are; the input joins, rounded to the pool's type
#pragma unroll
            for (int j = 0; j + 2 < W; ++j) st[k][j + 1].store(p.pool, to[k] * p.ps[0] + j * p.ps[1] + c0);
            float f[8];
            x[k].widen(f);
            st8(p.pool, to[k] * p.ps[0] + (W - 2) * p.ps[1] + c0, p.pool_dt, f);
        }
    }
}

// Tiles of all spans in a row: span n takes max(1, ceil(len / kTile)) of them.  A
// block takes an equal share of the row, in runs of tiles of one span.
struct Run {
    int seq, begin, len;   // the span
    int first, end;        // the run's tokens in it
    int64_t next, last;    // the tile behind the run, and behind the block's share
};

__device__ __forceinline__ int tiles_of(int len) { return len > kTile ? (len + kTile - 1) / kTile : 1; }

// The run that starts with tile `tile` of this block's share (tile < 0: with its
// first one).  False past the share's end.  Every thread of the block calls it.
__device__ __forceinline__ bool find_run(const SlotParams& s, int64_t tile, Run* found, int64_t* sums) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tile >= 0) {   // the tiles behind a run are the next span's
        const int64_t last = found->last;
        if (tile >= last) return false;
        __syncthreads();
        if (tid == 0) {
            int32_t bits = 0;
            const int seq = found->seq + 1;
            int begin, len;
            span_of(s, seq, &begin, &len, &bits);
            const int64_t k = min(static_cast<int64_t>(tiles_of(len)), last - tile);
            *found = {seq, begin, len, 0, static_cast<int>(min(k * kTile, static_cast<int64_t>(len))), tile + k, last};
        }
        __syncthreads();
        return true;
    }
    const int per = (s.n + kPre - 1) / kPre;
    const int lo = min(tid * per, s.n), hi = min(lo + per, s.n);
    int32_t bits = 0;
    int begin, len;
    int64_t own = 0;
    for (int n = lo; n < hi; ++n) {
        span_of(s, n, &begin, &len, &bits);
        own += tiles_of(len);
    }
    int64_t incl = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += y;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    int64_t at = incl - own, total = 0;
#pragma unroll
    for (int w = 0; w < kPre / 32; ++w) {
        if (w < warp) at += sums[w];
        total += sums[w];
    }
    tile = total * blockIdx.y / gridDim.y;
    const int64_t end = total * (blockIdx.y + 1) / gridDim.y;
    if (tile >= end) return false;
    for (int n = lo; n < hi && tile >= at; ++n) {
        span_of(s, n, &begin, &len, &bits);
        const int k = tiles_of(len);
        if (tile < at + k) {
            const int64_t next = min(at + k, end);
            *found = {n, begin, len, static_cast<int>(tile - at) * kTile,
                      static_cast<int>(min((next - at) * kTile, static_cast<int64_t>(len))), next, end};
        }
        at += k;
    }
    __syncthreads();
    return true;
}

// The final state of span f.seq: its last W - 1 inputs, the seed's (h) where it is
// shorter.  The thread of the span's first tile does this for its channels: it has
// read the seed, and the final state may go to the same slot.
template <int W, int VEC, typename Input>
__device__ __forceinline__ void close_span(const ConvParams& p, const Run& f, int c0, const float (*h)[VEC],
                                           int64_t slot, const Input& input) {
    float e[W - 1][VEC];
#pragma unroll
    for (int j = 0; j + 1 < W; ++j) {
        const int t = f.len - (W - 1) + j;   // may lie before the span: input f.len + j of the seed
        if (t >= 0) {
            input(t, e[j]);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                e[j][i] = h[j][i];
#pragma unroll
                for (int m = 1; m + j + 1 < W; ++m)
                    if (f.len == m) e[j][i] = h[j + m][i];
            }
        }
    }
    store_state<W, VEC>(p, slot, c0, e);
}

// The W - 1 inputs ahead of a run are read again.  Any layout, element by element.
template <int W>
__global__ void __launch_bounds__(kPre) conv_prefill_any_kernel(const ConvParams p) {
    __shared__ Run run_s;
    __shared__ int64_t sums[kPre / 32];
    const int c0 = blockIdx.x * kPre + threadIdx.x;
    stream_order();
    for (int64_t tile = -1; find_run(p.s, tile, &run_s, sums);) {
        const Run f = run_s;
        tile = f.next;
        int32_t bits = 0;
        if (c0 < p.C) {
            Taps<W, 1> taps;
            taps.load(p, c0);
            float h[W - 1][1];
            const auto input = [&](int t, float* u) {
                u[0] = ld_in(p.x, static_cast<int64_t>(f.begin + t) * p.xs[1] + c0 * p.xs[2], p.x_dt);
            };
            if (f.first == 0) {
                int begin, len;
                span_of(p.s, f.seq, &begin, &len, &bits);
                load_state<W, 1>(p, read_slot(p.s, f.seq, &bits), c0, h);
                close_span<W, 1>(p, f, c0, h, write_slot(p.s, f.seq, 0, &bits), input);
            } else {
#pragma unroll
                for (int j = 0; j + 1 < W; ++j) input(f.first - (W - 1) + j, h[j]);
            }
#pragma unroll 4
            for (int t = f.first; t < f.end; ++t) {
                float u[1], y[1];
                input(t, u);
                taps.step(h, u, y, p.silu);
                st_out(p.out, static_cast<int64_t>(f.begin + t) * p.os[1] + c0 * p.os[2], p.out_dt, y[0]);
            }
        }
        if (blockIdx.x == 0 && threadIdx.x == 0) flag_err(p.s.dev_err, bits);
        __syncthreads();   // all have read run_s; sums is used again
    }
}

// The same, 8 channels a thread, inputs on their way through a ring of cp.async
// copies.  A thread reads back only what it copied: the ring needs no barrier.
template <int W, typename X>
__global__ void __launch_bounds__(kPre, kBlocks) conv_prefill_kernel(const ConvParams p) {
    constexpr int NCH = sizeof(X) / 2;   // 16-byte pieces of 8 channels
    extern __shared__ __align__(16) unsigned char ring[];   // [kRing][NCH][kPre] pieces
    __shared__ Run run_s;
    __shared__ int64_t sums[kPre / 32];
    const int c0 = (blockIdx.x * kPre + threadIdx.x) * 8;
    unsigned char* mine = ring + threadIdx.x * 16;
    stream_order();
    for (int64_t tile = -1; find_run(p.s, tile, &run_s, sums);) {
        const Run f = run_s;
        tile = f.next;
        int32_t bits = 0;
        if (c0 < p.C) {
            const int nt = f.end - f.first;
            const X* src = static_cast<const X*>(p.x) + static_cast<int64_t>(f.begin + f.first) * p.xs[1] + c0;
            const auto ask = [&](int g) {   // tokens of group g of the run
#pragma unroll
                for (int u = 0; u < kGroup; ++u) {
                    const int t = g * kGroup + u;
                    if (t < nt) {
                        const X* from = src + t * p.xs[1];
                        unsigned char* dst = mine + ((g % (kAhead + 1)) * kGroup + u) * NCH * kPre * 16;
#pragma unroll
                        for (int k = 0; k < NCH; ++k) cp_async16(dst + k * kPre * 16, from + k * (16 / sizeof(X)));
                    }
                }
                cp_async_commit();
            };
#pragma unroll
            for (int g = 0; g < kAhead; ++g) ask(g);
            Taps8<W> taps;
            taps.load(p, c0);
            float win[W - 1 + kGroup][8];   // the inputs before a group, and the group's
            const auto input = [&](int t, float* u) {
                ld8<true>(p.x, static_cast<int64_t>(f.begin + t) * p.xs[1] + c0, p.x_dt, u);
            };
            if (f.first == 0) {
                int begin, len;
                span_of(p.s, f.seq, &begin, &len, &bits);
                load_state<W, 8>(p, read_slot(p.s, f.seq, &bits), c0, win);
                close_span<W, 8>(p, f, c0, win, write_slot(p.s, f.seq, 0, &bits), input);
            } else {
#pragma unroll
                for (int j = 0; j + 1 < W; ++j) input(f.first - (W - 1) + j, win[j]);
            }
            int64_t o = static_cast<int64_t>(f.begin + f.first) * p.os[1] + c0;
            for (int g = 0; g * kGroup < nt; ++g) {
                ask(g + kAhead);
                cp_async_wait<kAhead>();
                const unsigned char* at = mine + (g % (kAhead + 1)) * kGroup * NCH * kPre * 16;
#pragma unroll
                for (int u = 0; u < kGroup; ++u) {   // past the last token: what the ring holds, not used
                    Eight<X, false> e;
#pragma unroll
                    for (int k = 0; k < NCH; ++k)
                        e.u[k] = *reinterpret_cast<const uint4*>(at + (u * NCH + k) * kPre * 16);
                    e.widen(win[W - 1 + u]);
                }
#pragma unroll
                for (int u = 0; u < kGroup; ++u) {
                    if (g * kGroup + u < nt) {
                        float y[8];
                        taps.at(win + u, y, p.silu);
                        st8(p.out, o + u * p.os[1], p.out_dt, y);
                    }
                }
                o += kGroup * p.os[1];
#pragma unroll
                for (int j = 0; j + 1 < W; ++j)
#pragma unroll
                    for (int i = 0; i < 8; ++i) win[j][i] = win[kGroup + j][i];
            }
        }
        if (blockIdx.x == 0 && threadIdx.x == 0) flag_err(p.s.dev_err, bits);
        cp_async_wait<0>();
        __syncthreads();   // all have read run_s; sums is used again
    }
}

template <int W, typename X, typename S, int NB>
lar_status token(const ConvParams& p, cudaStream_t st) {
    const unsigned cb = (p.C + kThreads * 8 - 1) / (kThreads * 8);
    return launch_ordered(conv_token_kernel<W, X, S, NB>, dim3(cb, (p.s.n + NB - 1) / NB), kThreads, 0, 1, st, p);
}

template <int W>
lar_status step(const ConvParams& p, cudaStream_t st) {
    using F = float;
    using H = unsigned short;
    const unsigned per = kThreads * (p.vec ? 8 : 1), cb = (p.C + per - 1) / per;
    if (!p.vec) return launch_ordered(conv_step_kernel<W, 1>, dim3(cb, p.s.n), kThreads, 0, 1, st, p);
    if (p.s.T > 1) return launch_ordered(conv_step_kernel<W, 8>, dim3(cb, p.s.n), kThreads, 0, 1, st, p);
    const bool many = static_cast<int64_t>(cb) * p.s.n >= 4 * 152;
    if (p.x_dt == LAR_BF16) {
        if (p.pool_dt == LAR_BF16) return many ? token<W, H, H, 4>(p, st) : token<W, H, H, 1>(p, st);
        return many ? token<W, H, F, 2>(p, st) : token<W, H, F, 1>(p, st);
    }
    if (p.pool_dt == LAR_BF16) return many ? token<W, F, H, 2>(p, st) : token<W, F, H, 1>(p, st);
    return many ? token<W, F, F, 2>(p, st) : token<W, F, F, 1>(p, st);
}

template <int W, typename X>
lar_status prefill_vec(const ConvParams& p, dim3 grid, cudaStream_t st) {
    const auto kern = conv_prefill_kernel<W, X>;
    const size_t smem = static_cast<size_t>(kRing) * kPre * 8 * sizeof(X);
    if (cudaFuncSetAttribute(reinterpret_cast<const void*>(kern), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem)) != cudaSuccess)
        return LAR_ERR_LAUNCH;
    return launch_ordered(kern, grid, kPre, smem, 1, st, p);
}

template <int W>
lar_status prefill(const ConvParams& p, cudaStream_t st) {
    const unsigned per = kPre * (p.vec ? 8 : 1), cb = (p.C + per - 1) / per;
    // as many blocks as the device holds at once (in bf16: see kBlocks), if disjoint spans
    // have the tiles (element by element, a thread keeps a third of the registers)
    const int64_t tiles = p.s.ntok / kTile + p.s.n, held = (kBlocks * (p.vec ? 1 : 3) * 152 + cb - 1) / cb;
    const dim3 grid(cb, static_cast<unsigned>(std::min(tiles, std::max<int64_t>(held, 1))));
    if (!p.vec) return launch_ordered(conv_prefill_any_kernel<W>, grid, kPre, 0, 1, st, p);
    return p.x_dt == LAR_BF16 ? prefill_vec<W, unsigned short>(p, grid, st) : prefill_vec<W, float>(p, grid, st);
}

}  // namespace

lar_status launch_conv_step(const ConvParams& p, void* stream) {
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return p.W == 2 ? step<2>(p, st) : p.W == 3 ? step<3>(p, st) : step<4>(p, st);
}

lar_status launch_conv_prefill(const ConvParams& p, void* stream) {
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return p.W == 2 ? prefill<2>(p, st) : p.W == 3 ? prefill<3>(p, st) : prefill<4>(p, st);
}

}  // namespace lar

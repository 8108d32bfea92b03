// conv.cu -- the short causal convolution in front of a recurrent layer, with its
// state (the last W - 1 inputs of a sequence) in pool slots:
//
//     y[t, c] = bias[c] + sum_{j < W} w[c, j] x[t - (W - 1) + j, c],  out = y or silu(y)
//
// Inputs before the sequence's first token come from its state; rows of a state
// are the inputs, oldest first, channels innermost.  Bound by memory: 2 W + 5
// operations for every element that is read and written once.
#include "layer_common.cuh"

namespace lar {

namespace {

constexpr int kThreads = 128;
constexpr int kTile = 32;    // tokens of a prefill tile

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

// The taps and bias of VEC channels.
template <int W, int VEC>
struct Taps {
    float w[VEC][W], b[VEC];
    __device__ __forceinline__ void load(const ConvParams& p, int c0) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[i][j] = ld_in(p.w, (c0 + i) * p.ws[0] + j * p.ws[1], p.w_dt);
            b[i] = p.bias ? ld_in(p.bias, (c0 + i) * p.b_s, p.bias_dt) : 0.f;
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
        float h[W - 1][VEC];
        load_state<W, VEC>(p, slot, c0, h);
        for (int t = 0; t < p.s.T; ++t) {
            float u[VEC], y[VEC];
            ld_ch<VEC, true>(p.x, b * p.xs[0] + t * p.xs[1], p.xs[2], c0, p.x_dt, u);
            taps.step(h, u, y, p.silu);
            st_ch<VEC>(p.out, b * p.os[0] + t * p.os[1], p.os[2], c0, p.out_dt, y);
            if (p.s.tslot) store_state<W, VEC>(p, write_slot(p.s, b, t, &bits), c0, h);
        }
        if (!p.s.tslot) store_state<W, VEC>(p, write_slot(p.s, b, 0, &bits), c0, h);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) flag_err(p.s.dev_err, bits);
}

// Which span and tokens tile `tile` covers: span n takes max(1, ceil(len / kTile))
// tiles, in order.  False past the last one.  Every thread of the block calls it.
struct TileOf {
    int seq, begin, len, first;   // the span, and the tile's first token in it
};

__device__ __forceinline__ int tiles_of(int len) { return len > kTile ? (len + kTile - 1) / kTile : 1; }

__device__ __forceinline__ bool find_tile(const SlotParams& s, int64_t tile, TileOf* found, int64_t* sums) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (s.n + kThreads - 1) / kThreads;
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
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) at += sums[w];
        total += sums[w];
    }
    if (tile >= total) return false;
    for (int n = lo; n < hi && tile >= at; ++n) {
        span_of(s, n, &begin, &len, &bits);
        const int k = tiles_of(len);
        if (tile < at + k) *found = {n, begin, len, static_cast<int>(tile - at) * kTile};
        at += k;
    }
    __syncthreads();
    return true;
}

// One tile of tokens of one span a block and step; the tile before supplies the
// W - 1 inputs ahead of it by reading them again.  The block of a span's first
// tile alone touches its slots: it reads the seed before it writes the final
// state, which may go to the same slot.
template <int W, int VEC>
__global__ void __launch_bounds__(kThreads) conv_prefill_kernel(const ConvParams p) {
    __shared__ TileOf tile_s;
    __shared__ int64_t sums[kThreads / 32];
    const int c0 = (blockIdx.x * kThreads + threadIdx.x) * VEC;
    stream_order();
    for (int64_t tile = blockIdx.y; find_tile(p.s, tile, &tile_s, sums); tile += gridDim.y) {
        const TileOf f = tile_s;
        int32_t bits = 0;
        if (c0 < p.C) {
            Taps<W, VEC> taps;
            taps.load(p, c0);
            float h[W - 1][VEC];
            const auto input = [&](int t, float* u) {
                ld_ch<VEC, true>(p.x, static_cast<int64_t>(f.begin + t) * p.xs[1], p.xs[2], c0, p.x_dt, u);
            };
            if (f.first == 0) {
                int begin, len;
                span_of(p.s, f.seq, &begin, &len, &bits);
                load_state<W, VEC>(p, read_slot(p.s, f.seq, &bits), c0, h);
                // the last W - 1 inputs, the seed's where the span is shorter
                float e[W - 1][VEC];
#pragma unroll
                for (int j = 0; j + 1 < W; ++j) {
                    const int t = f.len - (W - 1) + j;   // may lie before the span
                    if (t >= 0) {
                        input(t, e[j]);
                    } else {
#pragma unroll
                        for (int i = 0; i < VEC; ++i) {
                            e[j][i] = h[0][i];
#pragma unroll
                            for (int k = 1; k + 1 < W; ++k)
                                if (t + W - 1 == k) e[j][i] = h[k][i];
                        }
                    }
                }
                store_state<W, VEC>(p, write_slot(p.s, f.seq, 0, &bits), c0, e);
            } else {
#pragma unroll
                for (int j = 0; j + 1 < W; ++j) input(f.first - (W - 1) + j, h[j]);
            }
            const int end = min(f.first + kTile, f.len);
#pragma unroll 4
            for (int t = f.first; t < end; ++t) {
                float u[VEC], y[VEC];
                input(t, u);
                taps.step(h, u, y, p.silu);
                st_ch<VEC>(p.out, static_cast<int64_t>(f.begin + t) * p.os[1], p.os[2], c0, p.out_dt, y);
            }
        }
        if (blockIdx.x == 0 && threadIdx.x == 0) flag_err(p.s.dev_err, bits);
        __syncthreads();   // tile_s and sums are used again
    }
}

template <int W, int VEC>
lar_status step(const ConvParams& p, cudaStream_t st) {
    const unsigned cb = (p.C + kThreads * VEC - 1) / (kThreads * VEC);
    return launch_ordered(conv_step_kernel<W, VEC>, dim3(cb, p.s.n), kThreads, 0, 1, st, p);
}

template <int W, int VEC>
lar_status prefill(const ConvParams& p, cudaStream_t st) {
    const unsigned cb = (p.C + kThreads * VEC - 1) / (kThreads * VEC);
    // disjoint spans make at most this many tiles; a block goes on to others where they are not
    const int64_t tiles = p.s.ntok / kTile + p.s.n;
    return launch_ordered(conv_prefill_kernel<W, VEC>, dim3(cb, static_cast<unsigned>(tiles < 65535 ? tiles : 65535)),
                          kThreads, 0, 1, st, p);
}

}  // namespace

lar_status launch_conv_step(const ConvParams& p, void* stream) {
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (p.W) {
        case 2: return p.vec ? step<2, 8>(p, st) : step<2, 1>(p, st);
        case 3: return p.vec ? step<3, 8>(p, st) : step<3, 1>(p, st);
        default: return p.vec ? step<4, 8>(p, st) : step<4, 1>(p, st);
    }
}

lar_status launch_conv_prefill(const ConvParams& p, void* stream) {
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (p.W) {
        case 2: return p.vec ? prefill<2, 8>(p, st) : prefill<2, 1>(p, st);
        case 3: return p.vec ? prefill<3, 8>(p, st) : prefill<3, 1>(p, st);
        default: return p.vec ? prefill<4, 8>(p, st) : prefill<4, 1>(p, st);
    }
}

}  // namespace lar

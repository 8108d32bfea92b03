// attn.cu -- attention of a step's T tokens over a paged cache of keys and values
// (attn_decode): out = softmax(scale q K^T) V, causal among the step's tokens, G query
// heads to a key/value head, optionally the last `window` tokens alone.
//
// Mathematics.  Pages hold codes c with one scale a (page, head): K = s c, V = r c.
// Scores are kept in base 2 and r is moved into the exponent: with
//     e_j = scale log2(e) q.K_j + log2 r_j,   M = max e_j
// the output is sum 2^(e_j - M) c_j / sum 2^(e_j - M) / r_j, so that the products take
// codes as they lie (an e4m3 number is exact in fp16, and so is a bf16 query once its
// row is scaled by a power of two), and what fp16 rounds is a weight in [0, 2^8].
// Both products run on the tensor cores with fp32 sums.  bf16 pages take weights split
// into two bf16 terms (16 bits of each weight).
//
// Work.  A tile is WT tokens of one pair (sequence, key/value head, 16 MT query rows).
// The tiles of all pairs in a row are dealt out to the blocks in equal shares, a
// multiple of four tiles, whatever the lengths, which only the device knows: a block's
// four warps take its tiles in turn, every warp with a ring of its own in shared memory
// that no other warp waits for, its own running maximum, sum and output, joined
// once a pair.  A pair that several blocks share leaves its parts in the workspace, and
// attn_join adds them.
#include <cuda_fp16.h>

#include <type_traits>

#include "layer_common.cuh"
#include "serve_params.h"

namespace lar {

int cached_occupancy(const void* kern, int threads, size_t smem, size_t smem_max, int* sms_out);

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxBlocks = 608;    // of a call: bounds the workspace
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.f;      // a weight may grow to 2^8 before the sums are scaled down

// Tokens of a warp's tile: 8 KB of keys and values, at least a granule of 16.
constexpr int tile_tokens(int D, bool f8) {
    const int t = 8192 / (2 * D * (f8 ? 1 : 2));
    return t > 32 ? 32 : t < 16 ? 16 : t;
}

constexpr int kStages = 3;

template <int D, bool F8, int MT>
struct Shape {
    static constexpr int WT = tile_tokens(D, F8);
    static constexpr int ROW = D * (F8 ? 1 : 2);       // bytes of a token's row
    static constexpr int CH = ROW / 16;                // its 16-byte chunks
    static constexpr int TILE = WT * ROW;              // bytes of a tile's keys
    static constexpr int RING = kStages * 2 * TILE;    // a warp's
    static constexpr int KS = D / 16;                  // steps of the first product
    static constexpr int NT = D / 8;                   // column tiles of the second
    static constexpr int ROWS = 16 * MT;
    static constexpr int QF = KS * MT * 32 * 16;       // query fragments, bytes
    static constexpr int PART = ROWS * (D + 2);        // floats of a part: sums, maxima, outputs
    static constexpr int JOIN = kWarps * PART * 4;
    static constexpr int BODY = kWarps * RING > JOIN ? kWarps * RING : JOIN;
    static constexpr int SMEM = BODY + QF + ROWS * 4;
    static constexpr bool QREG = D * MT <= 128;        // fragments stay in registers
};

__device__ __forceinline__ void cp16_zfill(unsigned dst, const void* src, bool take) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}

__device__ __forceinline__ uint4 lds16(unsigned a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

__device__ __forceinline__ uint2 lds8(unsigned a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}

// Where chunk c of a tile's row lies: the rows that a warp reads at once fall on
// different banks.  Rows of 64 bytes share a line of 128 in pairs.
template <int CH, bool KEYS>
__device__ __forceinline__ int place(int row, int c) {
    if constexpr (CH == 4) {
        const int line = row >> 1, cc = ((row & 1) << 2) + c;
        return line * 128 + ((cc ^ ((line & 3) << 1)) << 4);
    } else {
        return row * (CH * 16) + ((KEYS ? c ^ ((row & 1) << 2) : c ^ (((row >> 1) & 3) << 1)) << 4);
    }
}

// two e4m3 codes as fp16 numbers (exact)
__device__ __forceinline__ unsigned f16_of_e4m3(unsigned short x) {
    unsigned y;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(y) : "h"(x));
    return y;
}

__device__ __forceinline__ unsigned pack_f16x2(float lo, float hi) {
    unsigned y;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
    return y;
}

// d += a b, 16 x 8 x 16, fp32 sums
template <bool F8>
__device__ __forceinline__ void mma(float* d, const unsigned* a, unsigned b0, unsigned b1) {
    if constexpr (F8)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The places that any of sequence b's rows see: [lo, hi); own: the first token's place.
struct Seen {
    int lo, hi, own;
};

__device__ __forceinline__ Seen seen_of(const AttnParams& p, int b, int32_t* bits) {
    const int64_t len = ld_idx(p.c.lens, b * p.c.len_s, p.c.len_dt);
    const int cap = p.c.M * p.c.page;
    if (len < 0) return {0, 0, 0};   // no sequence here
    if (len + p.T > cap) *bits |= LAR_DEVERR_SEQLEN;
    const int own = static_cast<int>(len < cap ? len : cap);
    const int hi = min(own + p.T, cap), lo = p.window ? max(0, own - p.window + 1) : 0;
    return {lo, max(hi, lo), own};
}

template <int WT>
__device__ __forceinline__ int tiles_of(const Seen& s) {
    return s.hi > s.lo ? (s.hi + WT - 1) / WT - s.lo / WT : 0;
}

// All tiles of the call, and for a block that asks with `first`: the sequence that
// holds tile `first` and how many tiles come before it.  By the whole block.
struct Deal {
    int64_t total;
    int b;
    int64_t before;
};

template <int WT, int THREADS>
__device__ __forceinline__ int64_t sum_tiles(const AttnParams& p, int64_t* part, int lo, int hi, int32_t* bits) {
    int64_t mine = 0;
    for (int b = lo; b < hi; ++b) mine += tiles_of<WT>(seen_of(p, b, bits));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t run = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, run, off);
        if (lane >= off) run += y;
    }
    if (lane == 31) part[warp] = run;
    __syncthreads();
    int64_t before = 0;
    for (int w = 0; w < warp; ++w) before += part[w];
    if (threadIdx.x == THREADS - 1) part[THREADS / 32] = before + run;
    __syncthreads();
    return before + run - mine;   // tiles before this thread's sequences
}

template <int D, bool F8, int MT>
__global__ void __launch_bounds__(kThreads, 2) attn_kernel(const __grid_constant__ AttnParams p, int row_blocks) {
    using S = Shape<D, F8, MT>;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int64_t scan_s[kWarps + 1];
    __shared__ int at_b;
    __shared__ int64_t at_before;
    unsigned char* qf = smem + S::BODY;
    float* qc = reinterpret_cast<float*>(qf + S::QF);   // what a row's products are multiplied by
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
    const unsigned ring = static_cast<unsigned>(__cvta_generic_to_shared(smem)) + warp * S::RING;
    stream_order();
    int32_t bits = 0;

    // this block's share of the tiles
    const int per = (p.B + kThreads - 1) / kThreads, sb0 = min(p.B, tid * per), sb1 = min(p.B, sb0 + per);
    const int pairs = p.c.H * row_blocks;   // of a sequence
    const int64_t before = sum_tiles<S::WT, kThreads>(p, scan_s, sb0, sb1, &bits);
    const int64_t total = scan_s[kWarps] * pairs;
    int64_t share = (total + gridDim.x - 1) / gridDim.x;
    share = (share + kWarps - 1) / kWarps * kWarps;
    int64_t i0 = share * blockIdx.x;
    const int64_t i1 = min(total, i0 + share);
    if (blockIdx.x == 0) flag_err(p.dev_err, bits);
    if (i0 >= i1) return;
    {
        int64_t run = before * pairs;
        for (int b = sb0; b < sb1; ++b) {
            const int64_t n = static_cast<int64_t>(tiles_of<S::WT>(seen_of(p, b, &bits))) * pairs;
            if (i0 >= run && i0 < run + n) {
                at_b = b;
                at_before = run;
            }
            run += n;
        }
    }
    __syncthreads();
    int b = at_b;
    int64_t b_first = at_before;   // tile index of sequence b's first tile

    while (i0 < i1) {
        const Seen seen = seen_of(p, b, &bits);
        const int n_tiles = tiles_of<S::WT>(seen);
        if (n_tiles == 0 || i0 >= b_first + static_cast<int64_t>(n_tiles) * pairs) {
            b_first += static_cast<int64_t>(n_tiles) * pairs;
            ++b;
            continue;
        }
        const int pair = static_cast<int>((i0 - b_first) / n_tiles);
        const int64_t pair_first = b_first + static_cast<int64_t>(pair) * n_tiles;
        const int s0 = static_cast<int>(i0 - pair_first);
        const int s1 = static_cast<int>(min(static_cast<int64_t>(n_tiles), i1 - pair_first));
        const int h = pair / row_blocks, rb = pair % row_blocks;
        const int rows = min(S::ROWS, p.G * p.T - rb * S::ROWS), row0 = rb * S::ROWS;   // row = token G + head of the group

        // the queries as fragments: lane (g, t4) of step ks holds dimensions
        // (ks / CS * 4 + t4) * CD + ks % CS * 4 + {0, 1, 2, 3} of rows g and g + 8
        constexpr int CD = F8 ? 16 : 8, CS = CD / 4;   // dimensions and steps of a chunk
        for (int r = warp; r < S::ROWS; r += kWarps) {
            float x[D / 32];
            float top = 0.f;
            const int row = row0 + r, tk = row / p.G, hq = h * p.G + row % p.G;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const int d = (lane + (i >> 1 << 5)) * 2 + (i & 1);   // pairs of neighbours
                x[i] = r < rows ? ld_in(p.q, b * p.qs[0] + tk * p.qs[1] + hq * p.qs[2] + d * p.qs[3], p.q_dt) : 0.f;
                top = fmaxf(top, fabsf(x[i]));
            }
            float mul = 1.f, back = 1.f;
            if constexpr (F8) {   // the greatest to 2^14 .. 2^15: fp16 holds what bf16 does, 2^-28 of it downwards
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                const int e = static_cast<int>(__float_as_uint(top) >> 23);   // biased
                if (e > 15 && e < 240) {
                    mul = __uint_as_float(static_cast<unsigned>(254 + 14 - e) << 23);
                    back = __uint_as_float(static_cast<unsigned>(e - 14) << 23);
                }
            }
#pragma unroll
            for (int i = 0; i < D / 32; i += 2) {
                const int d = (lane + (i >> 1 << 5)) * 2;
                const int c = d / CD, ks = (c >> 2) * CS + d % CD / 4, w = (d & 3) >> 1;   // w: a0/a1 or a2/a3
                const int owner = ((r & 7) << 2) + (c & 3);
                const unsigned v = F8 ? pack_f16x2(x[i] * mul, x[i + 1] * mul) : pack_bf16x2(x[i], x[i + 1]);
                *reinterpret_cast<unsigned*>(qf + (((r >> 4) * S::KS + ks) * 32 + owner) * 16 + (w * 2 + ((r >> 3) & 1)) * 4) = v;
            }
            if (lane == 0) qc[r] = p.scale * kLog2e * back;
        }
        __syncthreads();

        unsigned qr[S::QREG ? MT : 1][S::QREG ? S::KS : 1][4];
        if constexpr (S::QREG) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int k = 0; k < S::KS; ++k)
                    *reinterpret_cast<uint4*>(qr[m][k]) = *reinterpret_cast<const uint4*>(qf + ((m * S::KS + k) * 32 + lane) * 16);
        }
        float c0[MT], c1[MT];
        int e0[MT], e1[MT];   // one past the last place that the rows see
        float m0[MT], m1[MT], l0[MT], l1[MT];
        float o[MT][S::NT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            c0[m] = qc[m * 16 + g];
            c1[m] = qc[m * 16 + g + 8];
            e0[m] = seen.own + (row0 + m * 16 + g) / p.G + 1;
            e1[m] = seen.own + (row0 + m * 16 + g + 8) / p.G + 1;
            m0[m] = m1[m] = -INFINITY;
            l0[m] = l1[m] = 0.f;
#pragma unroll
            for (int n = 0; n < S::NT; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[m][n][k] = 0.f;
        }

        // This warp's tiles: s0 + warp, + 4, ...  Lane j of a batch knows the page and the
        // scales of granule (16 tokens) j % GR of tile j / GR; batches are read one ahead.
        constexpr int GR = S::WT / 16, BT = 32 / GR;
        const int first_tile = seen.lo / S::WT;
        const int mine = s1 - s0 > warp ? (s1 - s0 - warp + kWarps - 1) / kWarps : 0;
        auto place_of = [&](int i) { return (first_tile + s0 + warp + i * kWarps) * S::WT; };
        auto page_of = [&](int batch) {   // -1: nothing to see there
            const int i = batch * BT + lane / GR;
            const int pos = place_of(i) + lane % GR * 16;
            if (i >= mine || pos >= seen.hi || pos + 16 <= seen.lo) return -1;
            const int64_t id = ld_idx(p.c.table, b * p.c.tab_s[0] + (pos / p.c.page) * p.c.tab_s[1], p.c.tab_dt);
            if (id >= p.c.P) bits |= LAR_DEVERR_PAGE;
            return id < 0 || id >= p.c.P ? -1 : static_cast<int>(id);
        };
        auto scales_of = [&](int id, float& ks, float& vs) {
            if (F8 && id >= 0) {
                ks = __ldg(p.c.k_scale + id * p.c.kss[0] + h * p.c.kss[1]);
                vs = __ldg(p.c.v_scale + id * p.c.vss[0] + h * p.c.vss[1]);
            } else {
                ks = vs = 1.f;
            }
        };
        int id0 = page_of(0), id1 = page_of(1);
        float ks0, vs0, ks1, vs1;
        scales_of(id0, ks0, vs0);
        scales_of(id1, ks1, vs1);
        int load_batch = 0, id_l0 = id0, id_l1 = id1;   // the loads run ahead of the products

        auto load = [&](int i) {
            if (i < mine) {
                if (i / BT != load_batch) {
                    load_batch = i / BT;
                    id_l0 = id_l1;
                    id_l1 = page_of(load_batch + 1);
                }
                const int pos = place_of(i);
                const unsigned dst = ring + i % kStages * (2 * S::TILE);
#pragma unroll
                for (int gr = 0; gr < GR; ++gr) {
                    const int id = __shfl_sync(0xffffffffu, id_l0, i % BT * GR + gr);
                    const int in_page = (pos + gr * 16) % p.c.page;
                    const int64_t idc = id < 0 ? 0 : id;
                    const char* kp = static_cast<const char*>(p.c.k) + (idc * p.c.ks[0] + in_page * p.c.ks[1] + h * p.c.ks[2]) * (F8 ? 1 : 2);
                    const char* vp = static_cast<const char*>(p.c.v) + (idc * p.c.vs[0] + in_page * p.c.vs[1] + h * p.c.vs[2]) * (F8 ? 1 : 2);
#pragma unroll
                    for (int j = 0; j < 16 * S::CH / 32; ++j) {
                        const int row = (lane + j * 32) / S::CH, c = (lane + j * 32) % S::CH;
                        const int at = pos + gr * 16 + row;
                        const bool take = id >= 0 && at >= seen.lo && at < seen.hi;
                        const int64_t kof = row * p.c.ks[1] * (F8 ? 1 : 2) + c * 16, vof = row * p.c.vs[1] * (F8 ? 1 : 2) + c * 16;
                        cp16_zfill(dst + place<S::CH, true>(gr * 16 + row, c), take ? kp + kof : static_cast<const char*>(p.c.k), take);
                        cp16_zfill(dst + S::TILE + place<S::CH, false>(gr * 16 + row, c), take ? vp + vof : static_cast<const char*>(p.c.v), take);
                    }
                }
            }
            cp_async_commit();   // always, so that groups are counted alike
        };
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) load(i);

        for (int i = 0; i < mine; ++i) {
            if (i > 0 && i % BT == 0) {
                const int batch = i / BT;
                id0 = id1;
                ks0 = ks1;
                vs0 = vs1;
                id1 = page_of(batch + 1);
                scales_of(id1, ks1, vs1);
            }
            cp_async_wait<kStages - 2>();
            __syncwarp();
            load(i + kStages - 1);
            const unsigned kt = ring + i % kStages * (2 * S::TILE), vt = kt + S::TILE;
            const int pos = place_of(i);

            float s[MT][S::WT / 8][4];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < S::WT / 8; ++n)
#pragma unroll
                    for (int k = 0; k < 4; ++k) s[m][n][k] = 0.f;
#pragma unroll
            for (int j = 0; j < S::CH / 4; ++j) {
                unsigned qs[MT][CS][4];
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int w = 0; w < CS; ++w)
                        if constexpr (S::QREG) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) qs[m][w][k] = qr[m][j * CS + w][k];
                        } else {
                            *reinterpret_cast<uint4*>(qs[m][w]) =
                                *reinterpret_cast<const uint4*>(qf + ((m * S::KS + j * CS + w) * 32 + lane) * 16);
                        }
#pragma unroll
                for (int n = 0; n < S::WT / 8; ++n) {
                    const uint4 u = lds16(kt + place<S::CH, true>(n * 8 + g, j * 4 + t4));
                    const unsigned x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int w = 0; w < CS; ++w) {
                        unsigned b0, b1;
                        if constexpr (F8) {
                            b0 = f16_of_e4m3(static_cast<unsigned short>(x[w]));
                            b1 = f16_of_e4m3(static_cast<unsigned short>(x[w] >> 16));
                        } else {
                            b0 = x[2 * w];
                            b1 = x[2 * w + 1];
                        }
#pragma unroll
                        for (int m = 0; m < MT; ++m) mma<F8>(s[m][n], qs[m][w], b0, b1);
                    }
                }
            }

            // scores in base 2, with the values' scale, and the running maximum
            const bool inner = pos >= (p.window ? seen.own + p.T - p.window : 0) && pos + S::WT <= seen.own + 1;   // all rows see all of it
            float inv[GR];
            unsigned pa[MT][S::WT / 16][4], pb[F8 ? 1 : MT][F8 ? 1 : S::WT / 16][4];
            float gk[GR], gv[GR];
#pragma unroll
            for (int gr = 0; gr < GR; ++gr) {
                const int src = i % BT * GR + gr;
                gk[gr] = __shfl_sync(0xffffffffu, ks0, src);
                const float r = __shfl_sync(0xffffffffu, vs0, src);
                const int id = __shfl_sync(0xffffffffu, id0, src);
                gv[gr] = id < 0 ? -INFINITY : F8 ? log2f(r) : 0.f;
                inv[gr] = F8 ? 1.f / r : 1.f;
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
                for (int n = 0; n < S::WT / 8; ++n) {
                    const float f0 = c0[m] * gk[n / 2], f1 = c1[m] * gk[n / 2];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float x = fmaf(s[m][n][k], k < 2 ? f0 : f1, gv[n / 2]);
                        if (!inner) {
                            const int at = pos + n * 8 + t4 * 2 + (k & 1), e = k < 2 ? e0[m] : e1[m];
                            if (at >= min(e, seen.hi) || (p.window && at < e - p.window) || gv[n / 2] == -INFINITY) x = -INFINITY;
                        }
                        s[m][n][k] = x;
                        if (k < 2) t0 = fmaxf(t0, x);
                        else t1 = fmaxf(t1, x);
                    }
                }
#pragma unroll
                for (int off = 1; off < 4; off <<= 1) {
                    t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, off));
                    t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, off));
                }
                const bool up = t0 > m0[m] + kSlack || t1 > m1[m] + kSlack;
                if (__any_sync(0xffffffffu, up)) {
                    const float n0 = fmaxf(m0[m], t0), n1 = fmaxf(m1[m], t1);
                    const float a0 = m0[m] == -INFINITY ? 0.f : exp2_f(m0[m] - n0), a1 = m1[m] == -INFINITY ? 0.f : exp2_f(m1[m] - n1);
                    m0[m] = n0;
                    m1[m] = n1;
                    l0[m] *= a0;
                    l1[m] *= a1;
#pragma unroll
                    for (int n = 0; n < S::NT; ++n) {
                        o[m][n][0] *= a0;
                        o[m][n][1] *= a0;
                        o[m][n][2] *= a1;
                        o[m][n][3] *= a1;
                    }
                }
                const float b0 = m0[m] == -INFINITY ? 0.f : m0[m], b1 = m1[m] == -INFINITY ? 0.f : m1[m];
#pragma unroll
                for (int gr = 0; gr < GR; ++gr) {
                    float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
                    for (int n = 2 * gr; n < 2 * gr + 2; ++n) {
                        float x[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) x[k] = exp2_f(s[m][n][k] - (k < 2 ? b0 : b1));
                        sum0 += x[0] + x[1];
                        sum1 += x[2] + x[3];
                        if constexpr (F8) {
                            pa[m][gr][(n & 1) * 2] = pack_f16x2(x[0], x[1]);
                            pa[m][gr][(n & 1) * 2 + 1] = pack_f16x2(x[2], x[3]);
                        } else {
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const unsigned hi = pack_bf16x2(x[2 * k], x[2 * k + 1]);
                                pa[m][gr][(n & 1) * 2 + k] = hi;
                                pb[m][gr][(n & 1) * 2 + k] = pack_bf16x2(x[2 * k] - __uint_as_float(hi << 16), x[2 * k + 1] - __uint_as_float(hi & 0xffff0000u));
                            }
                        }
                    }
                    l0[m] = fmaf(sum0, inv[gr], l0[m]);
                    l1[m] = fmaf(sum1, inv[gr], l1[m]);
                }
            }

            // the values.  A weight of 0 does not keep an infinity or NaN out of a sum: where a
            // tile that not all rows see all of holds one, each of the step's tokens has its
            // product with the places that it sees, and its rows alone take it.
            bool apart = false;
            if (!inner && p.T > 1) {
                for (int j = lane; j < S::TILE / 16; j += 32) {
                    const uint4 u = lds16(vt + j * 16);
                    const unsigned x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        apart |= F8 ? (__vcmpeq4(x[w] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0u)
                                    : (__vcmpgeu2(x[w] & 0x7fff7fffu, 0x7f807f80u) != 0u);
                }
                apart = __any_sync(0xffffffffu, apart);
            }
            auto values = [&](auto careful) {
#pragma unroll
                for (int gr = 0; gr < GR; ++gr) {
                    const int ra = gr * 16 + t4 * 2;
                    auto add = [&](int n, unsigned b0, unsigned b1) {
                        if constexpr (!decltype(careful)::value) {
#pragma unroll
                            for (int m = 0; m < MT; ++m) {
                                mma<F8>(o[m][n], pa[m][gr], b0, b1);
                                if constexpr (!F8) mma<F8>(o[m][n], pb[m][gr], b0, b1);
                            }
                        } else {
                            for (int tk = 0; tk < p.T; ++tk) {
                                const int end = min(seen.own + tk + 1, seen.hi), begin = p.window ? seen.own + tk + 1 - p.window : 0;
                                unsigned keep[2];
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const int at = pos + ra + k * 8;
                                    keep[k] = (at >= begin && at < end ? 0xffffu : 0u) | (at + 1 >= begin && at + 1 < end ? 0xffff0000u : 0u);
                                }
#pragma unroll
                                for (int m = 0; m < MT; ++m) {
                                    float y[4] = {0.f, 0.f, 0.f, 0.f};
                                    mma<F8>(y, pa[m][gr], b0 & keep[0], b1 & keep[1]);
                                    if constexpr (!F8) mma<F8>(y, pb[m][gr], b0 & keep[0], b1 & keep[1]);
                                    if (e0[m] == seen.own + tk + 1) {
                                        o[m][n][0] += y[0];
                                        o[m][n][1] += y[1];
                                    }
                                    if (e1[m] == seen.own + tk + 1) {
                                        o[m][n][2] += y[2];
                                        o[m][n][3] += y[3];
                                    }
                                }
                            }
                        }
                    };
#pragma unroll
                    for (int ci = 0; ci < (S::CH + 7) / 8; ++ci) {
                        uint4 u[4];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int row = ra + (r & 1) + (r >> 1) * 8;
                            if constexpr (S::CH == 4) {   // half a chunk a lane
                                const uint2 w = lds8(vt + place<S::CH, false>(row, g >> 1) + (g & 1) * 8);
                                u[r] = make_uint4(w.x, w.y, 0u, 0u);
                            } else {
                                u[r] = lds16(vt + place<S::CH, false>(row, g + ci * 8));
                            }
                        }
                        constexpr int W = S::CH == 4 ? 2 : 4;
#pragma unroll
                        for (int w = 0; w < W; ++w) {
                            auto word = [&](int r) { return w == 0 ? u[r].x : w == 1 ? u[r].y : w == 2 ? u[r].z : u[r].w; };
                            if constexpr (F8) {
                                unsigned x[2], y[2];
                                x[0] = __byte_perm(word(0), word(1), 0x5140);
                                x[1] = __byte_perm(word(0), word(1), 0x7362);
                                y[0] = __byte_perm(word(2), word(3), 0x5140);
                                y[1] = __byte_perm(word(2), word(3), 0x7362);
#pragma unroll
                                for (int d = 0; d < 4; ++d)
                                    add((ci * W + w) * 4 + d, f16_of_e4m3(static_cast<unsigned short>(x[d >> 1] >> ((d & 1) * 16))),
                                        f16_of_e4m3(static_cast<unsigned short>(y[d >> 1] >> ((d & 1) * 16))));
                            } else {
#pragma unroll
                                for (int d = 0; d < 2; ++d)
                                    add((ci * W + w) * 2 + d, __byte_perm(word(0), word(1), d ? 0x7632 : 0x5410),
                                        __byte_perm(word(2), word(3), d ? 0x7632 : 0x5410));
                            }
                        }
                    }
                }
            };
            if (apart) values(std::true_type{});
            else values(std::false_type{});
        }

        // the warps' parts together
        cp_async_wait<0>();
        __syncthreads();
        float* part = reinterpret_cast<float*>(smem) + warp * S::PART;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
            for (int off = 1; off < 4; off <<= 1) {
                l0[m] += __shfl_xor_sync(0xffffffffu, l0[m], off);
                l1[m] += __shfl_xor_sync(0xffffffffu, l1[m], off);
            }
            const int r0 = m * 16 + g, r1 = r0 + 8;
            if (t4 == 0) {
                part[r0] = m0[m];
                part[r1] = m1[m];
                part[S::ROWS + r0] = l0[m];
                part[S::ROWS + r1] = l1[m];
            }
            // column tile n of lane t4 holds dimensions of the groups 2 t4 and 2 t4 + 1
            constexpr int PER = S::CH == 4 ? 8 : F8 ? 16 : 8;   // column tiles (and neighbouring dimensions) of a group's piece
#pragma unroll
            for (int n = 0; n < S::NT; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int d = ((n / PER) * 8 + t4 * 2 + (k & 1)) * PER + n % PER;
                    part[2 * S::ROWS + (k < 2 ? r0 : r1) * D + d] = o[m][n][k];
                }
        }
        __syncthreads();
        const bool whole = s0 == 0 && s1 == n_tiles;
        float* ws = p.ws + (2 * static_cast<int64_t>(blockIdx.x) + (s0 == 0)) * S::PART;
        const float* parts = reinterpret_cast<const float*>(smem);
        for (int idx = tid; idx < rows * (D / 4); idx += kThreads) {
            const int r = idx / (D / 4), d = idx % (D / 4) * 4;
            float mx = -INFINITY, l = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, parts[w * S::PART + r]);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float pm = parts[w * S::PART + r], pl = parts[w * S::PART + S::ROWS + r];
                const float f = pm == -INFINITY ? 0.f : exp2_f(pm - mx);
                if (pm == -INFINITY && !(pl != pl)) continue;   // saw nothing; but NaN goes on
                const float4 x = *reinterpret_cast<const float4*>(parts + w * S::PART + 2 * S::ROWS + r * D + d);
                const float fu = pm == -INFINITY ? 1.f : f;
                l += fu * pl;
                acc.x += fu * x.x;
                acc.y += fu * x.y;
                acc.z += fu * x.z;
                acc.w += fu * x.w;
            }
            if (whole) {
                const int row = row0 + r, tk = row / p.G, hq = h * p.G + row % p.G;
                const float il = l == 0.f ? 0.f : 1.f / l;
                const float y[4] = {acc.x * il, acc.y * il, acc.z * il, acc.w * il};
                const int64_t at = b * p.os[0] + tk * p.os[1] + hq * p.os[2];
#pragma unroll
                for (int k = 0; k < 4; ++k) st_out(p.out, at + (d + k) * p.os[3], p.o_dt, y[k]);
                if (d == 0 && p.lse) p.lse[b * p.ls[0] + tk * p.ls[1] + hq * p.ls[2]] = l == 0.f ? -INFINITY : (mx + log2f(l)) * kLn2;
            } else {
                *reinterpret_cast<float4*>(ws + 2 * S::ROWS + r * D + d) = acc;
                if (d == 0) {
                    ws[r] = mx;
                    ws[S::ROWS + r] = l;
                }
            }
        }
        __syncthreads();   // the ring and the fragments are written again
        i0 = pair_first + s1;
    }
    flag_err(p.dev_err, bits);
}

// Adds the parts of pairs that several blocks shared; rows of sequences that see
// nothing get zeros.  A block a (pair, row), its warps taking parts in turn.
constexpr int kJoinWarps = 8;

template <int D, bool F8, int MT>
__global__ void __launch_bounds__(kJoinWarps * 32) attn_join(const __grid_constant__ AttnParams p, int row_blocks, int blocks) {
    using S = Shape<D, F8, MT>;
    constexpr int PER = D / 32;   // dimensions of a lane
    __shared__ int64_t scan_s[kJoinWarps + 1];
    __shared__ int64_t before_s;
    __shared__ float m_s[kJoinWarps], l_s[kJoinWarps], o_s[kJoinWarps][D];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    stream_order();
    const int pairs = p.c.H * row_blocks, threads = kJoinWarps * 32;
    const int b = blockIdx.x / pairs, pair = blockIdx.x % pairs, h = pair / row_blocks, row0 = pair % row_blocks * S::ROWS;
    const int r = blockIdx.y;
    if (row0 + r >= p.G * p.T) return;
    int32_t bits = 0;
    const int per = (p.B + threads - 1) / threads, sb0 = min(p.B, tid * per), sb1 = min(p.B, sb0 + per);
    int64_t before = sum_tiles<S::WT, kJoinWarps * 32>(p, scan_s, sb0, sb1, &bits);
    const int64_t total = scan_s[kJoinWarps] * pairs;
    if (b >= sb0 && b < sb1) {
        for (int i = sb0; i < b; ++i) before += tiles_of<S::WT>(seen_of(p, i, &bits));
        before_s = before;
    }
    __syncthreads();
    const int n = tiles_of<S::WT>(seen_of(p, b, &bits));
    const int row = row0 + r, tk = row / p.G, hq = h * p.G + row % p.G;
    const int64_t at = b * p.os[0] + tk * p.os[1] + hq * p.os[2];
    if (n == 0) {
        for (int d = tid; d < D; d += threads) st_out(p.out, at + d * p.os[3], p.o_dt, 0.f);
        if (tid == 0 && p.lse) p.lse[b * p.ls[0] + tk * p.ls[1] + hq * p.ls[2]] = -INFINITY;
        return;
    }
    int64_t share = (total + blocks - 1) / blocks;
    share = (share + kWarps - 1) / kWarps * kWarps;
    const int64_t first = before_s * pairs + static_cast<int64_t>(pair) * n;
    const int64_t g0 = first / share, g1 = (first + n - 1) / share;
    if (g0 == g1) return;   // one block had all of it
    float m = -INFINITY, l = 0.f, o[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) o[k] = 0.f;
    for (int64_t i = g0 + warp; i <= g1; i += kJoinWarps) {
        const float* part = p.ws + (2 * i + (i == g0)) * S::PART;
        const float pm = part[r], pl = part[S::ROWS + r];
        float x[PER];
#pragma unroll
        for (int k = 0; k < PER; ++k) x[k] = part[2 * S::ROWS + r * D + lane + k * 32];
        const float nm = fmaxf(m, pm);
        const float a = m == -INFINITY ? 0.f : exp2_f(m - nm), c = pm == -INFINITY ? 0.f : exp2_f(pm - nm);
        const bool none = pm == -INFINITY && pl == 0.f;
        l = fmaf(l, a, none ? 0.f : pl * (pm == -INFINITY ? 1.f : c));
#pragma unroll
        for (int k = 0; k < PER; ++k) o[k] = fmaf(o[k], a, none ? 0.f : x[k] * (pm == -INFINITY ? 1.f : c));
        m = nm;
    }
    if (lane == 0) {
        m_s[warp] = m;
        l_s[warp] = l;
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) o_s[warp][lane + k * 32] = o[k];
    __syncthreads();
    float mx = -INFINITY, ls = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) mx = fmaxf(mx, m_s[w]);
    float f[kJoinWarps];
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
        f[w] = m_s[w] == -INFINITY ? (l_s[w] != l_s[w] ? 1.f : 0.f) : exp2_f(m_s[w] - mx);
        ls += f[w] * l_s[w];
    }
    const float il = ls == 0.f ? 0.f : 1.f / ls;
    for (int d = tid; d < D; d += threads) {
        float y = 0.f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) y += f[w] * o_s[w][d];
        st_out(p.out, at + d * p.os[3], p.o_dt, y * il);
    }
    if (tid == 0 && p.lse) p.lse[b * p.ls[0] + tk * p.ls[1] + hq * p.ls[2]] = ls == 0.f ? -INFINITY : (mx + log2f(ls)) * kLn2;
}

// Rows of a pair: 16, or 32 where a step has more and the registers hold their outputs
int row_tiles(int T, int G, int D) { return T * G > 16 && D <= 128 ? 2 : 1; }

template <int D, bool F8, int MT>
lar_status launch(const AttnParams& p, cudaStream_t stream) {
    using S = Shape<D, F8, MT>;
    const int row_blocks = (p.G * p.T + S::ROWS - 1) / S::ROWS;
    auto kern = attn_kernel<D, F8, MT>;
    int sms = 0;
    const int occ = cached_occupancy(reinterpret_cast<const void*>(kern), kThreads, S::SMEM, S::SMEM, &sms);
    if (occ < 1) return LAR_ERR_LAUNCH;
    // no more blocks than the longest sequences that the table admits could fill
    const int64_t cap = static_cast<int64_t>(p.c.M) * p.c.page;
    const int64_t most = (static_cast<int64_t>(p.B) * p.c.H * row_blocks * ((cap + S::WT - 1) / S::WT + 1) + kWarps - 1) / kWarps;
    int64_t blocks = static_cast<int64_t>(sms) * occ;
    if (blocks > kMaxBlocks) blocks = kMaxBlocks;
    if (blocks > most) blocks = most;
    const int64_t pairs = static_cast<int64_t>(p.B) * p.c.H * row_blocks;
    if (pairs > (int64_t{1} << 31) - 1) return LAR_ERR_SHAPE;
    const lar_status st = launch_ordered(kern, dim3(static_cast<unsigned>(blocks)), kThreads, S::SMEM, 1, stream, p, row_blocks);
    if (st != LAR_OK) return st;
    return launch_ordered(attn_join<D, F8, MT>, dim3(static_cast<unsigned>(pairs), S::ROWS), kJoinWarps * 32, 0, 1, stream, p,
                          row_blocks, static_cast<int>(blocks));
}

template <int D>
lar_status launch_d(const AttnParams& p, cudaStream_t stream) {
    const int mt = row_tiles(p.T, p.G, D);
    if constexpr (D <= 128) {
        if (mt == 2) return p.c.e4m3 ? launch<D, true, 2>(p, stream) : launch<D, false, 2>(p, stream);
    }
    return p.c.e4m3 ? launch<D, true, 1>(p, stream) : launch<D, false, 1>(p, stream);
}

}  // namespace

int64_t attn_workspace_floats(int T, int G, int D) {
    return int64_t{2} * kMaxBlocks * 16 * row_tiles(T, G, D) * (D + 2);
}

lar_status launch_attn(const AttnParams& p, void* stream) {
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return p.c.D == 64 ? launch_d<64>(p, s) : p.c.D == 128 ? launch_d<128>(p, s) : launch_d<256>(p, s);
}

}  // namespace lar

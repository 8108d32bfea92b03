// attn.cu -- attention of a step's T tokens over a paged cache of keys and values
// (attn_decode): out = softmax(scale q K^T) V, causal among the step's tokens, G query
// heads to a key/value head, optionally the last `window` tokens alone.
//
// Mathematics.  Pages hold codes c with one scale a (page, head): K = s c, V = r c.
// Scores are kept in base 2 and r is moved into the exponent: with
//     e_j = scale log2(e) q.K_j + log2 r_j,   M = max e_j
// the output is sum 2^(e_j - M) c_j / sum 2^(e_j - M) / r_j, so that the products take
// codes as they lie (an e4m3 number is exact in fp16, and so is a bf16 query once its
// row is scaled by a power of two), and what fp16 rounds is a weight in [0, 2^15].
// Both products run on the tensor cores with fp32 sums.  bf16 pages take weights split
// into two bf16 terms (16 bits of each weight).
//
// Both products are taken transposed, S^T = K Q^T and O^T = V^T P^T, tokens and dimensions
// along the 16 rows of an instruction and 8 query rows along its columns: the G T rows of a
// step are few, and the other way around half of every instruction, and of every register
// of sums, would be padding.  A lane's 16 bytes of a key are four steps' operands in an
// order that the queries are laid out to match; a value's 16 bytes are the same dimensions
// of eight steps.
//
// A weight is taken against a reference that is moved only when a weight passes 2^8 of what
// the greatest was then: no maximum is looked for, only that none is too large.  The greatest
// is 2^7 then in fp16, which reaches 2^16, and so keeps 11 bits of weights down to 2^-21 of it and
// 2^-32 of it below (a long tail of those may be all that a row has, beside values near 0); 1 in
// bf16, whose range is fp32's.
//
// The sums are not divided before the end, and those of 16-bit values near the end of their
// range pass fp32's: a warp with a sum past 2^115 takes its tiles once more, against references
// 2^60 higher, where 2^30 values sum up to less than 2^107.  The joins add up 2432 such sums at
// most.
//
// Work.  A tile is WT tokens of one pair (sequence, key/value head, 8 NR query rows).
// The tiles of all pairs in a row, each pair with kStart more for what its beginning and
// end cost, are dealt out to the blocks in equal shares, a multiple of four, whatever the
// lengths, which only the device knows: a block's
// four warps take its tiles in turn, every warp with a ring of its own in shared memory
// that no other warp waits for, its own running maximum, sum and output, joined
// once a pair.  A pair that several blocks share leaves its parts in the workspace, and
// attn_join adds them.
//
// Bound: the bytes of the visible codes.  64 sequences of 0 to 8192 places, 8 heads of 128,
// e4m3: 97 to 112 us by the lengths drawn where the copy rate admits 81; bf16 163 to 170 of 161; 1 x
// 131000, 2 heads of 256: 35 of 20; 32 x 4 tokens x 0 to 4096: 42 to 47 of 21 (twice the
// instructions of one token).  What is lost: a block's beginning and end (3 and 4 us), and issue: 37
// to 47 % of the cycles at 8 to 12 warps an SM.  Of 8 NR rows a pair, as many as registers hold, more
// rows walk the pages again: 16 sequences of 0 to 4096, groups of 8 heads of 128, 48 us for 4 tokens
// (32 rows), 73 for 5, 81 for 8, 145 for 16; of 256, 25 for 2 (16 rows), 31 for 4.
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
// Tiles that a pair's beginning and end count as: 64 sequences and 32 x 4 tokens take 125 and
// 110 us at 4 tiles of 8 KB, 101 and 46 at 16 of 4 KB, 104 and 42 at 24, 105 and 45 at 48.
constexpr int kStart = 20;
constexpr float kSlack = 8.f;      // a weight may grow to 2^8 of its first before the sums are scaled down
constexpr float kMost = 4.1538374868278621e34f;   // 2^115: sums that the joins have room for
constexpr float kFresh16 = 7.f;    // log2 of the greatest weight where a reference is moved, in fp16
constexpr float kLow = -60.f;      // log2 of first weights where there are greater ones

// Tokens of a warp's tile: 4 KB of keys and values, at least a granule of 16.  Of 8 KB, one
// sequence takes 10.2 us instead of 9.5 and 32 x 4 tokens 56 instead of 46; 64 sequences the same.
constexpr int tile_tokens(int D, bool f8) {
    const int t = 4096 / (2 * D * (f8 ? 1 : 2));
    return t > 32 ? 32 : t < 16 ? 16 : t;
}

constexpr float kNone = -3e38f;    // the maximum of a row that has seen nothing: below any score

template <int D, bool F8, int NR>
struct Shape {
    static constexpr int WT = tile_tokens(D, F8);
    static constexpr int GR = WT / 16;                 // granules of 16 tokens: a page at most
    static constexpr int ES = F8 ? 1 : 2;
    static constexpr int ROW = D * ES;                 // bytes of a token's row
    static constexpr int CH = ROW / 16;                // its 16-byte chunks
    static constexpr int TILE = WT * ROW;              // bytes of a tile's keys
    static constexpr int STAGES = 2;                   // three and four: 64 sequences 113 and 110 us instead of 102
    static constexpr int RING = STAGES * 2 * TILE;     // a warp's
    static constexpr int KS = D / 16;                  // steps of the first product
    static constexpr int MT = D / 16;                  // row tiles of the second
    static constexpr int ROWS = 8 * NR;
    static constexpr int QF = KS * NR * 32 * 8;        // query fragments, bytes
    static constexpr int PART = ROWS * (D + 2);        // floats of a part: maxima, sums, outputs
    static constexpr int JOIN = kWarps * PART * 4;
    static constexpr int BODY = kWarps * RING > JOIN ? kWarps * RING : JOIN;
    static constexpr int SMEM = BODY + QF + ROWS * 4;
    // fragments stay in registers, unless a third block fits an SM without them (32 x 4 tokens 52 -> 46 us)
    static constexpr bool QREG = D * NR <= 128 || (D == 256 && NR == 1);
    static constexpr int BLOCKS = D < 256 && D * NR <= 256 ? 3 : 2;   // an SM, by registers
};

__device__ __forceinline__ void cp16_zfill(unsigned dst, const void* src, bool take) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}

__device__ __forceinline__ void cp16(unsigned dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}

// Plain loads, so that the compiler may ask for them early (never past a wait, which clobbers memory)
__device__ __forceinline__ uint4 lds16(const unsigned char* a) { return *reinterpret_cast<const uint4*>(a); }
__device__ __forceinline__ uint2 lds8(const unsigned char* a) { return *reinterpret_cast<const uint2*>(a); }

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

// four e4m3 codes as fp16 numbers (exact)
__device__ __forceinline__ void f16_of_e4m3(unsigned x, unsigned& lo, unsigned& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
}

__device__ __forceinline__ unsigned pack_f16x2(float lo, float hi) {
    unsigned y;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
    return y;
}

// An 8 x 8 matrix of 16-bit numbers, two neighbours of row lane / 4 in a lane: transposed
__device__ __forceinline__ unsigned turned(unsigned x) {
    unsigned y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// d += a b, 16 x 8 x 16, fp32 sums
template <bool F8>
__device__ __forceinline__ void mma(float* d, const unsigned* a, unsigned b0, unsigned b1) {
    if constexpr (F8)
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The places that any of sequence b's rows see: [lo, hi), none where they are equal; own: the
// first token's place, which may lie past the table and its window still reach back into it.
// Up to 2^30 places and windows below 2^31: from 3 2^30 + 64 on no window does, and what is
// reckoned with `own`, modulo 2^32, comes out right where there is anything to see.
struct Seen {
    int lo, hi;
    unsigned own;
};

__device__ __forceinline__ Seen seen_of(const AttnParams& p, int b, int32_t* bits) {
    const int64_t len = ld_idx(p.c.lens, b * p.c.len_s, p.c.len_dt);
    const unsigned cap = static_cast<unsigned>(p.c.M) * p.c.page, far = (3u << 30) + 64u, window = p.window;
    if (len < 0) return {0, 0, 0u};   // no sequence here
    const unsigned own = len < far ? static_cast<unsigned>(len) : far;
    if (own + p.T > cap) *bits |= LAR_DEVERR_SEQLEN;
    const unsigned hi = min(own + p.T, cap), lo = window && own >= window ? own + 1 - window : 0u;
    return {static_cast<int>(min(lo, hi)), static_cast<int>(hi), own};
}

// Tiles of a pair, and what it counts as where the work is dealt out: kStart in front of them
template <int WT>
__device__ __forceinline__ int tiles_of(const Seen& s) {
    return s.hi > s.lo ? (s.hi + WT - 1) / WT - s.lo / WT : 0;
}

template <int WT>
__device__ __forceinline__ int weight_of(const Seen& s) {
    const int n = tiles_of<WT>(s);
    return n ? n + kStart : 0;
}

// Tiles of a block: equal shares, in whole turns of its warps
__device__ __forceinline__ int64_t share_of(int64_t total, int64_t blocks) {
    return ((total + blocks - 1) / blocks + kWarps - 1) / kWarps * kWarps;
}

// What the sequences' pairs count as, one pair a sequence, in part[THREADS / 32]; returns
// those before sequence `lo` of this thread's [lo, hi).  By the whole block.
template <int WT, int THREADS>
__device__ __forceinline__ int64_t sum_weights(const AttnParams& p, int64_t* part, int lo, int hi, int32_t* bits) {
    int64_t mine = 0;
    for (int b = lo; b < hi; ++b) mine += weight_of<WT>(seen_of(p, b, bits));
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

template <int D, bool F8, int NR>
__global__ void __launch_bounds__(kThreads, (Shape<D, F8, NR>::BLOCKS)) attn_kernel(const __grid_constant__ AttnParams p, int row_blocks, int by_row) {
    using S = Shape<D, F8, NR>;
    constexpr int GR = S::GR, CH = S::CH;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int64_t scan_s[kWarps + 1];
    __shared__ int at_b;
    __shared__ int64_t at_before;
    unsigned char* qf = smem + S::BODY;
    float* qc = reinterpret_cast<float*>(qf + S::QF);   // what a row's products are multiplied by
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
    unsigned char* const ring = smem + warp * S::RING;
    const unsigned ring_a = static_cast<unsigned>(__cvta_generic_to_shared(ring));
    stream_order();
    int32_t bits = 0;

    // this block's share of the tiles
    const int per = (p.B + kThreads - 1) / kThreads, sb0 = min(p.B, tid * per), sb1 = min(p.B, sb0 + per);
    const int pairs = p.c.H * row_blocks;   // of a sequence
    const int64_t before = sum_weights<S::WT, kThreads>(p, scan_s, sb0, sb1, &bits);
    const int64_t total = scan_s[kWarps] * pairs;
    const int64_t share = share_of(total, gridDim.x);
    int64_t i0 = share * blockIdx.x;
    const int64_t i1 = min(total, i0 + share);
    // Pairs that end in another block than they begin in: one a block at most, or, where pairs
    // are few, by pair.
    int4* const split = reinterpret_cast<int4*>(p.ws);
    float* const parts_at = p.ws + 4 * kMaxBlocks;
    if (tid == 0 && !by_row) split[blockIdx.x].x = -1;
    // rows of sequences that see nothing
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        const Seen seen = seen_of(p, b, &bits);
        if (seen.hi > seen.lo) continue;
        if (by_row && tid < pairs) split[b * pairs + tid].x = -1;
        for (int i = tid; i < p.T * p.Hq * D; i += kThreads) {
            const int d = i % D, hq = i / D % p.Hq, tk = i / D / p.Hq;
            st_out(p.out, b * p.os[0] + tk * p.os[1] + hq * p.os[2] + d * p.os[3], p.o_dt, 0.f);
            if (d == 0 && p.lse) p.lse[b * p.ls[0] + tk * p.ls[1] + hq * p.ls[2]] = -INFINITY;
        }
    }
    flag_err(p.dev_err, bits);
    if (i0 >= i1) return;
    {
        int64_t run = before * pairs;
        for (int b = sb0; b < sb1; ++b) {
            const int64_t n = static_cast<int64_t>(weight_of<S::WT>(seen_of(p, b, &bits))) * pairs;
            if (i0 >= run && i0 < run + n) {
                at_b = b;
                at_before = run;
            }
            run += n;
        }
    }
    __syncthreads();
    int b = at_b;
    int64_t b_first = at_before;   // where sequence b begins

    // where this lane's pieces of 32 chunks of a granule lie, here and there
    constexpr int RS = 32 / CH > 0 ? 32 / CH : 1;    // rows that 32 chunks cover
    const int row_l = lane / CH, c_l = lane % CH;
    const int64_t k_step = p.c.ks[1] * S::ES * RS, v_step = p.c.vs[1] * S::ES * RS;
    const int64_t k_lane = p.c.ks[1] * S::ES * row_l + c_l * 16, v_lane = p.c.vs[1] * S::ES * row_l + c_l * 16;

    while (i0 < i1) {
        const Seen seen = seen_of(p, b, &bits);
        const int n_tiles = tiles_of<S::WT>(seen), weight = weight_of<S::WT>(seen);
        if (i0 >= b_first + static_cast<int64_t>(weight) * pairs) {
            b_first += static_cast<int64_t>(weight) * pairs;
            ++b;
            continue;
        }
        const int pair = static_cast<int>((i0 - b_first) / weight);
        const int64_t pair_first = b_first + static_cast<int64_t>(pair) * weight + kStart;
        const int s0 = static_cast<int>(max(int64_t{0}, i0 - pair_first));
        const int s1 = static_cast<int>(min(static_cast<int64_t>(n_tiles), i1 - pair_first));
        i0 = pair_first + n_tiles;   // on to the next pair
        if (s1 <= s0) continue;      // its beginning alone
        const int h = pair / row_blocks, rb = pair % row_blocks;
        const int rows = min(S::ROWS, p.G * p.T - rb * S::ROWS), row0 = rb * S::ROWS;   // row = token G + head of the group

        // This warp's tiles: s0 + warp, + 4, ...  Lane j of a batch knows where granule j % GR
        // of tile j / GR lies and its scales; batches are read one ahead.
        constexpr int BT = 32 / GR;
        const int tile0 = seen.lo / S::WT + s0 + warp;
        const int mine = s1 - s0 > warp ? (s1 - s0 - warp + kWarps - 1) / kWarps : 0;
        auto place_of = [&](int i) { return (tile0 + i * kWarps) * S::WT; };
        auto page_of = [&](int batch) {   // -1: nothing to see there
            const int i = batch * BT + lane / GR;
            const int pos = place_of(i) + lane % GR * 16;
            if (i >= mine || pos >= seen.hi || pos + 16 <= seen.lo) return -1;
            const int64_t id = ld_idx(p.c.table, b * p.c.tab_s[0] + (pos / p.c.page) * p.c.tab_s[1], p.c.tab_dt);
            if (id >= p.c.P) bits |= LAR_DEVERR_PAGE;
            return id < 0 || id >= p.c.P ? -1 : static_cast<int>(id);
        };
        int id_next = page_of(0);
        int64_t k_at = -1, v_at = -1;      // bytes from the caches' beginnings to the granule, this lane's pieces apart
        float ks_raw = 1.f, vs_raw = 1.f;  // the scales of the batch that is being loaded
        bool there = false;
        auto load_batch = [&](int batch) {
            there = id_next >= 0;
            const int in_page = (place_of(batch * BT + lane / GR) + lane % GR * 16) % p.c.page;
            k_at = there ? (id_next * p.c.ks[0] + in_page * p.c.ks[1] + h * p.c.ks[2]) * S::ES : -1;
            v_at = there ? (id_next * p.c.vs[0] + in_page * p.c.vs[1] + h * p.c.vs[2]) * S::ES : -1;
            if (F8 && there) {
                ks_raw = __ldg(p.c.k_scale + id_next * p.c.kss[0] + h * p.c.kss[1]);
                vs_raw = __ldg(p.c.v_scale + id_next * p.c.vss[0] + h * p.c.vss[1]);
            }
            id_next = page_of(batch + 1);
        };
        load_batch(0);
        auto load = [&](int i) {
            if (i < mine) {
                if (i > 0 && i % BT == 0) load_batch(i / BT);
                const int pos = place_of(i);
                const unsigned dst = ring_a + i % S::STAGES * (2 * S::TILE);
#pragma unroll
                for (int gr = 0; gr < GR; ++gr) {
                    const int src = i % BT * GR + gr, p0 = pos + gr * 16;
                    const int64_t ka = __shfl_sync(0xffffffffu, k_at, src), va = __shfl_sync(0xffffffffu, v_at, src);
                    const char *kp = static_cast<const char*>(p.c.k) + ka + k_lane, *vp = static_cast<const char*>(p.c.v) + va + v_lane;
                    if (ka >= 0 && p0 >= seen.lo && p0 + 16 <= seen.hi) {
#pragma unroll
                        for (int j = 0; j < CH / 2; ++j) {
                            const int row = gr * 16 + row_l + j * RS;
                            cp16(dst + place<CH, true>(row, c_l), kp);
                            cp16(dst + S::TILE + place<CH, false>(row, c_l), vp);
                            kp += k_step;
                            vp += v_step;
                        }
                    } else {   // zeros where there is nothing to see (there may be no page at all: any address will do)
                        const char* const nowhere = reinterpret_cast<const char*>(p.ws);
                        for (int j = 0; j < CH / 2; ++j) {
                            const int row = gr * 16 + row_l + j * RS, at = pos + row;
                            const bool take = ka >= 0 && at >= seen.lo && at < seen.hi;
                            cp16_zfill(dst + place<CH, true>(row, c_l), take ? kp : nowhere, take);
                            cp16_zfill(dst + S::TILE + place<CH, false>(row, c_l), take ? vp : nowhere, take);
                            kp += k_step;
                            vp += v_step;
                        }
                    }
                }
            }
            cp_async_commit();   // always, so that groups are counted alike
        };
#pragma unroll
        for (int i = 0; i < S::STAGES - 1; ++i) load(i);

        // the queries as fragments: lane (g, t4) of step ks holds dimensions
        // (ks / CS * 4 + t4) * CD + ks % CS * 4 + {0, 1, 2, 3} of row g
        constexpr int CD = F8 ? 16 : 8, CS = CD / 4;   // dimensions and steps of a chunk
        unsigned xq[S::ROWS / kWarps][D / 64];   // pairs of neighbours; all of a warp's rows asked for at once
#pragma unroll
        for (int e = 0; e < S::ROWS / kWarps; ++e) {
            const int r = warp + e * kWarps, row = row0 + r, tk = row / p.G, hq = h * p.G + row % p.G;
            const unsigned short* src = static_cast<const unsigned short*>(p.q) + b * p.qs[0] + tk * p.qs[1] + hq * p.qs[2];
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const int64_t d = (lane + i * 32) * 2;
                xq[e][i] = r >= rows ? 0u
                           : p.q_pairs ? __ldg(reinterpret_cast<const unsigned*>(src + d))
                                       : __ldg(src + d * p.qs[3]) | static_cast<unsigned>(__ldg(src + (d + 1) * p.qs[3])) << 16;
            }
        }
#pragma unroll
        for (int e = 0; e < S::ROWS / kWarps; ++e) {
            const int r = warp + e * kWarps;
            float mul = 1.f, back = 1.f;
            if constexpr (F8) {   // the greatest to 2^14 .. 2^15: fp16 holds what bf16 does, 2^-28 of it downwards
                unsigned top = 0;   // bf16 magnitudes in order as whole numbers
#pragma unroll
                for (int i = 0; i < D / 64; ++i) top = max(top, max(xq[e][i] & 0x7fffu, xq[e][i] >> 16 & 0x7fffu));
                const int x = static_cast<int>(__reduce_max_sync(0xffffffffu, top) >> 7);   // biased exponent
                if (x > 15 && x < 255) {
                    mul = __uint_as_float(static_cast<unsigned>(254 + 14 - x) << 23);
                    back = __uint_as_float(static_cast<unsigned>(x - 14) << 23);
                }
            }
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const int d = (lane + i * 32) * 2;
                const int c = d / CD, ks = (c >> 2) * CS + d % CD / 4, w = (d & 3) >> 1;
                const int owner = ((r & 7) << 2) + (c & 3);
                const unsigned v = F8 ? pack_f16x2(__uint_as_float(xq[e][i] << 16) * mul, __uint_as_float(xq[e][i] & 0xffff0000u) * mul) : xq[e][i];
                *reinterpret_cast<unsigned*>(qf + (((r >> 3) * S::KS + ks) * 32 + owner) * 8 + w * 4) = v;
            }
            if (lane == 0) qc[r] = p.scale * kLog2e * back;
        }
        __syncthreads();

        uint2 qr[S::QREG ? NR : 1][S::QREG ? S::KS : 1];
        auto query = [&](int n, int k) { return *reinterpret_cast<const uint2*>(qf + ((n * S::KS + k) * 32 + lane) * 8); };
        if constexpr (S::QREG) {
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int k = 0; k < S::KS; ++k) qr[n][k] = query(n, k);
        }
        // this lane's rows: n 8 + t4 2 + {0, 1}
        float cf[NR][2], mx[NR][2], l[NR][2];
        unsigned end[NR][2];   // one past the row's own place
        float o[NR][S::MT][4];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int r = n * 8 + t4 * 2 + k;
                cf[n][k] = qc[r];
                end[n][k] = seen.own + (row0 + r) / p.G + 1;
                mx[n][k] = kNone;
                l[n][k] = 0.f;
            }
#pragma unroll
            for (int m = 0; m < S::MT; ++m)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[n][m][k] = 0.f;
        }
        float gk_l = 1.f, gv_l = 0.f, gi_l = 1.f;   // of this lane's granule: the keys' scale, log2 and inverse of the values'
        float fresh = F8 ? kFresh16 : 0.f;   // log2 of the greatest weight where a reference is moved

        for (int i = 0;; ++i) {
            if (i >= mine) {
                if (F8 || fresh != 0.f) break;
                unsigned over = 0;   // rows with sums that are too large, or no numbers
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int m = 0; m < S::MT; ++m)
#pragma unroll
                        for (int k = 0; k < 4; ++k) over |= !(fabsf(o[n][m][k]) <= kMost) ? 1u << (n * 2 + (k & 1)) : 0u;
                if (!__any_sync(0xffffffffu, over != 0)) break;
                // rows whose scores are no numbers are not helped, and leave the others as they are
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float all = l[n][r];
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) all += __shfl_xor_sync(0xffffffffu, all, off);
                        if (!(all < INFINITY)) over &= ~(1u << (n * 2 + r));
                    }
                if (!__any_sync(0xffffffffu, over != 0)) break;
                // once more from the beginning, with room
                fresh = kLow;
#pragma unroll
                for (int n = 0; n < NR; ++n) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        mx[n][k] = kNone;
                        l[n][k] = 0.f;
                    }
#pragma unroll
                    for (int m = 0; m < S::MT; ++m)
#pragma unroll
                        for (int k = 0; k < 4; ++k) o[n][m][k] = 0.f;
                }
                id_next = page_of(0);
                load_batch(0);
                __syncwarp();   // the ring is read no more
#pragma unroll
                for (int j = 0; j < S::STAGES - 1; ++j) load(j);
                i = 0;
            }
            if (i % BT == 0) {   // the loads are at this batch already, and not at the next one
                gk_l = ks_raw;
                gv_l = !there ? -INFINITY : F8 ? log2f(vs_raw) : 0.f;
                gi_l = F8 ? 1.f / vs_raw : 1.f;
            }
            cp_async_wait<S::STAGES - 2>();
            __syncwarp();
            load(i + S::STAGES - 1);
            const unsigned char *kt = ring + i % S::STAGES * (2 * S::TILE), *vt = kt + S::TILE;
            const int pos = place_of(i);

            float s[GR][NR][4];
#pragma unroll
            for (int gr = 0; gr < GR; ++gr)
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int k = 0; k < 4; ++k) s[gr][n][k] = 0.f;
#pragma unroll
            for (int j = 0; j < CH / 4; ++j) {
                uint2 qs[NR][CS];
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int w = 0; w < CS; ++w) {
                        if constexpr (S::QREG) qs[n][w] = qr[n][j * CS + w];
                        else qs[n][w] = query(n, j * CS + w);
                    }
#pragma unroll
                for (int gr = 0; gr < GR; ++gr) {
                    const uint4 u = lds16(kt + place<CH, true>(gr * 16 + g, j * 4 + t4)), v = lds16(kt + place<CH, true>(gr * 16 + g + 8, j * 4 + t4));
                    const unsigned x[4] = {u.x, u.y, u.z, u.w}, y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int w = 0; w < CS; ++w) {
                        unsigned a[4];
                        if constexpr (F8) {
                            f16_of_e4m3(x[w], a[0], a[2]);
                            f16_of_e4m3(y[w], a[1], a[3]);
                        } else {
                            a[0] = x[2 * w];
                            a[1] = y[2 * w];
                            a[2] = x[2 * w + 1];
                            a[3] = y[2 * w + 1];
                        }
#pragma unroll
                        for (int n = 0; n < NR; ++n) mma<F8>(s[gr][n], a, qs[n][w].x, qs[n][w].y);
                    }
                }
            }

            // scores in base 2 with the values' scale, against the maximum so far
            float gk[GR], gv[GR], gi[GR];
#pragma unroll
            for (int gr = 0; gr < GR; ++gr) {
                const int src = i % BT * GR + gr;
                gk[gr] = __shfl_sync(0xffffffffu, gk_l, src);
                gv[gr] = __shfl_sync(0xffffffffu, gv_l, src);
                gi[gr] = __shfl_sync(0xffffffffu, gi_l, src);
            }
            // all rows see all of it (a granule that no page has is not seen: a query that is no number
            // would make one of it)
            bool inner = pos >= (p.window ? static_cast<int>(seen.own + p.T - p.window) : 0) && pos + S::WT <= seen.own + 1;
#pragma unroll
            for (int gr = 0; gr < GR; ++gr) inner &= gv[gr] != -INFINITY;
            // element k of granule gr, row tile n: token g + 8 (k / 2), row k % 2 of the lane's
            auto against = [&](int gr, int n, int k, float top) {
                const float x = fmaf(s[gr][n][k], cf[n][k & 1] * gk[gr], gv[gr] - top);
                if (inner) return x;
                const int at = pos + gr * 16 + g + (k >> 1) * 8;
                const unsigned e = end[n][k & 1];
                return at >= min(e, static_cast<unsigned>(seen.hi)) || (p.window && at < static_cast<int>(e - p.window)) || gv[gr] == -INFINITY ? -INFINITY : x;
            };
            float w[GR][NR][4];
            float high = -INFINITY;
#pragma unroll
            for (int gr = 0; gr < GR; ++gr)
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        w[gr][n][k] = against(gr, n, k, mx[n][k & 1]);
                        high = fmaxf(high, w[gr][n][k]);
                    }
            if (__any_sync(0xffffffffu, high > kSlack + fresh)) {
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float top = mx[n][r];
#pragma unroll
                        for (int gr = 0; gr < GR; ++gr) top = fmaxf(top, fmaxf(against(gr, n, r, fresh), against(gr, n, r + 2, fresh)));
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                        const float f = exp2_f(mx[n][r] - top);
                        mx[n][r] = top;
                        l[n][r] *= f;
#pragma unroll
                        for (int m = 0; m < S::MT; ++m) {
                            o[n][m][r] *= f;
                            o[n][m][r + 2] *= f;
                        }
#pragma unroll
                        for (int gr = 0; gr < GR; ++gr) {
                            w[gr][n][r] = against(gr, n, r, top);
                            w[gr][n][r + 2] = against(gr, n, r + 2, top);
                        }
                    }
            }
            // the weights, turned so that a lane has tokens t4 2 + {0, 1} (and + 8) of row g
            unsigned pa[GR][NR][2], pb[F8 ? 1 : GR][F8 ? 1 : NR][2];
#pragma unroll
            for (int gr = 0; gr < GR; ++gr)
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float x = exp2_f(w[gr][n][2 * k]), y = exp2_f(w[gr][n][2 * k + 1]);
                        l[n][0] = fmaf(x, gi[gr], l[n][0]);
                        l[n][1] = fmaf(y, gi[gr], l[n][1]);
                        if constexpr (F8) {
                            pa[gr][n][k] = turned(pack_f16x2(x, y));
                        } else {
                            const unsigned hi = pack_bf16x2(x, y);
                            pa[gr][n][k] = turned(hi);
                            pb[gr][n][k] = turned(pack_bf16x2(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u)));
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
                    for (int e = 0; e < 4; ++e)
                        apart |= F8 ? (__vcmpeq4(x[e] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0u)
                                    : (__vcmpgeu2(x[e] & 0x7fff7fffu, 0x7f807f80u) != 0u);
                }
                apart = __any_sync(0xffffffffu, apart);
            }
            auto values = [&](auto careful) {
#pragma unroll
                for (int gr = 0; gr < GR; ++gr) {
                    const int ra = gr * 16 + t4 * 2;
                    auto add = [&](int m, const unsigned* a) {
                        if constexpr (!decltype(careful)::value) {
#pragma unroll
                            for (int n = 0; n < NR; ++n) {
                                mma<F8>(o[n][m], a, pa[gr][n][0], pa[gr][n][1]);
                                if constexpr (!F8) mma<F8>(o[n][m], a, pb[gr][n][0], pb[gr][n][1]);
                            }
                        } else {
                            for (int tk = 0; tk < p.T; ++tk) {
                                const int last = min(seen.own + tk + 1, static_cast<unsigned>(seen.hi)), first = p.window ? static_cast<int>(seen.own + tk + 1 - p.window) : 0;
                                unsigned keep[2];
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const int at = pos + ra + k * 8;
                                    keep[k] = (at >= first && at < last ? 0xffffu : 0u) | (at + 1 >= first && at + 1 < last ? 0xffff0000u : 0u);
                                }
                                const unsigned v[4] = {a[0] & keep[0], a[1] & keep[0], a[2] & keep[1], a[3] & keep[1]};
#pragma unroll
                                for (int n = 0; n < NR; ++n) {
                                    float y[4] = {0.f, 0.f, 0.f, 0.f};
                                    mma<F8>(y, v, pa[gr][n][0], pa[gr][n][1]);
                                    if constexpr (!F8) mma<F8>(y, v, pb[gr][n][0], pb[gr][n][1]);
#pragma unroll
                                    for (int r = 0; r < 2; ++r)
                                        if (end[n][r] == seen.own + tk + 1) {
                                            o[n][m][r] += y[r];
                                            o[n][m][r + 2] += y[r + 2];
                                        }
                                }
                            }
                        }
                    };
#pragma unroll
                    for (int ci = 0; ci < (CH + 7) / 8; ++ci) {
                        uint4 u[4];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int row = ra + (r & 1) + (r >> 1) * 8;
                            if constexpr (CH == 4) {   // half a chunk a lane
                                const uint2 h2 = lds8(vt + place<CH, false>(row, g >> 1) + (g & 1) * 8);
                                u[r] = make_uint4(h2.x, h2.y, 0u, 0u);
                            } else {
                                u[r] = lds16(vt + place<CH, false>(row, g + ci * 8));
                            }
                        }
                        // row tile m has dimensions 2 m and 2 m + 1 (of the lane's piece) in its rows g and g + 8
                        constexpr int W = CH == 4 ? 2 : 4;
#pragma unroll
                        for (int e = 0; e < W; ++e) {
                            auto word = [&](int r) { return e == 0 ? u[r].x : e == 1 ? u[r].y : e == 2 ? u[r].z : u[r].w; };
                            if constexpr (F8) {
#pragma unroll
                                for (int d = 0; d < 2; ++d) {
                                    const unsigned x = __byte_perm(word(0), word(1), d ? 0x7362 : 0x5140), y = __byte_perm(word(2), word(3), d ? 0x7362 : 0x5140);
                                    unsigned a[4];
                                    f16_of_e4m3(x, a[0], a[1]);
                                    f16_of_e4m3(y, a[2], a[3]);
                                    add((ci * W + e) * 2 + d, a);
                                }
                            } else {
                                const unsigned a[4] = {__byte_perm(word(0), word(1), 0x5410), __byte_perm(word(0), word(1), 0x7632),
                                                       __byte_perm(word(2), word(3), 0x5410), __byte_perm(word(2), word(3), 0x7632)};
                                add(ci * W + e, a);
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
        constexpr int PER = CH == 4 ? 8 : CD;   // neighbouring dimensions of a lane's piece
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int at = n * 8 + t4 * 2 + r;
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) l[n][r] += __shfl_xor_sync(0xffffffffu, l[n][r], off);
                if (g == 0) {
                    part[at] = mx[n][r];
                    part[S::ROWS + at] = l[n][r];
                }
#pragma unroll
                for (int m = 0; m < S::MT; ++m) {
                    const int d = (m / (PER / 2) * 8 + g) * PER + m % (PER / 2) * 2;
                    *reinterpret_cast<float2*>(part + 2 * S::ROWS + at * D + d) = make_float2(o[n][m][r], o[n][m][r + 2]);
                }
            }
        __syncthreads();
        const bool whole = s0 == 0 && s1 == n_tiles;
        if (s0 == 0 && tid == 0 && (by_row || !whole))
            split[by_row ? b * pairs + pair : blockIdx.x] =
                make_int4(whole ? -1 : b, pair, static_cast<int>((pair_first + n_tiles - 1) / share), blockIdx.x);
        float* ws = parts_at + (2 * static_cast<int64_t>(blockIdx.x) + (s0 == 0)) * S::PART;
        const float* parts = reinterpret_cast<const float*>(smem);
        for (int idx = tid; idx < rows * (D / 4); idx += kThreads) {
            const int r = idx / (D / 4), d = idx % (D / 4) * 4;
            float top = kNone, sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, parts[w * S::PART + r]);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = exp2_f(parts[w * S::PART + r] - top);
                const float4 x = *reinterpret_cast<const float4*>(parts + w * S::PART + 2 * S::ROWS + r * D + d);
                sum = fmaf(f, parts[w * S::PART + S::ROWS + r], sum);
                acc.x = fmaf(f, x.x, acc.x);
                acc.y = fmaf(f, x.y, acc.y);
                acc.z = fmaf(f, x.z, acc.z);
                acc.w = fmaf(f, x.w, acc.w);
            }
            if (whole) {
                const int row = row0 + r, tk = row / p.G, hq = h * p.G + row % p.G;
                const float il = sum == 0.f ? 0.f : 1.f / sum;
                const float y[4] = {acc.x * il, acc.y * il, acc.z * il, acc.w * il};
                const int64_t at = b * p.os[0] + tk * p.os[1] + hq * p.os[2];
#pragma unroll
                for (int k = 0; k < 4; ++k) st_out(p.out, at + (d + k) * p.os[3], p.o_dt, y[k]);
                if (d == 0 && p.lse) p.lse[b * p.ls[0] + tk * p.ls[1] + hq * p.ls[2]] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
            } else {
                *reinterpret_cast<float4*>(ws + 2 * S::ROWS + r * D + d) = acc;
                if (d == 0) {
                    ws[r] = top;
                    ws[S::ROWS + r] = sum;
                }
            }
        }
        __syncthreads();   // the ring and the fragments are written again
    }
    flag_err(p.dev_err, bits);
}

// Adds the parts of a pair that begins in one block and ends in another.  A block has
// 8 rows, a warp each, or, where pairs are spread over many blocks, 64 dimensions of one
// row, its half-warps taking parts in turn.
constexpr int kJoinWarps = 8;
constexpr int kSlice = 64;

template <int D, bool F8, int NR>
__global__ void __launch_bounds__(kJoinWarps * 32) attn_join(const __grid_constant__ AttnParams p, int row_blocks, int by_row) {
    using S = Shape<D, F8, NR>;
    constexpr int GROUPS = kJoinWarps * 2;
    __shared__ float top_s[kJoinWarps], sum_s[kJoinWarps], f_s[kMaxBlocks];
    __shared__ float4 o_s[GROUPS][kSlice / 4];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    stream_order();
    const int4 split = reinterpret_cast<const int4*>(p.ws)[blockIdx.x];
    const int b = split.x, pair = split.y, g1 = split.z, g0 = split.w, h = pair / row_blocks, row0 = pair % row_blocks * S::ROWS;
    if (b < 0) return;
    const float* const parts_at = p.ws + 4 * kMaxBlocks;
    auto part_of = [&](int i) { return parts_at + (2 * static_cast<int64_t>(i) + (i == g0)) * S::PART; };
    const int r = by_row ? blockIdx.y : blockIdx.y * 8 + warp, row = row0 + r;
    if (row >= p.G * p.T) return;   // a block's, or a warp's
    const int tk = row / p.G, hq = h * p.G + row % p.G;
    const int64_t at = b * p.os[0] + tk * p.os[1] + hq * p.os[2];
    float* const lse = p.lse ? p.lse + b * p.ls[0] + tk * p.ls[1] + hq * p.ls[2] : nullptr;
    if (by_row) {
        float m = kNone, l = 0.f;
        for (int i = g0 + tid; i <= g1; i += kJoinWarps * 32) m = fmaxf(m, part_of(i)[r]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        if (lane == 0) top_s[warp] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, top_s[w]);
        for (int i = g0 + tid; i <= g1; i += kJoinWarps * 32) {
            const float* part = part_of(i);
            const float f = exp2_f(part[r] - m);
            f_s[i - g0] = f;
            l = fmaf(f, part[S::ROWS + r], l);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
        if (lane == 0) sum_s[warp] = l;
        __syncthreads();
        l = 0.f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) l += sum_s[w];
        const int grp = tid / (kSlice / 4), q = tid % (kSlice / 4), d = blockIdx.z * kSlice + q * 4;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int i = g0 + grp; i <= g1; i += GROUPS) {
            const float4 x = *reinterpret_cast<const float4*>(part_of(i) + 2 * S::ROWS + r * D + d);
            const float f = f_s[i - g0];
            acc.x = fmaf(f, x.x, acc.x);
            acc.y = fmaf(f, x.y, acc.y);
            acc.z = fmaf(f, x.z, acc.z);
            acc.w = fmaf(f, x.w, acc.w);
        }
        o_s[grp][q] = acc;
        __syncthreads();
        if (tid < kSlice) {
            float y = 0.f;
#pragma unroll
            for (int w = 0; w < GROUPS; ++w) y += reinterpret_cast<const float*>(o_s[w])[tid];
            st_out(p.out, at + (blockIdx.z * kSlice + tid) * p.os[3], p.o_dt, y * (l == 0.f ? 0.f : 1.f / l));
        }
        if (tid == 0 && blockIdx.z == 0 && lse) *lse = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        return;
    }
    constexpr int PER = D / 32;   // dimensions of a lane
    float m = kNone, l = 0.f, o[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) o[k] = 0.f;
#pragma unroll 2
    for (int i = g0; i <= g1; ++i) {
        const float* part = part_of(i);
        const float pm = part[r], pl = part[S::ROWS + r];
        float x[PER];
#pragma unroll
        for (int k = 0; k < PER; ++k) x[k] = part[2 * S::ROWS + r * D + lane + k * 32];
        const float top = fmaxf(m, pm), a = exp2_f(m - top), c = exp2_f(pm - top);
        l = fmaf(l, a, pl * c);
#pragma unroll
        for (int k = 0; k < PER; ++k) o[k] = fmaf(o[k], a, x[k] * c);
        m = top;
    }
    const float il = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int k = 0; k < PER; ++k) st_out(p.out, at + (lane + k * 32) * p.os[3], p.o_dt, o[k] * il);
    if (lane == 0 && lse) *lse = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// Tiles of 8 rows that a pair has: as many as its rows need, while registers hold their outputs
constexpr int most_rows(int D) { return D <= 128 ? 4 : 2; }

int row_tiles(int T, int G, int D) {
    const int need = (T * G + 7) / 8;
    return need <= 1 ? 1 : need <= 2 || most_rows(D) == 2 ? 2 : 4;
}

template <int D, bool F8, int NR>
lar_status launch(const AttnParams& p, cudaStream_t stream) {
    using S = Shape<D, F8, NR>;
    const int row_blocks = (p.G * p.T + S::ROWS - 1) / S::ROWS;
    auto kern = attn_kernel<D, F8, NR>;
    int sms = 0;
    const int occ = cached_occupancy(reinterpret_cast<const void*>(kern), kThreads, S::SMEM, S::SMEM, &sms);
    if (occ < 1) return LAR_ERR_LAUNCH;
    const int64_t pairs = static_cast<int64_t>(p.B) * p.c.H * row_blocks;
    if (pairs > (int64_t{1} << 31) - 1) return LAR_ERR_SHAPE;
    // no more blocks than the longest sequences that the table admits could fill
    const int64_t cap = static_cast<int64_t>(p.c.M) * p.c.page;
    const int64_t most = (pairs * ((cap + S::WT - 1) / S::WT + 1 + kStart) + kWarps - 1) / kWarps;
    int64_t blocks = static_cast<int64_t>(sms) * occ;
    if (blocks > kMaxBlocks) blocks = kMaxBlocks;
    if (blocks > most) blocks = most;
    const int by_row = blocks >= kJoinWarps * pairs;
    const lar_status st = launch_ordered(kern, dim3(static_cast<unsigned>(blocks)), kThreads, S::SMEM, 1, stream, p, row_blocks, by_row);
    if (st != LAR_OK) return st;
    return launch_ordered(attn_join<D, F8, NR>, dim3(static_cast<unsigned>(by_row ? pairs : blocks), by_row ? S::ROWS : NR, by_row ? D / kSlice : 1), kJoinWarps * 32, 0, 1,
                          stream, p, row_blocks, by_row);
}

template <int D, bool F8>
lar_status launch_rows(const AttnParams& p, cudaStream_t stream) {
    const int nr = row_tiles(p.T, p.G, D);
    if (nr == 1) return launch<D, F8, 1>(p, stream);
    if constexpr (most_rows(D) == 4) {
        if (nr == 4) return launch<D, F8, 4>(p, stream);
    }
    return launch<D, F8, 2>(p, stream);
}

template <int D>
lar_status launch_d(const AttnParams& p, cudaStream_t stream) {
    return p.c.e4m3 ? launch_rows<D, true>(p, stream) : launch_rows<D, false>(p, stream);
}

}  // namespace

int64_t attn_workspace_floats(int T, int G, int D) {
    return int64_t{4} * kMaxBlocks + int64_t{2} * kMaxBlocks * 8 * row_tiles(T, G, D) * (D + 2);
}

lar_status launch_attn(const AttnParams& p, void* stream) {
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return p.c.D == 64 ? launch_d<64>(p, s) : p.c.D == 128 ? launch_d<128>(p, s) : launch_d<256>(p, s);
}

}  // namespace lar

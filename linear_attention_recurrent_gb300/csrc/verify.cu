// verify.cu -- verification of drafted tokens against the target model's
// probabilities (spec_verify).  Sequence b drafted tokens d_0 .. d_{k-1} from
// q_0 .. q_{k-1}; the target gives p_0 .. p_k.  d_t is accepted if all before it
// are and u_t q_t(d_t) < p_t(d_t).  With n accepted, the next token is drawn from
// w = max(p_n - q_n, 0) (n < k) or w = p_k, by inversion: the first index whose
// running sum of w exceeds v times the whole sum.
//
// Only the row of the first rejection is read, in full: it bounds the call.  The
// vocabulary is split over the blocks of a cluster, every warp owning a
// contiguous stretch; after the sums are joined through distributed shared memory
// the one warp whose stretch holds the threshold reads its stretch again.
//
// A chosen index has to be the one that exact sums give, and a flat row has
// neighbours 1e-5 apart of which a sum in 32 bits gets the last digits wrong.
// So weights and sums are kept as unevaluated sums of two floats (the rounding
// error of p - q is itself a float), good to about 2^-48.  Doubles would do as well,
// but fp64 additions are so slow here that joining the lanes' sums in them took most
// of the call: 15.6 us for one sequence and 51 us for 64 x 131072 fp32, against 7.0
// and 18 us so.  Of the 18 us the rows' bytes are 8.5 (10 if every sequence read both; one
// whose drafts all stand reads the target's alone); the rest is the way from the drafts
// to the row (three loads one after another) and from the sums to the token.
#include "layer_common.cuh"

namespace lar {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kStep = 256;      // tokens of a warp's step

// (hi, lo) + x, the error of the sum kept: two-sum (Knuth)
__device__ __forceinline__ void add_exact(float& hi, float& lo, float x) {
    const float s = hi + x;
    const float t = s - hi;
    lo += (hi - (s - t)) + (x - t);
    hi = s;
}

// hi + lo, |lo| at most half a unit in the last place of hi
struct Sum {
    float hi, lo;
};

__device__ __forceinline__ Sum renormal(float hi, float lo) {
    const float s = hi + lo;
    return {s, lo - (s - hi)};
}

__device__ __forceinline__ Sum plus(Sum a, Sum b) {
    float hi = a.hi, lo = a.lo + b.lo;
    add_exact(hi, lo, b.hi);
    return renormal(hi, lo);
}

__device__ __forceinline__ bool below(Sum a, Sum b) { return a.hi < b.hi || (a.hi == b.hi && a.lo < b.lo); }
__device__ __forceinline__ bool same(Sum a, Sum b) { return a.hi == b.hi && a.lo == b.lo; }
__device__ __forceinline__ Sum least(Sum a, Sum b) { return below(b, a) ? b : a; }

__device__ __forceinline__ Sum shfl(Sum a, int lane) {
    return {__shfl_sync(0xffffffffu, a.hi, lane), __shfl_sync(0xffffffffu, a.lo, lane)};
}

__device__ __forceinline__ Sum warp_sum(Sum a) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        a = plus(a, {__shfl_xor_sync(0xffffffffu, a.hi, off), __shfl_xor_sync(0xffffffffu, a.lo, off)});
    return a;
}

// sums of lanes 0 .. this one
__device__ __forceinline__ Sum warp_scan(Sum a, int lane) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const Sum y = {__shfl_up_sync(0xffffffffu, a.hi, off), __shfl_up_sync(0xffffffffu, a.lo, off)};
        if (lane >= off) a = plus(y, a);
    }
    return a;
}

// The weight of a token with target probability a and draft probability b, as hi +
// lo; 0 unless positive and finite.  The error of a float difference is a float.
__device__ __forceinline__ void weight_of(float a, float b, float& hi, float& lo) {
    hi = a - b;
    const float t = hi - a;
    lo = (a - (hi - t)) + (-b - t);
    if (!(hi > 0.f && hi < INFINITY)) hi = lo = 0.f;
}

// The same where nothing is infinite: fmaxf takes NaN and negative numbers to 0.
__device__ __forceinline__ void weight_finite(float a, float b, float& hi, float& lo) {
    const float d = a - b, t = d - a;
    lo = (a - (d - t)) + (-b - t);
    hi = fmaxf(d, 0.f);
    lo = d > 0.f ? lo : 0.f;
}

struct Row {
    const void *p, *q;      // q NULL: nothing to subtract
    int64_t ps, qs;         // element strides
    int p_dt, q_dt;
    int64_t hot;            // one-hot q: the drafted token, else -1
    int64_t V;
    bool vec;               // 16-byte loads fit both

    __device__ __forceinline__ void weight(int64_t i, float& hi, float& lo) const {
        const float a = i == hot ? 0.f : ld_in(p, i * ps, p_dt);
        weight_of(a, q ? ld_in(q, i * qs, q_dt) : 0.f, hi, lo);
    }

    // tokens [i, i + 8), in order; past the end they weigh nothing
    __device__ __forceinline__ void weights8(int64_t i, float* hi, float* lo) const {
        if (vec && i + 8 <= V) {
            float a[8], b[8];
            ld8<true>(p, i, p_dt, a);
#pragma unroll
            for (int k = 0; k < 8; ++k) b[k] = 0.f;
            if (q) ld8<true>(q, i, q_dt, b);
#pragma unroll
            for (int k = 0; k < 8; ++k) weight_of(i + k == hot ? 0.f : a[k], b[k], hi[k], lo[k]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                hi[k] = lo[k] = 0.f;
                if (i + k < V) weight(i + k, hi[k], lo[k]);
            }
        }
    }
};

// Adds the weights of whole steps [s0, s1) of a row that 16-byte loads fit.  A sum
// that is not finite says that some weight was not: the caller adds them again, with
// each looked at.
template <typename P, typename Q, bool HAS_Q>
__device__ __forceinline__ void add_steps(const Row& row, int64_t s0, int64_t s1, int lane, float& hi, float& lo) {
    constexpr int U = 2;
    for (int64_t s = s0; s < s1; s += U) {
        Eight<P> a[U];
        Eight<Q> b[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {   // the last one may ask for a step again, to no effect
            const int64_t i = min(s + u, s1 - 1) * kStep + lane * 8;
            a[u].load(row.p, i);
            if (HAS_Q) b[u].load(row.q, i);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s + u >= s1) break;
            const int64_t i = (s + u) * kStep + lane * 8;
            float fa[8], fb[8];
            a[u].widen(fa);
            if (HAS_Q) b[u].widen(fb);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float w, e;
                if (HAS_Q) {
                    weight_finite(fa[k], fb[k], w, e);
                    add_exact(hi, lo, w);
                    lo += e;
                } else {
                    w = fmaxf(fa[k], 0.f);
                    add_exact(hi, lo, i + k == row.hot ? 0.f : w);
                }
            }
        }
    }
}

__device__ __forceinline__ void put_token(const VerifyParams& p, int64_t b, int t, int64_t v) {
    const int64_t o = b * p.os[0] + t * p.os[1];
    if (p.out_dt == LAR_I32) static_cast<int32_t*>(p.out)[o] = static_cast<int32_t>(v);
    else static_cast<int64_t*>(p.out)[o] = v;
}

__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyParams p) {
    __shared__ Sum warp_tot[kWarps];
    __shared__ Sum blocks[2][kMaxCluster];   // every block's sum, in both passes
    __shared__ Sum before_s, after_s, total_s, start_s;
    __shared__ int owner_s;
    __shared__ int found[2];
    __shared__ int64_t last_seen;
    const unsigned rank = cluster_rank(), size = cluster_size();
    const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    cluster_arrive();   // this block has started: its memory may be written from now on
    stream_order();
    int32_t bits = 0;

    // accepted drafts, by every warp for itself: lane t looks at draft t
    int64_t k = p.T - 1;
    if (p.nd) {
        const int64_t v = ld_idx(p.nd, b * p.nd_s, p.nd_dt);
        if (v < 0 || v > k) bits |= LAR_DEVERR_DRAFT;
        else k = v;
        if (v < 0) k = 0;
    }
    int64_t tok = -1;
    bool good = false;
    if (lane < k) {
        tok = ld_idx(p.tok, b * p.tk_s[0] + lane * p.tk_s[1], p.tok_dt);
        if (tok < 0 || tok >= p.V) {
            bits |= LAR_DEVERR_DRAFT;
        } else {
            const float pt = ld_in(p.p, b * p.ps[0] + lane * p.ps[1] + tok * p.ps[2], p.p_dt);
            const float qt = p.q ? ld_in(p.q, b * p.qs[0] + lane * p.qs[1] + tok * p.qs[2], p.q_dt) : 1.f;
            // u q < p for the product itself: where it rounds to p, its error decides, which
            // is an fp32 number once numbers near the least ones are scaled up
            const float u = __ldg(p.ua + b * p.ua_s[0] + lane * p.ua_s[1]), uq = u * qt;
            const float up = pt < 0x1p-60f ? 0x1p60f : 1.f;
            good = uq < pt || (uq == pt && fmaf(u, qt * up, -pt * up) < 0.f);
        }
    }
    const unsigned bad = ~__ballot_sync(0xffffffffu, good);
    const int n = min(static_cast<int>(k), __ffs(bad) - 1);   // lane 31 never holds a draft: bad is not 0
    const int64_t rejected = __shfl_sync(0xffffffffu, tok, n);

    Row row;
    row.p = static_cast<const char*>(p.p) + (b * p.ps[0] + n * p.ps[1]) * (p.p_dt == LAR_F32 ? 4 : 2);
    row.ps = p.ps[2];
    row.p_dt = p.p_dt;
    row.q = nullptr;
    row.qs = 0;
    row.q_dt = p.q_dt;
    row.hot = -1;
    row.V = p.V;
    if (n < k) {
        if (p.q) {
            row.q = static_cast<const char*>(p.q) + (b * p.qs[0] + n * p.qs[1]) * (p.q_dt == LAR_F32 ? 4 : 2);
            row.qs = p.qs[2];
        } else {
            row.hot = rejected;
        }
    }

    row.vec = row.ps == 1 && reinterpret_cast<uintptr_t>(row.p) % 16 == 0 &&
              (!row.q || (row.qs == 1 && reinterpret_cast<uintptr_t>(row.q) % 16 == 0));

    // this warp's stretch of the vocabulary, in steps of 256 tokens, 8 a lane
    const int64_t steps = (p.V + kStep - 1) / kStep;
    const int64_t w_all = static_cast<int64_t>(size) * kWarps, w_me = static_cast<int64_t>(rank) * kWarps + warp;
    const int64_t s0 = steps * w_me / w_all, s1 = steps * (w_me + 1) / w_all;

    Sum total = {0.f, 0.f};
    for (int pass = 0; pass < 2; ++pass) {
        float hi = 0.f, lo = 0.f;
        int64_t done = s0;
        if (row.vec) {
            done = max(s0, min(s1, p.V / kStep));   // whole steps
            const bool pb = row.p_dt == LAR_BF16, qb = row.q_dt == LAR_BF16;
            using F = float;
            using H = unsigned short;
            if (!row.q) pb ? add_steps<H, H, false>(row, s0, done, lane, hi, lo) : add_steps<F, F, false>(row, s0, done, lane, hi, lo);
            else if (qb) pb ? add_steps<H, H, true>(row, s0, done, lane, hi, lo) : add_steps<F, H, true>(row, s0, done, lane, hi, lo);
            else pb ? add_steps<H, F, true>(row, s0, done, lane, hi, lo) : add_steps<F, F, true>(row, s0, done, lane, hi, lo);
            if (__any_sync(0xffffffffu, !(hi < INFINITY && lo < INFINITY))) {
                done = s0;
                hi = lo = 0.f;
            }
        }
        for (int64_t s = done; s < s1; ++s) {   // neighbours on neighbouring lanes: the order is free here
            float a[8], e[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                a[k] = e[k] = 0.f;
                const int64_t i = s * kStep + k * 32 + lane;
                if (i < p.V) row.weight(i, a[k], e[k]);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                add_exact(hi, lo, a[k]);
                lo += e[k];
            }
        }
        const Sum mine = warp_sum(renormal(hi, lo));
        if (lane == 0) warp_tot[warp] = mine;
        __syncthreads();
        if (pass == 0) cluster_wait();   // all blocks have
        if (warp == 0) {
            // to every block of the cluster, so that none reads another's memory later
            const Sum own = warp_sum(lane < kWarps ? warp_tot[lane] : Sum{0.f, 0.f});
            if (lane < size) {
                st_peer_f32(&blocks[pass][rank].hi, lane, own.hi);
                st_peer_f32(&blocks[pass][rank].lo, lane, own.lo);
            }
        }
        cluster_sync();
        if (warp == 0) {
            const Sum all = lane < size ? blocks[pass][lane] : Sum{0.f, 0.f};
            Sum run = {0.f, 0.f};   // one after another: alike in every block, and never falling
            for (unsigned r = 0; r < size; ++r) {
                if (r == rank && lane == 0) before_s = run;
                run = plus(run, shfl(all, r));
                if (r == rank && lane == 0) after_s = run;
            }
            if (lane == 0) total_s = run;
        }
        __syncthreads();
        total = total_s;
        if (total.hi > 0.f || (row.q == nullptr && row.hot < 0)) break;
        // the residual is empty: draw from the target itself
        row.q = nullptr;
        row.hot = -1;
        __syncthreads();   // total_s is written again
    }
    if (rank == 0 && warp == 0) {
        if (lane < p.T && lane != n) put_token(p, b, lane, lane < n ? tok : -1);
        if (lane == 0) {
            if (p.acc_dt == LAR_I32) static_cast<int32_t*>(p.acc)[b * p.acc_s] = n + 1;
            else static_cast<int64_t*>(p.acc)[b * p.acc_s] = n + 1;
        }
        if (!(total.hi > 0.f)) bits |= LAR_DEVERR_PROBS;
        bits = static_cast<int32_t>(__reduce_or_sync(0xffffffffu, static_cast<unsigned>(bits)));
        if (lane == 0) flag_err(p.dev_err, bits);
    }

    if (!(total.hi > 0.f)) {   // no weight anywhere
        if (rank == 0 && tid == 0) put_token(p, b, n, -1);
        return;
    }
    // A number outside [0, 1) draws the first or the last token with any weight.
    const float us = __ldg(p.us + b * p.us_s), up = us * total.hi;
    const Sum zero = {0.f, 0.f}, thr = us >= 0.f ? renormal(up, fmaf(us, total.hi, -up) + us * total.lo) : zero;
    // Warp w's stretch of the whole sum is [lo, hi).  `after` is where the next block's
    // begins; the last warp with any weight ends there, so that the stretches of all
    // warps cover [0, total) once, whatever the sums round to.
    if (warp == 0) {
        const Sum own = lane < kWarps ? warp_tot[lane] : zero;
        const unsigned some = __ballot_sync(0xffffffffu, own.hi > 0.f);
        Sum run = before_s, lo = run, hi = run;
        for (int w = 0; w < kWarps; ++w) {
            if (lane == w) lo = run;
            run = least(plus(run, shfl(own, w)), after_s);
            if (lane == w) hi = some >> w == 1u ? after_s : run;
        }
        const bool mine = own.hi > 0.f && below(lo, hi) &&
                          ((!below(thr, lo) && below(thr, hi)) || (!below(thr, total) && same(hi, total)));
        const unsigned who = __ballot_sync(0xffffffffu, mine);
        if (lane == 0) owner_s = who ? __ffs(who) - 1 : -1;
        if (who && lane == __ffs(who) - 1) start_s = lo;
    }
    __syncthreads();
    const int owner = owner_s;
    if (owner < 0) return;   // another block's: one alone finds an owner
    Sum start = start_s;

    // The block goes through the owner's stretch, 8 neighbours a thread.
    const int64_t o_me = static_cast<int64_t>(rank) * kWarps + owner;
    const int64_t first = steps * o_me / w_all * kStep, end = min(steps * (o_me + 1) / w_all * kStep, p.V);
    for (int64_t base = first; base < end; base += kThreads * 8) {
        const int64_t i = base + tid * 8;
        float a[8], e[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) a[k] = e[k] = 0.f;
        if (i < end) row.weights8(i, a, e);
        float hi = 0.f, er = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            add_exact(hi, er, a[k]);
            er += e[k];
        }
        const Sum own = renormal(hi, er), incl = warp_scan(own, lane);
        __syncthreads();   // warp_tot and found are read no more
        if (lane == 31) warp_tot[warp] = incl;
        if (tid == 0) found[0] = found[1] = -1;
        __syncthreads();
        Sum run = start, block = start;   // up to this thread's tokens, and past the block's
        for (int w = 0; w < kWarps; ++w) {
            if (w == warp) run = block;
            block = plus(block, warp_tot[w]);
        }
        const Sum left = {__shfl_up_sync(0xffffffffu, incl.hi, 1), __shfl_up_sync(0xffffffffu, incl.lo, 1)};
        const Sum upto = plus(run, incl);
        if (lane > 0) run = plus(run, left);
        // the first thread that ends above the threshold holds the token
        if (own.hi > 0.f && below(thr, upto))
            atomicMin(reinterpret_cast<unsigned*>(&found[0]), static_cast<unsigned>(tid));
        if (own.hi > 0.f) atomicMax(&found[1], tid);
        __syncthreads();
        if (tid == found[0] || tid == found[1]) {
            int64_t chosen = -1, last = -1;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (!(a[k] > 0.f)) continue;
                run = plus(run, {a[k], e[k]});
                last = i + k;
                if (chosen < 0 && below(thr, run)) chosen = i + k;
            }
            if (tid == found[0]) put_token(p, b, n, chosen >= 0 ? chosen : last);
            else last_seen = last;
        }
        if (found[0] >= 0) return;
        start = block;
    }
    // rounding left none above: the last token of the stretch with any weight
    __syncthreads();
    if (tid == 0) put_token(p, b, n, last_seen);
}

}  // namespace

lar_status launch_verify(const VerifyParams& p, void* stream) {
    // a block a few thousand tokens, at most 8 (the portable cluster)
    int size = 1;
    while (size < kMaxCluster && static_cast<int64_t>(size) * 2048 < p.V) size *= 2;
    return launch_ordered(verify_kernel, dim3(size, p.B), kThreads, 0, size, static_cast<cudaStream_t>(stream), p);
}

}  // namespace lar

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
// So a weight is kept as the unevaluated sum of two floats (the rounding error
// of p - q is itself a float), a lane adds pairs, and lanes, warps and blocks
// are joined in 64 bits.
#include "layer_common.cuh"

namespace lar {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;

__device__ __forceinline__ double ld_peer_f64(const double* p, unsigned rank) {
    double v;
    asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(peer_addr(p, rank)));
    return v;
}

// (hi, lo) + x, the error of the sum kept: two-sum (Knuth)
__device__ __forceinline__ void add_exact(float& hi, float& lo, float x) {
    const float s = hi + x;
    const float t = s - hi;
    lo += (hi - (s - t)) + (x - t);
    hi = s;
}

struct Row {
    const void *p, *q;      // q NULL: nothing to subtract
    int64_t ps, qs;         // element strides
    int p_dt, q_dt;
    int64_t hot;            // one-hot q: the drafted token, else -1

    // the weight of token i as hi + lo; 0 unless positive and finite
    __device__ __forceinline__ void weight(int64_t i, float& hi, float& lo) const {
        const float a = ld_in(p, i * ps, p_dt);
        hi = a;
        lo = 0.f;
        if (q) {
            const float b = ld_in(q, i * qs, q_dt);
            hi = a - b;
            const float t = hi - a;
            lo = (a - (hi - t)) + (-b - t);
        } else if (i == hot) {
            hi = 0.f;
        }
        if (!(hi > 0.f && hi < INFINITY)) hi = lo = 0.f;
    }
};

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyParams p) {
    __shared__ double warp_tot[kWarps];
    __shared__ double block_tot;
    const unsigned rank = cluster_rank(), size = cluster_size();
    const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
            // the product of two floats is exact in 64 bits
            good = static_cast<double>(p.ua[b * p.ua_s[0] + lane * p.ua_s[1]]) * static_cast<double>(qt) <
                   static_cast<double>(pt);
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
    if (n < k) {
        if (p.q) {
            row.q = static_cast<const char*>(p.q) + (b * p.qs[0] + n * p.qs[1]) * (p.q_dt == LAR_F32 ? 4 : 2);
            row.qs = p.qs[2];
        } else {
            row.hot = rejected;
        }
    }

    // this warp's stretch of the vocabulary, in steps of 32 tokens
    const int64_t steps = (p.V + 31) / 32;
    const int64_t w_all = static_cast<int64_t>(size) * kWarps, w_me = static_cast<int64_t>(rank) * kWarps + warp;
    const int64_t s0 = steps * w_me / w_all, s1 = steps * (w_me + 1) / w_all;

    double total = 0., before = 0., after = 0., mine = 0.;
    for (int pass = 0; pass < 2; ++pass) {
        float hi = 0.f, lo = 0.f;
        for (int64_t s = s0; s < s1; ++s) {
            const int64_t i = s * 32 + lane;
            if (i >= p.V) continue;
            float a, e;
            row.weight(i, a, e);
            add_exact(hi, lo, a);
            lo += e;
        }
        mine = warp_sum(static_cast<double>(hi) + static_cast<double>(lo));
        if (lane == 0) warp_tot[warp] = mine;
        __syncthreads();
        if (tid == 0) {
            double t = 0.;
            for (int w = 0; w < kWarps; ++w) t += warp_tot[w];
            block_tot = t;
        }
        cluster_sync();
        total = before = 0.;
        for (unsigned r = 0; r < size; ++r) {
            if (r == rank) before = total;
            total += ld_peer_f64(&block_tot, r);
            if (r == rank) after = total;
        }
        cluster_sync();   // every block has read the sums: they may be written again
        if (total > 0. || (row.q == nullptr && row.hot < 0)) break;
        // the residual is empty: draw from the target itself
        row.q = nullptr;
        row.hot = -1;
    }
    // This warp's stretch of the whole sum, [lo_sum, hi_sum).  `after` is where the
    // next block's begins; the last warp with any weight ends there, so that the
    // stretches of all warps cover [0, total) once, whatever the sums round to.
    double lo_sum = before, hi_sum;
    int last_warp = -1;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) lo_sum += warp_tot[w];
        if (warp_tot[w] > 0.) last_warp = w;
    }
    hi_sum = warp == last_warp ? after : fmin(lo_sum + mine, after);
    lo_sum = fmin(lo_sum, after);

    if (rank == 0 && warp == 0) {
        if (lane < p.T && lane != n) {
            const int64_t o = b * p.os[0] + lane * p.os[1], v = lane < n ? tok : -1;
            if (p.out_dt == LAR_I32) static_cast<int32_t*>(p.out)[o] = static_cast<int32_t>(v);
            else static_cast<int64_t*>(p.out)[o] = v;
        }
        if (lane == 0) {
            if (p.acc_dt == LAR_I32) static_cast<int32_t*>(p.acc)[b * p.acc_s] = n + 1;
            else static_cast<int64_t*>(p.acc)[b * p.acc_s] = n + 1;
        }
        if (!(total > 0.)) bits |= LAR_DEVERR_PROBS;
        bits = static_cast<int32_t>(__reduce_or_sync(0xffffffffu, static_cast<unsigned>(bits)));
        if (lane == 0) flag_err(p.dev_err, bits);
    }

    // The warp whose stretch holds the threshold finds the token.  A number outside
    // [0, 1) draws the first or the last token with any weight.
    double thr = static_cast<double>(p.us[b * p.us_s]) * total;
    if (!(thr >= 0.)) thr = 0.;
    int64_t chosen = -1;
    const bool here = total > 0. ? mine > 0. && lo_sum < hi_sum &&
                                       ((lo_sum <= thr && thr < hi_sum) || (thr >= total && hi_sum == total))
                                 : rank == 0 && warp == 0;   // no weight anywhere: token -1
    if (here && total > 0.) {
        double run = lo_sum;
        int64_t last = -1;
        for (int64_t s = s0; s < s1 && chosen < 0; ++s) {
            const int64_t i = s * 32 + lane;
            float a = 0.f, e = 0.f;
            if (i < p.V) row.weight(i, a, e);
            const double w = static_cast<double>(a) + static_cast<double>(e);
            double incl = w;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += y;
            }
            const unsigned over = __ballot_sync(0xffffffffu, w > 0. && run + incl > thr);
            const unsigned any = __ballot_sync(0xffffffffu, w > 0.);
            if (over) chosen = s * 32 + __ffs(over) - 1;
            if (any) last = s * 32 + 31 - __clz(any);
            run += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (chosen < 0) chosen = last;
    }
    if (here && lane == 0) {
        const int64_t o = b * p.os[0] + n * p.os[1];
        if (p.out_dt == LAR_I32) static_cast<int32_t*>(p.out)[o] = static_cast<int32_t>(chosen);
        else static_cast<int64_t*>(p.out)[o] = chosen;
    }
}

}  // namespace

lar_status launch_verify(const VerifyParams& p, void* stream) {
    // a block a few thousand tokens, at most 8 (the portable cluster)
    int size = 1;
    while (size < kMaxCluster && static_cast<int64_t>(size) * 2048 < p.V) size *= 2;
    return launch_ordered(verify_kernel, dim3(size, p.B), kThreads, 0, size, static_cast<cudaStream_t>(stream), p);
}

}  // namespace lar

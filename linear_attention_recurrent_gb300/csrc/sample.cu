// sample.cu -- the draw of a token from a row of logits (sample_tokens): temperature,
// top-k, top-p, min-p and the inversion of the running sum by a given random number.
//
// Order and weights.  Logits are ordered by the bits of their fp32 value (a key that rises
// with it), equal ones by index; each filter keeps a prefix of that order.  A weight
// exp((x - max) / temperature) is a whole number of 2^-39: a token has to be the one that
// exact sums give, and whole numbers add up exactly in any order, at the rate of 32-bit
// adds, where fp64 is slow on this part.  Its argument is kept in two floats, 2^n comes
// from a table of 32 steps, and the rest, at most 1/64, from a polynomial: good to 2^-30 of
// the weight, or 2^-40 of the greatest.
//
// Thresholds.  The key at which a prefix has k tokens, or p of the weight, is found 11 bits
// at a time: sums a bin in shared memory, added over the blocks of a cluster.  Ties at the
// threshold are kept from the lowest index on.
//
// A row is a cluster's, every warp owning a contiguous stretch of the vocabulary.
#include "layer_common.cuh"
#include "serve_params.h"

namespace lar {

namespace {

using u64 = unsigned long long;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kStep = 256;       // tokens of a warp's step, 8 a lane
constexpr int kBits = 11;        // of a key, looked at in one go
constexpr int kBins = 1 << kBits;
constexpr u64 kOne = 1ull << 39;  // weight of the greatest logit

// 2^(39 + j / 32), to the nearest whole number
__constant__ u64 kPow[32] = {
    549755813888ull, 561793898668ull, 574095583180ull, 586666639507ull, 599512966123ull, 612640590662ull,
    626055672747ull, 639764506879ull, 653773525390ull, 668089301461ull, 682718552210ull, 697668141836ull,
    712945084849ull, 728556549354ull, 744509860419ull, 760812503507ull, 777472127994ull, 794496550755ull,
    811893759832ull, 829671918182ull, 847839367509ull, 866404632174ull, 885376423200ull, 904763642353ull,
    924575386327ull, 944820951003ull, 965509835819ull, 986651748221ull, 1008256608221ull, 1030334553053ull,
    1052895941925ull, 1075951360882ull};

// A logit as it is ordered: NaN is -infinity, and -0 is 0.
__device__ __forceinline__ float clean(float x) { return x == x ? x + 0.f : -INFINITY; }

__device__ __forceinline__ unsigned key_of(float x) {
    const unsigned b = __float_as_uint(x);
    return b ^ (static_cast<unsigned>(static_cast<int>(b) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float of_key(unsigned k) {
    return __uint_as_float(k ^ (static_cast<unsigned>(~static_cast<int>(k) >> 31) | 0x80000000u));
}

constexpr unsigned kLeast = 0x007fffffu;   // key of -infinity

struct Scale {
    float half_max;     // max / 2: differences of halves do not overflow
    float hi, lo;       // 2 log2(e) / temperature
    bool infinite;      // max is +infinity

    // (x - max) log2(e) / temperature as y + e
    __device__ __forceinline__ void exponent(float x, float& y, float& e) const {
        const float a = 0.5f * x, d = a - half_max, t = d - a;
        const float de = (a - (d - t)) + (-half_max - t);
        y = d * hi;
        e = fmaf(d, hi, -y) + fmaf(d, lo, de * hi);
    }

    __device__ __forceinline__ u64 weight(float x, const u64* pow) const {
        if (0.5f * x == half_max) return kOne;
        if (infinite) return 0;
        float y, e;
        exponent(x, y, e);
        if (!(y >= -41.f)) return 0;
        const float r32 = rintf(y * 32.f);
        const int j = static_cast<int>(r32), down = -(j >> 5);
        const float f = fmaf(r32, -1.f / 32, y) + e;
        // 2^f - 1 by ln 2, its powers over the factorials
        const float g = f * fmaf(f, fmaf(f, fmaf(f, 9.618129e-3f, 5.550411e-2f), 0.24022651f), 0.69314718f);
        const u64 t = pow[j & 31];
        const u64 w = t + static_cast<u64>(static_cast<long long>(__float2int_rn(g * (static_cast<float>(t) * 0.125f))) << 3);
        return down > 0 ? (w + (1ull << (down - 1))) >> down : w;
    }
};

struct Row {
    const char* x;      // element 0
    int64_t xs;         // stride
    int dt;
    int off;            // elements between the last 16-byte border and element 0
    int V;

    __device__ __forceinline__ float at(int i) const { return clean(ld_in(x, i * xs, dt)); }

    // f(i, x) for elements [j - off, j - off + 8), j a multiple of 8, if they are there
    template <typename F>
    __device__ __forceinline__ void eight(int j, F f) const {
        const int i = j - off;
        if (xs == 1 && i >= 0 && i + 8 <= V) {
            float a[8];
            ld8<true>(x, i, dt, a);
#pragma unroll
            for (int k = 0; k < 8; ++k) f(i + k, clean(a[k]));
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (i + k >= 0 && i + k < V) f(i + k, at(i + k));
        }
    }
};

__device__ __forceinline__ void st_peer_u64(u64* p, unsigned rank, u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(peer_addr(p, rank)), "l"(v) : "memory");
}

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

__device__ __forceinline__ u64 warp_max(u64 v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const u64 o = __shfl_xor_sync(0xffffffffu, v, off);
        v = o > v ? o : v;
    }
    return v;
}

// sum of lanes 0 .. this one
__device__ __forceinline__ u64 warp_scan(u64 v, int lane) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const u64 o = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += o;
    }
    return v;
}

struct Shared {
    u64 pow[32];
    u64 warp[kWarps];
    u64 peer[2][2][kMaxCluster];   // exchanges in turn; two values each
    u64 found[4];
    unsigned lo[kBins], hi[kBins];
    float scale_hi, scale_lo;
};

struct Block {
    Shared& s;
    unsigned rank, size;
    int tid, lane, warp;
    int turn = 0;

    // Sum (or greatest) of every thread's v over the cluster, and of the ranks before this
    // block; warp sums stay in s.warp.
    __device__ __forceinline__ u64 sum(u64 v, u64* before) {
        v = warp_sum(v);
        __syncthreads();   // s.warp is read no more
        if (lane == 0) s.warp[warp] = v;
        __syncthreads();
        if (warp == 0) {
            const u64 own = warp_sum(lane < kWarps ? s.warp[lane] : 0ull);
            if (lane < size) st_peer_u64(&s.peer[turn][0][rank], lane, own);
        }
        __syncwarp();
        cluster_sync();
        u64 all = 0, b = 0;
        for (unsigned r = 0; r < size; ++r) {
            if (r == rank) b = all;
            all += s.peer[turn][0][r];
        }
        turn ^= 1;
        if (before) *before = b;
        return all;
    }

    __device__ __forceinline__ u64 greatest(u64 v) {
        v = warp_max(v);
        __syncthreads();
        if (lane == 0) s.warp[warp] = v;
        __syncthreads();
        if (warp == 0) {
            const u64 own = warp_max(lane < kWarps ? s.warp[lane] : 0ull);
            if (lane < size) st_peer_u64(&s.peer[turn][0][rank], lane, own);
        }
        __syncwarp();
        cluster_sync();
        u64 all = 0;
        for (unsigned r = 0; r < size; ++r) all = max(all, s.peer[turn][0][r]);
        turn ^= 1;
        return all;
    }
};

// Where a prefix of the falling order ends: all keys above `key`, and of the tokens that
// have it those with index < limit.
struct Cut {
    unsigned key;
    int limit;
};

// u T for u in [0, 1], T < 2^63, rounded down, or up
template <bool UP>
__device__ __forceinline__ u64 part_of(float u, u64 T) {
    if (!(u > 0.f)) return 0;
    if (u >= 1.f) return T;
    const unsigned b = __float_as_uint(u), be = b >> 23;
    const u64 m = be ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
    const int down = 150 - static_cast<int>(be ? be : 1u);   // u = m 2^-down, down from 24 to 149
    const u64 lo = m * T, hi = __umul64hi(m, T);
    u64 whole = 0;
    bool rest;
    if (down >= 128) {   // hi has 23 bits at most
        rest = true;
    } else if (down >= 64) {
        whole = hi >> (down - 64);
        rest = lo != 0 || (hi & ((1ull << (down - 64)) - 1)) != 0;
    } else {
        whole = (lo >> down) | (hi << (64 - down));
        rest = (lo & ((1ull << down) - 1)) != 0;
    }
    return whole + (UP && rest ? 1u : 0u);
}

__global__ void __launch_bounds__(kThreads) sample_kernel(const __grid_constant__ SampleParams p) {
    __shared__ Shared s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Block c{s, cluster_rank(), cluster_size(), tid, lane, warp};
    cluster_arrive();
    if (tid < 32) s.pow[tid] = kPow[tid];
    stream_order();
    const int b = blockIdx.y / p.T, t = blockIdx.y % p.T;
    Row row;
    row.x = static_cast<const char*>(p.x) + (b * p.xs[0] + t * p.xs[1]) * (p.x_dt == LAR_F32 ? 4 : 2);
    row.xs = p.xs[2];
    row.dt = p.x_dt;
    row.V = static_cast<int>(p.V);
    row.off = row.xs == 1 ? static_cast<int>((reinterpret_cast<uintptr_t>(row.x) & 15) / (p.x_dt == LAR_F32 ? 4 : 2)) : 0;
    const int steps = (row.V + row.off + kStep - 1) / kStep;
    const int w_all = static_cast<int>(c.size) * kWarps, w_me = static_cast<int>(c.rank) * kWarps + warp;
    auto first_step = [&](int w) { return static_cast<int>(static_cast<int64_t>(steps) * w / w_all); };
    const int s0 = first_step(w_me), s1 = first_step(w_me + 1);
    auto each = [&](auto f) {
        for (int st = s0; st < s1; ++st) row.eight(st * kStep + lane * 8, f);
    };

    // the greatest logit and its lowest index, and how many are above -infinity
    u64 top = 0;
    unsigned some = 0;
    each([&](int i, float x) {
        const u64 v = static_cast<u64>(key_of(x)) << 32 | (0xffffffffu - static_cast<unsigned>(i));
        top = v > top ? v : top;
        some += x > -INFINITY;
    });
    cluster_wait();   // every block runs: its memory may be written
    top = c.greatest(top);
    const u64 N = c.sum(some, nullptr);
    const int first = static_cast<int>(0xffffffffu - static_cast<unsigned>(top));
    const unsigned top_key = static_cast<unsigned>(top >> 32);
    const float greatest = of_key(top_key);

    const float temp = p.temp ? __ldg(p.temp + b * p.temp_s) : 1.f;
    const float top_p = p.top_p ? __ldg(p.top_p + b * p.tp_s) : 1.f;
    const float min_p = p.min_p ? __ldg(p.min_p + b * p.mp_s) : 0.f;
    int64_t k = p.top_k ? ld_idx(p.top_k, b * p.tk_s, p.tk_dt) : 0;
    if (k < 0) k = 0;
    const float u = __ldg(p.u + b * p.us[0] + t * p.us[1]);
    const bool none = N == 0;
    const bool single = !(temp > 0.f) || k == 1 || !(top_p > 0.f) || min_p > 1.f;

    auto put = [&](int64_t v) {
        const int64_t o = b * p.ts[0] + t * p.ts[1];
        if (p.tok_dt == LAR_I32) static_cast<int32_t*>(p.tok)[o] = static_cast<int32_t>(v);
        else static_cast<int64_t*>(p.tok)[o] = v;
    };
    // neighbours on neighbouring lanes
    auto put_probs = [&](auto f) {
        if (!p.probs) return;
        float* out = p.probs + b * p.ps[0] + t * p.ps[1];
        const int lo = max(0, s0 * kStep - row.off), hi = min(row.V, s1 * kStep - row.off);
        for (int i = lo + lane; i < hi; i += 32) out[i * p.ps[2]] = f(i);
    };
    if (none || single) {
        if (c.rank == 0 && tid == 0) {
            put(none ? -1 : first);
            if (none) flag_err(p.dev_err, LAR_DEVERR_PROBS);
        }
        put_probs([&](int i) { return !none && i == first ? 1.f : 0.f; });
        cluster_sync();   // no block leaves while another may still write to it
        return;
    }

    if (tid == 0) {
        const double q = 2.0 * 1.4426950408889634074 / static_cast<double>(temp);
        s.scale_hi = static_cast<float>(q);
        s.scale_lo = q < 3e38 ? static_cast<float>(q - static_cast<double>(s.scale_hi)) : 0.f;
    }
    __syncthreads();
    Scale sc;
    sc.half_max = 0.5f * greatest;
    sc.hi = s.scale_hi;
    sc.lo = s.scale_lo;
    sc.infinite = greatest == INFINITY;

    Cut cut = {kLeast, row.V};   // keep everything above -infinity (its weight is 0)
    auto kept = [&](int i, unsigned key) { return key > cut.key || (key == cut.key && i < cut.limit); };

    // The first index (in order) with  sum of f up to it > target;  in s.found[0] of every block.
    auto select = [&](u64 before, u64 target, auto f) {
        // s.warp holds this block's warp sums of f, `before` the sum of the blocks before
        if (tid == 0) s.found[0] = ~0ull;
        u64 start = before;
        for (int w = 0; w < warp; ++w) start += s.warp[w];
        const u64 own = s.warp[warp];
        cluster_sync();
        if (start <= target && target < start + own) {   // one warp of the cluster
            for (int st = s0; st < s1; ++st) {
                u64 w8[8];
                int idx = -1;
#pragma unroll
                for (int e = 0; e < 8; ++e) w8[e] = 0;
                const int i0 = st * kStep + lane * 8 - row.off;
                row.eight(st * kStep + lane * 8, [&](int i, float x) { w8[i - i0] = f(i, x); });
                u64 sum8 = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) sum8 += w8[e];
                const u64 incl = warp_scan(sum8, lane);
                u64 run = start + incl - sum8;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    run += w8[e];
                    if (idx < 0 && run > target) idx = i0 + e;
                }
                const unsigned has = __ballot_sync(0xffffffffu, idx >= 0);
                if (has) {
                    idx = __shfl_sync(0xffffffffu, idx, __ffs(has) - 1);
                    if (lane < c.size) st_peer_u64(&s.found[0], lane, static_cast<u64>(idx));
                    break;
                }
                start += __shfl_sync(0xffffffffu, incl, 31);
            }
        }
        __syncwarp();
        cluster_sync();
    };

    // The cut at which the sum of f over a prefix reaches `target` (which the whole sum
    // does); `each_is` is what a token with the cut's own key adds.
    auto find_cut = [&](u64 target, auto f, auto of_one) {
        unsigned lo = cut.key, hi = top_key;
        u64 above = 0, at = 0;
        while (true) {
            int shift = 0;
            while (((hi - lo) >> shift) >= kBins) ++shift;
            for (int i = tid; i < kBins; i += kThreads) s.lo[i] = s.hi[i] = 0;
            __syncthreads();
            each([&](int i, float x) {
                const unsigned key = key_of(x);
                if (key < lo || key > hi || !kept(i, key)) return;
                const u64 w = f(x);
                if (w == 0) return;
                const unsigned bin = (key - lo) >> shift, wl = static_cast<unsigned>(w);
                const unsigned old = atomicAdd(&s.lo[bin], wl);
                const unsigned wh = static_cast<unsigned>(w >> 32) + (old + wl < old ? 1u : 0u);
                if (wh) atomicAdd(&s.hi[bin], wh);
            });
            __syncwarp();
            cluster_sync();
            // this block's bins, from the top: a thread `per` of them
            const int slice = kBins / static_cast<int>(c.size), per = (slice + kThreads - 1) / kThreads;
            const int base = kBins - 1 - static_cast<int>(c.rank) * slice;   // its highest bin
            u64 bins[kBins / kThreads];
            u64 mine = 0;
#pragma unroll
            for (int e = 0; e < kBins / kThreads; ++e) {
                bins[e] = 0;
                const int q = tid * per + e;
                if (e < per && q < slice) {
                    for (unsigned r = 0; r < c.size; ++r) {
                        unsigned l, h;
                        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(l) : "r"(peer_addr(&s.lo[base - q], r)));
                        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(h) : "r"(peer_addr(&s.hi[base - q], r)));
                        bins[e] += static_cast<u64>(h) << 32 | l;
                    }
                }
                mine += bins[e];
            }
            u64 before;
            c.sum(mine, &before);
            u64 run = above + before;
            for (int w = 0; w < warp; ++w) run += s.warp[w];
            run += warp_scan(mine, lane) - mine;
            if (run < target && run + mine >= target) {   // one thread of the cluster
                int e = 0;
                while (run + bins[e] < target) run += bins[e++];
                u64 got = 0;
#pragma unroll
                for (int q = 0; q < kBins / kThreads; ++q)
                    if (q == e) got = bins[q];
                for (unsigned r = 0; r < c.size; ++r) {
                    st_peer_u64(&s.found[1], r, static_cast<u64>(base - tid * per - e));
                    st_peer_u64(&s.found[2], r, run);
                    st_peer_u64(&s.found[3], r, got);
                }
            }
            __syncwarp();
            cluster_sync();
            above = s.found[2];
            at = s.found[3];
            lo += static_cast<unsigned>(s.found[1]) << shift;
            hi = min(hi, lo + ((1u << shift) - 1));
            if (shift == 0) break;
        }
        const u64 one = of_one(of_key(lo));
        const u64 n = (target - above + one - 1) / one;   // ties kept
        int limit = cut.key == lo ? cut.limit : row.V;
        if (n * one < at) {   // not all: the index behind the n-th
            unsigned same = 0;
            each([&](int i, float x) { same += key_of(x) == lo && i < limit; });
            u64 before;
            c.sum(same, &before);
            const int lim = limit;
            select(before, n - 1, [&](int i, float x) { return static_cast<u64>(key_of(x) == lo && i < lim); });
            limit = static_cast<int>(s.found[0]) + 1;
        }
        cut = {lo, limit};
    };

    if (k > 0 && static_cast<u64>(k) < N)
        find_cut(static_cast<u64>(k), [](float) { return 1ull; }, [](float) { return 1ull; });
    if (top_p < 1.f) {
        u64 mine = 0;
        each([&](int i, float x) { if (kept(i, key_of(x))) mine += sc.weight(x, s.pow); });
        const u64 all = c.sum(mine, nullptr);
        const u64 target = part_of<true>(top_p, all);
        find_cut(target, [&](float x) { return sc.weight(x, s.pow); }, [&](float x) { return sc.weight(x, s.pow); });
    }
    const u64 least = min_p > 0.f ? part_of<true>(min_p, kOne) : 0ull;

    auto weight = [&](int i, float x) {
        if (!kept(i, key_of(x))) return u64{0};
        const u64 w = sc.weight(x, s.pow);
        return w >= least ? w : u64{0};
    };
    u64 mine = 0, before;
    each([&](int i, float x) { mine += weight(i, x); });
    const u64 total = c.sum(mine, &before);
    u64 target = part_of<false>(u, total);
    if (target >= total) target = total - 1;
    select(before, target, weight);
    if (c.rank == 0 && tid == 0) put(static_cast<int64_t>(s.found[0]));
    if (p.probs) {
        const float inv = 1.f / (static_cast<float>(total) * 0x1p-39f);
        put_probs([&](int i) {
            const float x = row.at(i);
            if (!kept(i, key_of(x)) || (least && sc.weight(x, s.pow) < least)) return 0.f;
            if (0.5f * x == sc.half_max) return inv;
            if (sc.infinite) return 0.f;
            float y, e;
            sc.exponent(x, y, e);
            return y >= -200.f ? exp2_f(y) * fmaf(e, 0.69314718f, 1.f) * inv : 0.f;
        });
    }
}

}  // namespace

lar_status launch_sample(const SampleParams& p, void* stream) {
    // a block a few thousand tokens, at most 8 (the portable cluster)
    int size = 1;
    while (size < kMaxCluster && static_cast<int64_t>(size) * 4096 < p.V) size *= 2;
    SampleParams q = p;
    // rows are the grid's y: as many at once as that admits
    const int most = 65535 / p.T;
    for (int64_t b = 0; b < p.B; b += most) {
        q.B = static_cast<int>(p.B - b < most ? p.B - b : most);
        const lar_status st = launch_ordered(sample_kernel, dim3(size, q.B * p.T), kThreads, 0, size, static_cast<cudaStream_t>(stream), q);
        if (st != LAR_OK) return st;
        const int64_t es = p.x_dt == LAR_F32 ? 4 : 2;
        q.x = static_cast<const char*>(q.x) + most * p.xs[0] * es;
        q.u += most * p.us[0];
        if (q.temp) q.temp += most * p.temp_s;
        if (q.top_k) q.top_k = static_cast<const char*>(q.top_k) + most * p.tk_s * (p.tk_dt == LAR_I32 ? 4 : 8);
        if (q.top_p) q.top_p += most * p.tp_s;
        if (q.min_p) q.min_p += most * p.mp_s;
        q.tok = static_cast<char*>(q.tok) + most * p.ts[0] * (p.tok_dt == LAR_I32 ? 4 : 8);
        if (q.probs) q.probs += most * p.ps[0];
    }
    return LAR_OK;
}

}  // namespace lar

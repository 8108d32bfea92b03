// sample.cu -- the draw of a token from a row of logits (sample_tokens): temperature,
// top-k, top-p, min-p and the inversion of the running sum by a given random number.
//
// Order and weights.  Logits are ordered by the bits of their fp32 value (a key that rises
// with it), equal ones by index; each filter keeps a prefix of that order.  A weight
// exp((x - max) / temperature) is a whole number of 2^-(63 - log2 V): a token has to be the
// one that exact sums give, and whole numbers add up exactly in any order, at the rate of
// 32-bit adds, where fp64 is slow on this part.  Its argument is kept in two floats, 2^n
// comes from a table of 256 steps, and the rest, f of at most 1/512, from a polynomial: good to
// 2^-30 of the weight (the table and the product with it 2^-32 each, its rounding 2^-33, f and the
// polynomial's steps 2^-34 each; with 32 steps the last four are 8 times as much and more).
//
// Work.  A row is a cluster's, every warp owning a contiguous stretch of the vocabulary.
// One pass finds the greatest logit.  Then
//   top-k: the k-th of the threads' own maxima (two a thread) is a bound that k logits reach,
//     and hardly more (1.4 k where k is half as many as there are maxima); the logits from
//     it on go to one block, which finds all cuts, and the token, among them.
//   top-p alone: logits are counted in bins, which say in which one the cut lies if every bin
//     weighs its middle; one more pass has all exact sums and takes that bin (or, where they
//     are few, all above it as well) to one block.  Sums that place the cut elsewhere after
//     all are rare, and left to the passes below.
//   neither: the weights of each warp's stretch are added up.
// Where no list is left, the block whose stretch holds the threshold reads it again.  Lists
// that grow past their room (equal logits, sorted ones) are replaced by passes over the
// row that narrow the key down 11 bits at a time.  Ties at a cut are kept from the lowest
// index on.
//
// Measured, 64 x 131072 fp32 (the bytes: 5 us): the greatest alone 14 us, temperature 24,
// top-k 50 21, 1000 29, top-p 52 to 57, equal logits with top-p 271; one such row 6.3, 11, 12, 18,
// 26 and 98.  144 x 50257 bf16 with probabilities 33 (the bytes: 6.4).  64 x 131072 with filters as they
// come 54, of logits that lie two apart 93.  Bound: instructions (26 a
// weight, in each pass that needs them), and the exchanges over a cluster, 1 to 2 us each,
// three with a temperature alone and nine with top-p.
#include "layer_common.cuh"
#include "serve_params.h"

namespace lar {

int cached_occupancy(const void* kern, int threads, size_t smem, size_t smem_max, int* sms_out);

namespace {

using u64 = unsigned long long;

// 256: 64 rows of top-k 1000 46 us instead of 36, one row 28 instead of 23; 1024: no better, and one row slower
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kStep = 256;       // tokens of a warp's step, 8 a lane
constexpr int kBits = 11;        // of a key, looked at in one go
constexpr int kList = 2048;      // room for logits around a cut
constexpr int kBins = 1 << kBits;
constexpr int kSmall = 256;      // entries that are compared with one another

// 2^(31 + j / 256), to the nearest whole number
constexpr int kPowBits = 8, kPows = 1 << kPowBits;
__constant__ unsigned kPow[kPows] = {
    2147483648u, 2153306067u, 2159144272u, 2164998306u, 2170868212u, 2176754033u, 2182655811u, 2188573592u,
    2194507417u, 2200457330u, 2206423375u, 2212405596u, 2218404036u, 2224418739u, 2230449750u, 2236497113u,
    2242560872u, 2248641071u, 2254737756u, 2260850970u, 2266980759u, 2273127167u, 2279290240u, 2285470023u,
    2291666561u, 2297879899u, 2304110083u, 2310357160u, 2316621173u, 2322902170u, 2329200197u, 2335515300u,
    2341847524u, 2348196917u, 2354563524u, 2360947394u, 2367348571u, 2373767105u, 2380203040u, 2386656425u,
    2393127307u, 2399615734u, 2406121752u, 2412645410u, 2419186755u, 2425745836u, 2432322700u, 2438917396u,
    2445529972u, 2452160476u, 2458808958u, 2465475465u, 2472160047u, 2478862753u, 2485583632u, 2492322733u,
    2499080105u, 2505855799u, 2512649863u, 2519462348u, 2526293303u, 2533142779u, 2540010826u, 2546897494u,
    2553802834u, 2560726895u, 2567669730u, 2574631389u, 2581611923u, 2588611383u, 2595629821u, 2602667287u,
    2609723834u, 2616799513u, 2623894376u, 2631008476u, 2638141863u, 2645294591u, 2652466713u, 2659658279u,
    2666869345u, 2674099961u, 2681350181u, 2688620059u, 2695909648u, 2703219000u, 2710548171u, 2717897212u,
    2725266179u, 2732655125u, 2740064105u, 2747493172u, 2754942382u, 2762411789u, 2769901447u, 2777411411u,
    2784941738u, 2792492481u, 2800063696u, 2807655439u, 2815267765u, 2822900730u, 2830554390u, 2838228802u,
    2845924021u, 2853640104u, 2861377107u, 2869135087u, 2876914102u, 2884714207u, 2892535461u, 2900377920u,
    2908241642u, 2916126685u, 2924033107u, 2931960965u, 2939910317u, 2947881223u, 2955873740u, 2963887926u,
    2971923842u, 2979981545u, 2988061094u, 2996162550u, 3004285971u, 3012431416u, 3020598946u, 3028788621u,
    3037000500u, 3045234644u, 3053491112u, 3061769967u, 3070071267u, 3078395075u, 3086741451u, 3095110456u,
    3103502151u, 3111916599u, 3120353861u, 3128813999u, 3137297074u, 3145803149u, 3154332287u, 3162884549u,
    3171459999u, 3180058700u, 3188680714u, 3197326104u, 3205994934u, 3214687269u, 3223403170u, 3232142703u,
    3240905930u, 3249692918u, 3258503729u, 3267338429u, 3276197082u, 3285079754u, 3293986508u, 3302917412u,
    3311872529u, 3320851927u, 3329855670u, 3338883824u, 3347936457u, 3357013633u, 3366115421u, 3375241885u,
    3384393094u, 3393569115u, 3402770014u, 3411995860u, 3421246719u, 3430522660u, 3439823750u, 3449150059u,
    3458501653u, 3467878602u, 3477280975u, 3486708840u, 3496162267u, 3505641324u, 3515146082u, 3524676610u,
    3534232978u, 3543815256u, 3553423514u, 3563057822u, 3572718252u, 3582404874u, 3592117759u, 3601856978u,
    3611622603u, 3621414705u, 3631233356u, 3641078629u, 3650950594u, 3660849326u, 3670774895u, 3680727376u,
    3690706840u, 3700713361u, 3710747013u, 3720807869u, 3730896002u, 3741011488u, 3751154399u, 3761324810u,
    3771522796u, 3781748432u, 3792001792u, 3802282952u, 3812591987u, 3822928972u, 3833293984u, 3843687099u,
    3854108391u, 3864557939u, 3875035819u, 3885542107u, 3896076880u, 3906640216u, 3917232192u, 3927852886u,
    3938502376u, 3949180739u, 3959888054u, 3970624400u, 3981389855u, 3992184498u, 4003008408u, 4013861665u,
    4024744348u, 4035656537u, 4046598312u, 4057569753u, 4068570940u, 4079601955u, 4090662878u, 4101753790u,
    4112874773u, 4124025908u, 4135207276u, 4146418961u, 4157661043u, 4168933606u, 4180236731u, 4191570503u,
    4202935003u, 4214330316u, 4225756525u, 4237213713u, 4248701965u, 4260221365u, 4271771996u, 4283353945u};

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

constexpr float kRound = 12582912.f;   // 1.5 2^23: a sum with it is rounded to a whole number

struct Scale {
    float half_max;     // max / 2: differences of halves do not overflow
    float hi, lo;       // 2 log2(e) / temperature
    int up;             // the greatest weighs 2^up
    bool infinite;      // max is +infinity

    __device__ __forceinline__ u64 one() const { return 1ull << up; }

    // (x - max) log2(e) / temperature as y + e, two at once.  The difference is exact: its
    // error is a float (two-sum).
    __device__ __forceinline__ void exponents(f32x2 x, f32x2& y, f32x2& e) const {
        const f32x2 m = pack2(-half_max, -half_max), minus = pack2(-1.f, -1.f), h = pack2(hi, hi);
        const f32x2 a = mul2(x, pack2(0.5f, 0.5f)), d = add2(a, m), t = fma2(a, minus, d);
        const f32x2 de = add2(fma2(fma2(t, minus, d), minus, a), fma2(t, minus, m));
        y = mul2(d, h);
        e = fma2(d, pack2(lo, lo), fma2(de, h, fma2(d, h, mul2(y, minus))));
    }

    // Weights of two logits (NaN and -infinity weigh nothing): 2^y by whole number, 256th and
    // the rest
    __device__ __forceinline__ void weights(float x0, float x1, const uint2* pow, u64& w0, u64& w1) const {
        if (infinite) {
            w0 = x0 == INFINITY ? one() : 0ull;
            w1 = x1 == INFINITY ? one() : 0ull;
            return;
        }
        f32x2 y, e;
        exponents(pack2(x0, x1), y, e);
        float y0, y1, r0, r1, g0, g1;
        unpack2(y, y0, y1);
        const float least = static_cast<float>(-2 - up);   // from there on a weight is 0
        y = pack2(fmaxf(y0, least), fmaxf(y1, least));
        const f32x2 big = pack2(kRound, kRound), minus = pack2(-1.f, -1.f);
        const f32x2 r = fma2(y, pack2(1.f * kPows, 1.f * kPows), big);
        const f32x2 f = add2(fma2(add2(r, mul2(big, minus)), pack2(-1.f / kPows, -1.f / kPows), y), e);
        // 2^f - 1: ln 2, its powers over the factorials (the next one is below 2^-42)
        f32x2 g = fma2(f, pack2(5.550411e-2f, 5.550411e-2f), pack2(0.24022651f, 0.24022651f));
        g = fma2(f, g, pack2(0.69314718f, 0.69314718f));
        g = mul2(f, g);
        unpack2(r, r0, r1);
        unpack2(g, g0, g1);
        w0 = scaled(r0, g0, pow);
        w1 = scaled(r1, g1, pow);
    }

    // r has the 256ths in its low bits, as a whole number
    __device__ __forceinline__ u64 scaled(float r, float g, const uint2* pow) const {
        const int j = static_cast<int>(__float_as_uint(r));   // kRound's own low 22 bits are 0
        const uint2 t = pow[j & (kPows - 1)];
        const unsigned m = t.x + static_cast<unsigned>(__float2int_rn(g * __uint_as_float(t.y)));
        const int down = 63 - up + (static_cast<int>(__float_as_uint(kRound)) >> kPowBits) - (j >> kPowBits);
        u64 w;
        asm("shr.u64 %0, %1, %2;" : "=l"(w) : "l"(static_cast<u64>(m) << 32), "r"(down));   // by 64 and more: 0
        return w;
    }

    __device__ __forceinline__ u64 weight(float x, const uint2* pow) const {
        u64 a, b;
        weights(x, x, pow, a, b);
        return a;
    }
};

struct Row {
    const char* x;      // element 0
    int64_t xs;         // stride
    int dt;
    int off;            // elements between the last 16-byte border and element 0
    int V;

    __device__ __forceinline__ float at(int i) const { return clean(ld_in(x, i * xs, dt)); }

    // elements [j - off, j - off + 8) as they are, j a multiple of 8; -infinity where there is none
    __device__ __forceinline__ void eight_of(int j, float* a) const {
        const int i = j - off;
        if (xs == 1 && i >= 0 && i + 8 <= V) {
            ld8<true>(x, i, dt, a);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) a[k] = i + k >= 0 && i + k < V ? ld_in(x, (i + k) * xs, dt) : -INFINITY;
        }
    }

    // f(i, x) for them, if they are there
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

// A logit of a list: greater first, lower indices first
__device__ __forceinline__ u64 entry_of(unsigned key, int i) { return static_cast<u64>(key) << 32 | (0xffffffffu - static_cast<unsigned>(i)); }
__device__ __forceinline__ unsigned entry_key(u64 e) { return static_cast<unsigned>(e >> 32); }
__device__ __forceinline__ int entry_index(u64 e) { return static_cast<int>(0xffffffffu - static_cast<unsigned>(e)); }

struct Shared {
    uint2 pow[kPows];              // a whole number, and as a float
    u64 warp[kWarps];
    u64 peer[2][kMaxCluster];      // exchanges in turn
    u64 warp4[4][kWarps], peer4[2][4][kMaxCluster];
    u64 found[4];
    alignas(16) unsigned lo[kBins];
    alignas(16) unsigned hi[kBins];
    u64 list[kList];                // this block's
    union {                        // block 0: the cluster's; before that its threads' maxima
        u64 all[kList];
        unsigned maxima[2 * kList];
    };
    u64 small[kSmall], small_w[kSmall];
    unsigned count, small_n;
    float scale_hi, scale_lo;
};

struct Block {
    Shared& s;
    unsigned rank, size;
    int tid, lane, warp;
    int turn = 0;

    // Joins every thread's v over the cluster, and over the ranks before this block; the warps'
    // own stay in s.warp.
    template <typename F>
    __device__ __forceinline__ u64 over(u64 v, F join, u64* before) {
        __syncthreads();   // s.warp is read no more
        if (lane == 0) s.warp[warp] = v;
        __syncthreads();
        if (warp == 0) {
            u64 own = lane < kWarps ? s.warp[lane] : 0ull;
#pragma unroll
            for (int off = kWarps / 2; off > 0; off >>= 1) own = join(own, __shfl_xor_sync(0xffffffffu, own, off));
            if (lane < size) st_peer_u64(&s.peer[turn][rank], lane, own);
        }
        __syncwarp();
        cluster_sync();
        u64 of[kMaxCluster], all = 0, b = 0;
#pragma unroll
        for (unsigned r = 0; r < kMaxCluster; ++r) of[r] = r < size ? s.peer[turn][r] : 0ull;
#pragma unroll
        for (unsigned r = 0; r < kMaxCluster; ++r) {
            if (r == rank) b = all;
            all = join(all, of[r]);
        }
        turn ^= 1;
        if (before) *before = b;
        return all;
    }

    __device__ __forceinline__ u64 sum(u64 v, u64* before) {
        return over(warp_sum(v), [](u64 a, u64 b) { return a + b; }, before);
    }

    // Four sums at once
    __device__ __forceinline__ void sums(u64 (&v)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = warp_sum(v[e]);
            if (lane == 0) s.warp4[e][warp] = v[e];
        }
        __syncthreads();
        if (warp < 4) {
            u64 own = lane < kWarps ? s.warp4[warp][lane] : 0ull;
            own = warp_sum(own);
            if (lane < size) st_peer_u64(&s.peer4[turn][warp][rank], lane, own);
        }
        __syncwarp();
        cluster_sync();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = 0;
#pragma unroll
            for (unsigned r = 0; r < kMaxCluster; ++r) v[e] += r < size ? s.peer4[turn][e][r] : 0ull;
        }
        turn ^= 1;
    }

    __device__ __forceinline__ u64 greatest(u64 v) {
        return over(warp_max(v), [](u64 a, u64 b) { return a > b ? a : b; }, nullptr);
    }

    __device__ __forceinline__ unsigned own_least(unsigned v) {
        v = __reduce_min_sync(0xffffffffu, v);
        __syncthreads();
        if (lane == 0) s.warp[warp] = v;
        __syncthreads();
        u64 all = s.warp[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) all = s.warp[w] < all ? s.warp[w] : all;
        return static_cast<unsigned>(all);
    }

    // The same over this block alone
    __device__ __forceinline__ u64 own_sum(u64 v) {
        v = warp_sum(v);
        __syncthreads();
        if (lane == 0) s.warp[warp] = v;
        __syncthreads();
        u64 all = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) all += s.warp[w];
        return all;
    }

    // A bin's share of a sum
    __device__ __forceinline__ void add(unsigned bin, u64 w) {
        const unsigned wl = static_cast<unsigned>(w), old = atomicAdd(&s.lo[bin], wl);
        const unsigned wh = static_cast<unsigned>(w >> 32) + (old + wl < old ? 1u : 0u);
        if (wh) atomicAdd(&s.hi[bin], wh);
    }

    __device__ __forceinline__ void clear_bins() {
        for (int i = tid; i < kBins / 4; i += kThreads)
            reinterpret_cast<uint4*>(s.lo)[i] = reinterpret_cast<uint4*>(s.hi)[i] = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
    }

    // The highest bin down to which the bins' sums, as `value` takes them, reach `target_of`
    // (the whole sum), in s.found: bin, the sum above it, its own.  CL: bins of all the
    // cluster's blocks, to all of them.
    template <bool CL, typename V, typename T>
    __device__ __forceinline__ void find_bin(V value, T target_of) {
        const unsigned n = CL ? size : 1, me = CL ? rank : 0;
        if (CL) {
            __syncwarp();
            cluster_sync();
        } else {
            __syncthreads();
        }
        constexpr int E = kBins / kThreads;   // bins of a thread, at most
        const int slice = kBins / static_cast<int>(n), per = slice / kThreads > 0 ? slice / kThreads : 1;
        const int base = kBins - static_cast<int>(me) * slice - per * (tid + 1);   // this thread's lowest bin
        u64 bins[E];   // from its highest down
        u64 mine = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            bins[e] = 0;
            const int q = base + per - 1 - e;
            if (e < per && tid * per < slice) {
                if (CL) {
                    unsigned l[kMaxCluster], h[kMaxCluster];   // all asked for at once
#pragma unroll
                    for (unsigned r = 0; r < kMaxCluster; ++r) {
                        l[r] = h[r] = 0;
                        if (r < n) {
                            asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(l[r]) : "r"(peer_addr(&s.lo[q], r)));
                            asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(h[r]) : "r"(peer_addr(&s.hi[q], r)));
                        }
                    }
#pragma unroll
                    for (unsigned r = 0; r < kMaxCluster; ++r) bins[e] += static_cast<u64>(h[r]) << 32 | l[r];
                } else {
                    bins[e] = static_cast<u64>(s.hi[q]) << 32 | s.lo[q];
                }
                bins[e] = value(q, bins[e]);
            }
            mine += bins[e];
        }
        u64 run = 0;
        const u64 target = target_of(CL ? sum(mine, &run) : own_sum(mine));
        for (int w = 0; w < warp; ++w) run += s.warp[w];
        run += warp_scan(mine, lane) - mine;
        if (run < target && run + mine >= target) {   // one thread
            int at = -1;
            u64 got = 0;
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (at < 0) {
                    if (run + bins[e] >= target) {
                        at = e;
                        got = bins[e];
                    } else {
                        run += bins[e];
                    }
                }
            for (unsigned r = 0; r < n; ++r) {
                const unsigned to = CL ? r : rank;
                st_peer_u64(&s.found[1], to, static_cast<u64>(base + per - 1 - at));
                st_peer_u64(&s.found[2], to, run);
                st_peer_u64(&s.found[3], to, got);
            }
        }
        __syncwarp();
        if (CL) cluster_sync();
        else __syncthreads();
    }

    // The greatest key in [lo, hi] down to which the sums of f reach `target` (which they do):
    // s.found[2] is the sum above it, s.found[3] its own.  each(g) calls g(key, i, x) for
    // the values in question.
    template <bool CL, typename E, typename F>
    __device__ __forceinline__ unsigned find_key(unsigned lo, unsigned hi, u64 target, E each, F f) {
        u64 above = 0;
        for (int round = 0; round < 3; ++round) {   // 32 bits, 11 at a time
            int shift = 0;
            while (((hi - lo) >> shift) >= kBins) ++shift;
            clear_bins();
            each([&](unsigned key, int i, float x) {
                if (key < lo || key > hi) return;
                const u64 w = f(key, i, x);
                if (w) add((key - lo) >> shift, w);
            });
            find_bin<CL>([](int, u64 v) { return v; }, [&](u64) { return target - above; });
            above += s.found[2];
            lo += static_cast<unsigned>(s.found[1]) << shift;
            hi = lo + min(hi - lo, (1u << shift) - 1);
            if (shift == 0) break;
        }
        __syncthreads();
        if (tid == 0) s.found[2] = above;
        __syncthreads();
        return lo;
    }

    // By this block alone: of values with places in [lo, hi], no two the same, the one at which
    // the sums of the weights from the highest place down reach `target` (which they do).
    // each(g) calls g(place, weight).
    template <typename E>
    __device__ __forceinline__ u64 find_place(u64 lo, u64 hi, u64 target, E each) {
        u64 above = 0;
        for (int round = 0; round < 6; ++round) {   // 64 bits, 11 at a time
            const int shift = max(0, 64 - kBits - __clzll(static_cast<long long>(hi - lo)));
            clear_bins();
            each([&](u64 at, u64 w) {
                if (at >= lo && at <= hi && w) add(static_cast<unsigned>((at - lo) >> shift), w);
            });
            find_bin<false>([](int, u64 v) { return v; }, [&](u64) { return target - above; });
            above += s.found[2];
            lo += s.found[1] << shift;
            const u64 wide = (1ull << shift) - 1;
            hi = hi - lo < wide ? hi : lo + wide;
            if (shift == 0) break;
            // few in the bin: each is compared with all
            if (tid == 0) s.small_n = 0;
            __syncthreads();
            each([&](u64 at, u64 w) {
                if (at < lo || at > hi || !w) return;
                const unsigned n = atomicAdd(&s.small_n, 1u);
                if (n < kSmall) {
                    s.small[n] = at;
                    s.small_w[n] = w;
                }
            });
            __syncthreads();
            const int n = static_cast<int>(s.small_n);
            if (n > kSmall) continue;
            if (tid < n) {
                const u64 at = s.small[tid];
                u64 run = above;
#pragma unroll 8
                for (int i = 0; i < n; ++i) run += s.small[i] >= at ? s.small_w[i] : 0ull;
                if (run >= target && run - s.small_w[tid] < target) s.found[0] = at;   // one thread
            }
            __syncthreads();
            return s.found[0];
        }
        return lo;
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

__global__ void __launch_bounds__(kThreads, 1024 / kThreads) sample_kernel(const __grid_constant__ SampleParams p) {
    extern __shared__ __align__(16) unsigned char smem[];
    Shared& s = *reinterpret_cast<Shared*>(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Block c{s, cluster_rank(), cluster_size(), tid, lane, warp};
    cluster_arrive();
    static_assert(kPows <= kThreads, "");
    if (tid < kPows) s.pow[tid] = make_uint2(kPow[tid], __float_as_uint(static_cast<float>(kPow[tid])));
    if (tid == 0) s.count = 0;
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

    const float temp = p.temp ? __ldg(p.temp + b * p.temp_s) : 1.f;
    const float top_p = p.top_p ? __ldg(p.top_p + b * p.tp_s) : 1.f;
    const float min_p = p.min_p ? __ldg(p.min_p + b * p.mp_s) : 0.f;
    int64_t k = p.top_k ? ld_idx(p.top_k, b * p.tk_s, p.tk_dt) : 0;
    if (k < 0 || k >= row.V) k = 0;
    const float u = __ldg(p.u + b * p.us[0] + t * p.us[1]);
    const bool single = !(temp > 0.f) || k == 1 || !(top_p > 0.f) || min_p > 1.f;
    const bool by_k = k > 0 && !single;

    // the greatest logit, and two maxima a thread
    float most0 = -INFINITY, most1 = -INFINITY;
#pragma unroll 4
    for (int st = s0; st < s1; ++st) {
        float x[8];
        row.eight_of(st * kStep + lane * 8, x);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            most0 = fmaxf(most0, x[e]);
            most1 = fmaxf(most1, x[e + 4]);
        }
    }
    cluster_wait();   // every block runs: its memory may be written
    most0 += 0.f;   // -0 is 0
    most1 += 0.f;
    const float most = fmaxf(most0, most1);
    // maxima of as many groups of logits as there is room for: two a thread, or one
    static_assert(kMaxCluster * kThreads <= 2 * kList, "");
    const int groups = min(2 * static_cast<int>(c.size) * kThreads, 2 * kList);
    if (by_k) {
        const int id = static_cast<int>(c.rank) * kThreads + tid;
        auto push = [&](int at, float x) {
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer_addr(&s.maxima[at], 0)), "r"(key_of(x)) : "memory");
        };
        const int all = static_cast<int>(c.size) * kThreads;
        if (2 * all <= groups) {
            push(id, most0);
            push(id + all, most1);
        } else {
            push(id, most);
        }
    }
    const unsigned top_key = static_cast<unsigned>(c.greatest(key_of(most)));
    const float greatest = of_key(top_key);
    const bool none = top_key == kLeast;

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
#pragma unroll 4
        for (int i = lo + lane; i < hi; i += 32) out[i * p.ps[2]] = f(i);
    };
    if (none || single) {
        int first = row.V;
        if (!none) {
            each([&](int i, float x) { if (x == greatest) first = min(first, i); });
            first = static_cast<int>(0xffffffffu - static_cast<unsigned>(c.greatest(0xffffffffu - static_cast<unsigned>(first))));
        }
        if (c.rank == 0 && tid == 0) {
            put(none ? -1 : first);
            if (none) flag_err(p.dev_err, LAR_DEVERR_PROBS);
        }
        put_probs([&](int i) { return !none && i == first ? 1.f : 0.f; });
        return;   // every exchange is behind a barrier that all have passed
    }

    if (tid == 0) {
        const double q = 2.0 * 1.4426950408889634074 / static_cast<double>(temp);
        s.scale_hi = q < 3e38 ? static_cast<float>(q) : 3e38f;
        s.scale_lo = q < 3e38 ? static_cast<float>(q - static_cast<double>(s.scale_hi)) : 0.f;
    }
    __syncthreads();
    Scale sc;
    sc.half_max = 0.5f * greatest;
    sc.hi = s.scale_hi;
    sc.lo = s.scale_lo;
    sc.infinite = greatest == INFINITY;
    sc.up = 63 - (32 - __clz(row.V - 1));   // so that V of the greatest sum up to 2^63
    const u64 least = min_p > 0.f ? part_of<true>(min_p, sc.one()) : 0ull;

    Cut cut = {kLeast, row.V};   // everything above -infinity (whose weight is 0)
    auto kept = [&](int i, unsigned key) { return key > cut.key || (key == cut.key && i < cut.limit); };
    auto weight = [&](int i, float x) {   // of the draw
        if (!kept(i, key_of(x))) return u64{0};
        const u64 w = sc.weight(x, s.pow);
        return w >= least ? w : u64{0};
    };
    // f(i, x, x', w, w'): all of the warp's logits and their neighbours with their weights; i may
    // lie outside the row, where the weight is 0
    auto each_weight2 = [&](auto f) {
        for (int st = s0; st < s1; ++st) {
            float x[8];
            row.eight_of(st * kStep + lane * 8, x);
            const int i0 = st * kStep + lane * 8 - row.off;
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                u64 a, b;
                sc.weights(x[e], x[e + 1], s.pow, a, b);
                f(i0 + e, x[e], x[e + 1], a, b);
            }
        }
    };
    auto of_row = [&](auto g) {
        each([&](int i, float x) {
            const unsigned key = key_of(x);
            if (kept(i, key)) g(key, i, x);
        });
    };
    auto to_list = [&](unsigned key, int i) {
        const unsigned at = atomicAdd(&s.count, 1u);
        if (at < kList) s.list[at] = entry_of(key, i);
    };
    // How many logits the cluster's lists have; if they all fit, they are in block 0's s.all
    auto gather = [&] {
        __syncthreads();
        const unsigned mine = s.count;
        u64 before;
        const u64 n = c.sum(tid != 0 ? 0u : mine <= kList ? mine : kList + 1, &before);
        if (n <= kList)
            for (unsigned i = tid; i < mine; i += kThreads) st_peer_u64(&s.all[before + i], 0, s.list[i]);
        __syncwarp();
        cluster_sync();
        return n;
    };
    u64 n_list = 0;
    unsigned list_low = kLeast, list_high = top_key;   // no key of the list lies outside
    auto of_list = [&](auto g) {
        for (unsigned i = tid; i < n_list; i += kThreads) {
            const unsigned key = entry_key(s.all[i]);
            const int at = entry_index(s.all[i]);
            if (kept(at, key)) g(key, at, of_key(key));
        }
    };
    u64 total = 0;
    bool drawn = false;
    // Block 0's list: 0 the cut of top-k, 1 that of top-p, 2 the token; from stage `begin` on, whose
    // sum is `target` where that is known.  One loop for all: the code of a kernel has to fit
    // the instruction cache.
    auto work_list = [&](int begin, u64 target, bool to_draw) {
#pragma unroll 1
        for (int stage = begin; stage < 3; ++stage) {
            if (stage == 1 && !(top_p < 1.f)) continue;
            if (stage == 2 && !to_draw) break;
            auto each_of = [&](auto g) {
                of_list([&](unsigned key, int i, float x) {
                    const u64 w = stage == 0 ? 1ull : sc.weight(x, s.pow);
                    g(stage == 2 ? 0xffffffffull - static_cast<unsigned>(i) : entry_of(key, i), stage == 2 && w < least ? 0ull : w);
                });
            };
            if (target == 0) {
                u64 w = 0;
                each_of([&](u64, u64 v) { w += v; });
                const u64 all = c.own_sum(w);
                if (stage == 1) {
                    target = part_of<true>(top_p, all);
                } else {
                    total = all;
                    target = part_of<false>(u, all) + 1;
                    if (target > all) target = all;
                }
            }
            const u64 low = stage == 2 ? 0xffffffffull - static_cast<unsigned>(row.V) : entry_of(list_low, 0x7fffffff);
            const u64 at = c.find_place(low, stage == 2 ? 0xffffffffull : entry_of(list_high, 0), target, each_of);
            __syncthreads();
            if (stage < 2) cut = {entry_key(at), entry_index(at) + 1};
            else if (tid == 0) put(static_cast<int64_t>(0xffffffffull - at));
            target = 0;
        }
    };
    // The cut behind the first logits of the row whose sum of f reaches `target`
    auto cut_row = [&](u64 target, auto f) {
        const unsigned key = c.template find_key<true>(cut.key, top_key, target, of_row, f);
        const u64 above = s.found[2], at = s.found[3], w1 = f(key, 0, of_key(key));
        const u64 n = (target - above + w1 - 1) / w1;   // of the equal ones, this many
        int limit = cut.key == key ? cut.limit : row.V;
        __syncthreads();
        if (n * w1 < at) {
            const unsigned last = c.template find_key<true>(
                0xffffffffu - static_cast<unsigned>(row.V), 0xffffffffu, n,
                [&](auto g) { of_row([&](unsigned q, int i, float x) { if (q == key) g(0xffffffffu - static_cast<unsigned>(i), i, x); }); },
                [](unsigned, int, float) { return u64{1}; });
            limit = static_cast<int>(0xffffffffu - last) + 1;
        }
        cut = {key, limit};
    };

    // Block 0's cut and sum, to all blocks
    auto tell_all = [&] {
        if (tid < static_cast<int>(c.size)) {
            st_peer_u64(&s.found[0], tid, static_cast<u64>(cut.key) << 32 | static_cast<unsigned>(cut.limit));
            st_peer_u64(&s.found[1], tid, total);
        }
    };
    auto hear = [&] {
        __syncwarp();
        cluster_sync();
        cut = {static_cast<unsigned>(s.found[0] >> 32), static_cast<int>(static_cast<unsigned>(s.found[0]))};
        total = s.found[1];
    };
    bool summed = false;   // the warps' sums of what the draw is among
    u64 mine = 0;
    bool listed = false;   // block 0's list has the cuts: work_list's arguments
    int list_begin = 0;
    u64 list_target = 0;
    if (by_k) {
        unsigned bound = kLeast;
        if (k <= groups) {
            if (c.rank == 0) {
                // the k-th maximum, or a little less: one look at the bins between the least and the greatest
                unsigned low = 0xffffffffu;
                for (int i = tid; i < groups; i += kThreads) low = min(low, s.maxima[i]);
                low = c.own_least(low);
                const int shift = max(0, 32 - kBits - __clz(static_cast<int>(top_key - low)));
                c.clear_bins();
                for (int i = tid; i < groups; i += kThreads) atomicAdd(&s.lo[(s.maxima[i] - low) >> shift], 1u);
                c.template find_bin<false>([](int, u64 v) { return v; }, [&](u64) { return static_cast<u64>(k); });
                if (tid < static_cast<int>(c.size)) st_peer_u64(&s.found[0], tid, low + (s.found[1] << shift));
            }
            __syncwarp();
            cluster_sync();
            bound = static_cast<unsigned>(s.found[0]);
        }
        n_list = kList + 1;
        if (k <= groups || row.V <= kList) {
            // fewer maxima than k above -infinity, as a mask leaves: all logits above it
            if (k <= groups) bound = max(bound, kLeast + 1);
            const float least_x = of_key(bound);
            for (int st = s0; st < s1; ++st) {
                float x[8], high = -INFINITY;
                row.eight_of(st * kStep + lane * 8, x);
                const int i0 = st * kStep + lane * 8 - row.off;
#pragma unroll
                for (int e = 0; e < 8; ++e) high = fmaxf(high, x[e]);
                if (!(high >= least_x)) continue;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (clean(x[e]) >= least_x && i0 + e >= 0 && i0 + e < row.V) to_list(key_of(clean(x[e])), i0 + e);
            }
            n_list = gather();
        }
        list_low = bound;
        if (n_list <= kList) {
            if (c.rank == 0) {
                const bool all = n_list <= static_cast<u64>(k);
                if (all) cut = {bound, row.V};
                list_begin = all ? 1 : 0;
                list_target = all ? 0 : static_cast<u64>(k);
            }
            drawn = listed = true;
        }
    }
    bool p_done = false;
    if (!by_k && top_p < 1.f) {
        // bins of equal widths over the logits that weigh anything
        const float low = fmaxf(greatest - 0.6931472f * (sc.up + 1) * temp, -3e38f), to_bin = (kBins - 1) / (greatest - low);
        auto bin_of = [&](float x) { return min(kBins - 1, max(0, static_cast<int>((x - low) * to_bin))); };
        c.clear_bins();
#pragma unroll 2
        for (int st = s0; st < s1; ++st) {
            float x[8];
            row.eight_of(st * kStep + lane * 8, x);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (x[e] >= low) atomicAdd(&s.lo[bin_of(x[e])], 1u);
        }
        const float width = 1.f / to_bin;
        c.template find_bin<true>([&](int q, u64 n) { return n ? n * sc.weight(fminf(greatest, low + (q + 0.5f) * width), s.pow) : 0ull; },
                                  [&](u64 all) { return max(u64{1}, part_of<true>(top_p, all)); });
        const int bin = static_cast<int>(s.found[1]);
        // How many lie in and above it, and in the 3, 7 and 17 bins around it: a bin's middle is up
        // to 0.8 % off, so the cut may lie in a neighbour.  The list takes all of them or, where
        // they are too many, the widest of these windows that fits.
        u64 n[4] = {0, 0, 0, 0};
        for (int q = max(0, bin - 8) + tid; q < kBins; q += kThreads) {
            const unsigned v = s.lo[q];
            if (q >= bin - 3) n[0] += v;
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (abs(q - bin) <= (e == 0 ? 1 : e == 1 ? 3 : 8)) n[e + 1] += v;
        }
        c.sums(n);
        const bool few = n[0] <= kList;
        const int around = n[3] <= kList ? 8 : n[2] <= kList ? 3 : n[1] <= kList ? 1 : 0;
        const float from = low + (few ? bin - 3 : bin - around) * width, to = few ? INFINITY : low + (bin + around + 1) * width;
        // exact sums: of all, of what lies above the list's, of those
        u64 got[4] = {0, 0, 0, 0};
        each_weight2([&](int i, float x0, float x1, u64 w0, u64 w1) {
            got[0] += w0 + w1;
            if (!(fmaxf(x0, x1) >= from)) return;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float x = e ? x1 : x0;
                const u64 w = e ? w1 : w0;
                if (!(x >= from) || w == 0) continue;
                if (x > to) {
                    got[1] += w;
                    mine += w >= least ? w : 0ull;
                } else {
                    got[2] += w;
                    to_list(key_of(clean(x)), i + e);
                }
            }
        });
        c.sums(got);
        const u64 all = got[0], above = got[1], own = got[2];
        n_list = gather();
        list_low = key_of(clean(from));
        if (!few) list_high = key_of(clean(to));
        const u64 target = part_of<true>(top_p, all);
        if (n_list <= kList && above < target && target <= above + own) {
            list_begin = 1;
            list_target = target - above;
            p_done = listed = true;
            drawn = few;
        }
    }
    if (listed) {
        const bool tell = !drawn || p.probs != nullptr;   // else the other blocks may be gone: nothing is sent to them
        if (c.rank == 0) {
            work_list(list_begin, list_target, drawn);
            if (tell) tell_all();
        }
        if (tell) hear();
        if (!drawn) {
            // each warp its own of the lists'
            for (unsigned i = lane; i < s.count; i += 32) {
                const int at = entry_index(s.list[i]), st = (at + row.off) / kStep;
                if (st >= s0 && st < s1) mine += weight(at, of_key(entry_key(s.list[i])));
            }
            summed = true;
        }
    } else {
#pragma unroll 1
        for (int stage = 0; stage < 2; ++stage) {   // passes over the row instead: top-k, top-p
            if (stage == 0 ? !by_k : !(top_p < 1.f) || p_done) continue;
            auto f = [&](unsigned, int, float x) { return stage == 0 ? u64{1} : sc.weight(x, s.pow); };
            u64 target = static_cast<u64>(k);
            if (stage == 1) {
                u64 w = 0;
                of_row([&](unsigned, int, float x) { w += sc.weight(x, s.pow); });
                target = part_of<true>(top_p, c.sum(w, nullptr));
            }
            cut_row(target, f);
        }
    }
    if (!drawn) {
        u64 start;
        if (!summed) {
            mine = 0;
            if (cut.key == kLeast && !least)   // the same with a test in the loop is 4 % slower
                each_weight2([&](int, float, float, u64 w0, u64 w1) { mine += w0 + w1; });
            else
                each_weight2([&](int i, float x0, float x1, u64 w0, u64 w1) {
                    mine += w0 >= least && kept(i, key_of(clean(x0))) ? w0 : 0ull;
                    mine += w1 >= least && kept(i + 1, key_of(clean(x1))) ? w1 : 0ull;
                });
        }
        total = c.sum(mine, &start);
        u64 target = part_of<false>(u, total);
        if (target >= total) target = total - 1;
        // the one warp of the cluster whose stretch holds it; its block goes through that, 8
        // neighbours a thread
        int owner = -1;
        for (int w = 0; w < kWarps; ++w) {
            const u64 own = s.warp[w];
            if (start <= target && target < start + own) {
                owner = w;
                break;
            }
            start += own;
        }
        if (owner >= 0) {
            const int o_me = static_cast<int>(c.rank) * kWarps + owner, end = first_step(o_me + 1) * kStep;
            for (int j0 = first_step(o_me) * kStep; j0 < end; j0 += kThreads * 8) {
                const int j = j0 + tid * 8, i0 = j - row.off;
                u64 w8[8], sum8 = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) w8[e] = 0;
                if (j < end) row.eight(j, [&](int i, float x) { w8[i - i0] = weight(i, x); });
#pragma unroll
                for (int e = 0; e < 8; ++e) sum8 += w8[e];
                const u64 incl = warp_scan(sum8, lane);
                __syncthreads();   // s.warp is read no more
                if (lane == 31) s.warp[warp] = incl;
                __syncthreads();
                u64 run = start + incl - sum8, all = start;
                for (int w = 0; w < kWarps; ++w) {
                    if (w == warp) run += all - start;
                    all += s.warp[w];
                }
                if (run <= target && target < run + sum8) {   // one thread
                    int idx = -1;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        run += w8[e];
                        if (idx < 0 && run > target) idx = i0 + e;
                    }
                    put(idx);
                }
                if (target < all) break;
                start = all;
            }
        }
    }
    if (p.probs) {
        float* out = p.probs + b * p.ps[0] + t * p.ps[1];
        const float inv = 1.f / ldexpf(static_cast<float>(total), -sc.up);
        const bool all = cut.key == kLeast && !least;
        // Eight neighbours a lane are worked out, and written by neighbouring lanes: rows of
        // odd sizes have no 16-byte borders in common with what is read.
        float* const mine8 = reinterpret_cast<float*>(s.lo) + warp * kStep;   // the bins are done with
        static_assert(kWarps * kStep * sizeof(float) <= sizeof(s.lo) + sizeof(s.hi), "");
        for (int st = s0; st < s1; ++st) {
            float x[8];
            row.eight_of(st * kStep + lane * 8, x);
            const int i0 = st * kStep - row.off;
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                f32x2 y, er;
                sc.exponents(pack2(x[e], x[e + 1]), y, er);
                er = fma2(er, pack2(0.69314718f, 0.69314718f), pack2(1.f, 1.f));
                float v[2], q[2];
                unpack2(y, v[0], v[1]);
                unpack2(er, q[0], q[1]);
#pragma unroll
                for (int k = 0; k < 2; ++k) x[e + k] = v[k] >= -200.f ? exp2_f(v[k]) * inv * q[k] : sc.infinite && x[e + k] == INFINITY ? inv : 0.f;
            }
            if (!all) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int i = i0 + lane * 8 + e;
                    if (!(x[e] > 0.f) || i < 0 || i >= row.V) continue;
                    const float z = row.at(i);
                    if (!kept(i, key_of(z)) || (least && sc.weight(z, s.pow) < least)) x[e] = 0.f;
                }
            }
            __syncwarp();
            float4* to = reinterpret_cast<float4*>(mine8 + lane * 8);
            to[0] = make_float4(x[0], x[1], x[2], x[3]);
            to[1] = make_float4(x[4], x[5], x[6], x[7]);
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = i0 + e * 32 + lane;
                if (i >= 0 && i < row.V) out[i * p.ps[2]] = mine8[e * 32 + lane];
            }
        }
    }
}

}  // namespace

lar_status launch_sample(const SampleParams& p, void* stream) {
    // a block a few thousand tokens, at most 8 (the portable cluster), and no more blocks
    // than the device holds at once while rows are long enough to make up for that
    int sms = 0;
    const int occ = cached_occupancy(reinterpret_cast<const void*>(sample_kernel), kThreads, sizeof(Shared), sizeof(Shared), &sms);
    if (occ < 1) return LAR_ERR_LAUNCH;
    const int64_t rows = static_cast<int64_t>(p.B) * p.T;
    int size = 1;
    while (size < kMaxCluster && static_cast<int64_t>(size) * 2048 < p.V && 2 * size * rows <= static_cast<int64_t>(sms) * occ) size *= 2;
    SampleParams q = p;
    // rows are the grid's y: as many at once as that admits
    const int most = 65535 / p.T;
    for (int64_t b = 0; b < p.B; b += most) {
        q.B = static_cast<int>(p.B - b < most ? p.B - b : most);
        const lar_status st = launch_ordered(sample_kernel, dim3(size, q.B * p.T), kThreads, sizeof(Shared), size, static_cast<cudaStream_t>(stream), q);
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

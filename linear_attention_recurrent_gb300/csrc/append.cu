// append.cu -- keys and values enter a paged cache, keys and queries rotated by their
// place on the way (kv_append).
//
// Rotation: the pair (x, y) of frequency f at place t turns by t f.  The turn is kept in
// fixed point: f / 2 pi is worked out once a block to 2^-64 turns in whole numbers, its
// product with t wraps around like the angle itself, so a place of a million loses no
// more than one of a hundred (t 2^-64 turns); fp32 products would be off by 0.06 rad.
// Within an eighth of a turn, sine and cosine are their Taylor sums.
//
// 8-bit pages have a scale a (page, head), which has to be known before the first code:
// a job is the new tokens of one page of one head, keys and values, whose greatest
// magnitude is taken first.  Scales are powers of two, so that a page whose scale grows
// later is rescaled without loss but for codes that leave the normal range.
//
// Jobs are a warp's where they are small (a step of T <= 16 tokens) and a block's where
// they are whole pages; the queries, which belong to no page, are blocks of their own.
#include <cuda_fp8.h>

#include "layer_common.cuh"
#include "serve_params.h"

namespace lar {

namespace {

constexpr int kThreads = 256;
constexpr int kELo = -64, kEHi = 64;   // exponents of a scale

// f / 2 pi in units of 2^-64 turns, whole turns dropped: f = m 2^e, m of 24 bits, times
// the first 128 bits of 1 / 2 pi (good for f up to 2^60)
__device__ __forceinline__ unsigned long long turn_step(float f) {
    const unsigned long long hi = 0x28BE60DB9391054Aull, lo = 0x7F09D5F47D4D3770ull;
    const unsigned bits = __float_as_uint(f), be = (bits >> 23) & 255u;
    const unsigned long long m = be ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
    const int right = 64 - (static_cast<int>(be ? be : 1u) - 150);   // of the 152-bit product
    const unsigned long long w0 = m * lo, c = __umul64hi(m, lo), h = m * hi;
    const unsigned long long w1 = h + c, w2 = __umul64hi(m, hi) + (w1 < h ? 1u : 0u);
    unsigned long long r;
    if (right >= 128) r = right < 192 ? w2 >> (right - 128) : 0ull;
    else if (right >= 64) r = right == 64 ? w1 : (w1 >> (right - 64)) | (w2 << (128 - right));
    else r = right <= 0 ? w0 << min(63, -right) : (w0 >> right) | (w1 << (64 - right));
    return static_cast<int>(bits) < 0 ? 0ull - r : r;
}

// cosine and sine of `turn` 2^-64 turns
__device__ __forceinline__ void cos_sin(unsigned long long turn, float& c, float& s) {
    const unsigned a = static_cast<unsigned>((turn + (1ull << 31)) >> 32);
    const unsigned q = (a + (1u << 29)) >> 30;                       // quarter turns
    const float z = static_cast<float>(static_cast<int>(a - (q << 30))) * 1.4629180792671596e-9f;   // 2 pi 2^-32
    const float z2 = z * z;
    const float sz = fmaf(z * z2, fmaf(z2, fmaf(z2, fmaf(z2, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), z);
    const float cz = fmaf(z2, fmaf(z2, fmaf(z2, fmaf(z2, fmaf(z2, -1.f / 3628800, 1.f / 40320), -1.f / 720), 1.f / 24), -0.5f), 1.f);
    const float u = q & 1 ? sz : cz, v = q & 1 ? cz : sz;
    c = (q == 1 || q == 2) ? -u : u;
    s = q >= 2 ? -v : v;
}

// The least power of two with m <= 448 of it, within the range: 2^exponent
__device__ __forceinline__ int scale_exponent(float m) {
    if (!(m > 0.f)) return kELo;
    int e;
    const float f = frexpf(m, &e);   // m = f 2^e, f in [0.5, 1); 448 = 0.875 2^9
    return max(kELo, min(kEHi, f <= 0.875f ? e - 9 : e - 8));
}

__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<unsigned>(e + 127) << 23); }

// four values as codes; NaN where a value is not finite
__device__ __forceinline__ unsigned codes4(const float* x, float inv) {
    unsigned r = 0;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const float a = x[i], b = x[i + 1];
        unsigned short h;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(fabsf(b) < INFINITY ? b * inv : NAN), "f"(fabsf(a) < INFINITY ? a * inv : NAN));
        r |= static_cast<unsigned>(h) << (i * 8);
    }
    return r;
}

// A unit is 16 dimensions of a row.  Fast rows take them in two vectors of 8, the members
// of 8 pairs where they are rotated; other rows dimensions 16 u to 16 u + 15.
struct Unit {
    int d0, d1;      // the vectors' first dimensions
    int pair;        // first pair, or -1: copied
};

template <bool FAST>
__device__ __forceinline__ Unit unit_of(const AppendParams& p, int u, bool rotated) {
    if (!FAST || !rotated || u * 16 >= p.rot) return {u * 16, u * 16 + 8, -1};
    return p.interleaved ? Unit{u * 16, u * 16 + 8, u * 8} : Unit{u * 8, p.rot / 2 + u * 8, u * 8};
}

struct Angles {
    float c[8], s[8];
};

template <bool FAST>
__device__ __forceinline__ void angles_of(const AppendParams& p, const unsigned long long* steps, const Unit& un, int place, Angles& a) {
    if constexpr (FAST) {
        if (un.pair < 0) return;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            cos_sin(steps[un.pair + i] * static_cast<unsigned long long>(place), a.c[i], a.s[i]);
            a.c[i] *= p.rope_scale;
            a.s[i] *= p.rope_scale;
        }
    }
}

// The unit's values, rotated: x[0..8) at d0, x[8..16) at d1
template <bool FAST>
__device__ __forceinline__ void load_unit(const AppendParams& p, const unsigned long long* steps, const void* base, int64_t row, int64_t ds,
                                          int dt, const Unit& un, const Angles& a, int place, bool rotated, float* x) {
    if constexpr (FAST) {
        ld8<true>(base, row + un.d0, dt, x);
        ld8<true>(base, row + un.d1, dt, x + 8);
        if (un.pair < 0) return;
        if (p.interleaved) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float u = x[2 * i], v = x[2 * i + 1];
                x[2 * i] = fmaf(u, a.c[i], -(v * a.s[i]));
                x[2 * i + 1] = fmaf(v, a.c[i], u * a.s[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float u = x[i], v = x[i + 8];
                x[i] = fmaf(u, a.c[i], -(v * a.s[i]));
                x[i + 8] = fmaf(v, a.c[i], u * a.s[i]);
            }
        }
    } else {
        for (int i = 0; i < 16; ++i) {
            const int d = un.d0 + i;
            float v = ld_in(base, row + d * ds, dt);
            if (rotated && d < p.rot) {
                const int half = p.rot / 2, pair = p.interleaved ? d / 2 : d % half;
                const bool first = p.interleaved ? d % 2 == 0 : d < half;
                const float w = ld_in(base, row + (p.interleaved ? d ^ 1 : first ? d + half : d - half) * ds, dt);
                float c, s;
                cos_sin(steps[pair] * static_cast<unsigned long long>(place), c, s);
                c *= p.rope_scale;
                s *= p.rope_scale;
                v = first ? fmaf(v, c, -(w * s)) : fmaf(v, c, w * s);
            }
            x[i] = v;
        }
    }
}

// The sequence's length before the call; -1: no sequence
__device__ __forceinline__ int64_t length_of(const AppendParams& p, int n) {
    const int64_t len = ld_idx(p.c.lens, n * p.c.len_s, p.c.len_dt);
    return len < 0 ? -1 : min(len, int64_t{1} << 30);
}

__device__ __forceinline__ bool span(const AppendParams& p, int n, int* begin, int* len, int32_t* bits) {
    if (!p.cu) {
        *begin = 0;
        *len = p.T;
        return true;
    }
    const int64_t a = ld_idx(p.cu, n * p.cu_s, p.cu_dt), e = ld_idx(p.cu, (n + 1) * p.cu_s, p.cu_dt);
    const bool ok = a >= 0 && a <= e && e <= p.ntok;
    if (!ok) *bits |= LAR_DEVERR_SEQLEN;
    *begin = ok ? static_cast<int>(a) : 0;
    *len = ok ? static_cast<int>(e - a) : 0;
    return ok;
}

// The last sequence n with key(n) <= want, keys ascending; 0 if there is none
template <typename F>
__device__ __forceinline__ int last_at_most(int n, int64_t want, F key) {
    int lo = 0, hi = n;   // key(lo) <= want < key(hi)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (key(mid) <= want) lo = mid;
        else hi = mid;
    }
    return lo;
}

// One job: the tokens of a call that fall into page `j` (of the touched ones) of sequence
// n, for head h, by THR threads of which this is `me`.
template <bool F8, bool FAST, int THR>
__device__ __forceinline__ void kv_job(const AppendParams& p, const unsigned long long* steps, unsigned* top_s, int n, int j, int h, int me,
                                       int32_t* bits) {
    int begin, len;
    span(p, n, &begin, &len, bits);
    const int64_t start = length_of(p, n);
    if (start < 0 || len == 0) return;
    const int page = p.c.page;
    const int64_t pg = start / page + j;                                // page of the sequence
    const int64_t lo = max(start, pg * page), hi = min(start + len, (pg + 1) * page);
    if (lo >= hi) return;
    if (pg >= p.c.M) {
        *bits |= LAR_DEVERR_SEQLEN;
        return;
    }
    const int64_t id = ld_idx(p.c.table, n * p.c.tab_s[0] + pg * p.c.tab_s[1], p.c.tab_dt);
    if (id >= p.c.P) *bits |= LAR_DEVERR_PAGE;
    if (id < 0 || id >= p.c.P) return;
    const int first = static_cast<int>(lo - pg * page), cnt = static_cast<int>(hi - lo), t0 = static_cast<int>(lo - start);
    const int UN = p.c.D / 16, tasks = cnt * UN;
    const int64_t kq = p.cu ? 0 : n * p.ks[0], vq = p.cu ? 0 : n * p.vs[0];
    float kx[16], vx[16];
    float ktop = 0.f, vtop = 0.f;
    auto take = [&](int i) {
        const int t = i / UN, u = i % UN;
        const Unit ku = unit_of<FAST>(p, u, true), vu = {u * 16, u * 16 + 8, -1};
        const int tok = begin + t0 + t, place = static_cast<int>(lo) + t;
        Angles a;
        angles_of<FAST>(p, steps, ku, place, a);
        load_unit<FAST>(p, steps, p.k, kq + tok * p.ks[1] + h * p.ks[2], p.ks[3], p.k_dt, ku, a, place, true, kx);
        load_unit<FAST>(p, steps, p.v, vq + tok * p.vs[1] + h * p.vs[2], p.vs[3], p.v_dt, vu, a, place, false, vx);
    };
    float kinv = 1.f, vinv = 1.f;
    if constexpr (F8) {
        for (int i = me; i < tasks; i += THR) {
            take(i);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                if (fabsf(kx[e]) < INFINITY) ktop = fmaxf(ktop, fabsf(kx[e]));
                if (fabsf(vx[e]) < INFINITY) vtop = fmaxf(vtop, fabsf(vx[e]));
            }
        }
        unsigned kt = __reduce_max_sync(0xffffffffu, __float_as_uint(ktop)), vt = __reduce_max_sync(0xffffffffu, __float_as_uint(vtop));
        if constexpr (THR > 32) {
            if (me < 2) top_s[me] = 0u;
            __syncthreads();
            if (me % 32 == 0) {
                atomicMax(&top_s[0], kt);
                atomicMax(&top_s[1], vt);
            }
            __syncthreads();
            kt = top_s[0];
            vt = top_s[1];
        }
        float* kscale = p.c.k_scale + id * p.c.kss[0] + h * p.c.kss[1];
        float* vscale = p.c.v_scale + id * p.c.vss[0] + h * p.c.vss[1];
        const float kold = first ? *kscale : 0.f, vold = first ? *vscale : 0.f;
        const float kne = pow2(scale_exponent(__uint_as_float(kt))), vne = pow2(scale_exponent(__uint_as_float(vt)));
        const float know = kold > kne ? kold : kne, vnow = vold > vne ? vold : vne;
        kinv = 1.f / know;
        vinv = 1.f / vnow;
        // what stands before them, at the new scale
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const float was = w ? vold : kold, now = w ? vnow : know;
            if (first == 0 || !(now > was)) continue;
            const float f = was / now;
            unsigned char* pgp = static_cast<unsigned char*>(w ? p.c.v : p.c.k) + id * (w ? p.c.vs[0] : p.c.ks[0]) + h * (w ? p.c.vs[2] : p.c.ks[2]);
            for (int i = me; i < first * UN; i += THR) {
                uint4* at = reinterpret_cast<uint4*>(pgp + i / UN * (w ? p.c.vs[1] : p.c.ks[1]) + i % UN * 16);
                const uint4 old = *at;
                const unsigned in[4] = {old.x, old.y, old.z, old.w};
                unsigned out[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float x[4];
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        __nv_fp8_e4m3 c;
                        c.__x = static_cast<__nv_fp8_storage_t>(in[e] >> (8 * b));
                        x[b] = static_cast<float>(c);
                    }
                    out[e] = codes4(x, f);
                }
                *at = make_uint4(out[0], out[1], out[2], out[3]);
            }
        }
        if constexpr (THR > 32) __syncthreads();
        else __syncwarp();
        if (me == 0) {
            *kscale = know;
            *vscale = vnow;
        }
    }
    const bool kept = F8 && tasks <= THR;   // still in registers
    for (int i = me; i < tasks; i += THR) {
        if (!kept) take(i);
        const int t = i / UN, u = i % UN;
        const Unit ku = unit_of<FAST>(p, u, true);
        const int64_t krow = id * p.c.ks[0] + (first + t) * p.c.ks[1] + h * p.c.ks[2];
        const int64_t vrow = id * p.c.vs[0] + (first + t) * p.c.vs[1] + h * p.c.vs[2];
        if constexpr (F8) {
            unsigned char *kc = static_cast<unsigned char*>(p.c.k) + krow, *vc = static_cast<unsigned char*>(p.c.v) + vrow;
            *reinterpret_cast<uint2*>(kc + ku.d0) = make_uint2(codes4(kx, kinv), codes4(kx + 4, kinv));
            *reinterpret_cast<uint2*>(kc + ku.d1) = make_uint2(codes4(kx + 8, kinv), codes4(kx + 12, kinv));
            *reinterpret_cast<uint4*>(vc + u * 16) = make_uint4(codes4(vx, vinv), codes4(vx + 4, vinv), codes4(vx + 8, vinv), codes4(vx + 12, vinv));
        } else {
            st8(p.c.k, krow + ku.d0, LAR_BF16, kx);
            st8(p.c.k, krow + ku.d1, LAR_BF16, kx + 8);
            st8(p.c.v, vrow + u * 16, LAR_BF16, vx);
            st8(p.c.v, vrow + u * 16 + 8, LAR_BF16, vx + 8);
        }
    }
}

// Rotated queries: a thread a (token, unit), for `hpt` heads
template <bool FAST>
__device__ __forceinline__ void q_task(const AppendParams& p, const unsigned long long* steps, int64_t task, int hpt, int32_t* bits) {
    const int UN = p.c.D / 16, chunks = (p.Hq + hpt - 1) / hpt;
    const int u = static_cast<int>(task % UN), ch = static_cast<int>(task / UN % chunks);
    const int64_t tok = task / UN / chunks;
    int n, t;
    int64_t qrow, orow;
    if (p.cu) {
        n = last_at_most(p.n, tok, [&](int i) { return ld_idx(p.cu, i * p.cu_s, p.cu_dt); });
        int begin, len;
        span(p, n, &begin, &len, bits);
        if (tok < begin || tok >= begin + len) return;
        t = static_cast<int>(tok) - begin;
        qrow = tok * p.qs[1];
        orow = tok * p.os[1];
    } else {
        n = static_cast<int>(tok / p.T);
        t = static_cast<int>(tok % p.T);
        qrow = n * p.qs[0] + t * p.qs[1];
        orow = n * p.os[0] + t * p.os[1];
    }
    const int64_t start = length_of(p, n);
    if (start < 0) return;
    const int place = static_cast<int>(start) + t;
    const Unit un = unit_of<FAST>(p, u, true);
    Angles a;
    angles_of<FAST>(p, steps, un, place, a);
    const int h1 = min(p.Hq, (ch + 1) * hpt);
    for (int h = ch * hpt; h < h1; ++h) {
        float x[16];
        load_unit<FAST>(p, steps, p.q, qrow + h * p.qs[2], p.qs[3], p.q_dt, un, a, place, true, x);
        const int64_t row = orow + h * p.os[2];
        if constexpr (FAST) {
            st8(p.q_out, row + un.d0, p.o_dt, x);
            st8(p.q_out, row + un.d1, p.o_dt, x + 8);
        } else {
            for (int i = 0; i < 16; ++i) st_out(p.q_out, row + (un.d0 + i) * p.os[3], p.o_dt, x[i]);
        }
    }
}

// Blocks [0, kv_blocks) are jobs, the others queries
template <bool F8, bool FAST, int THR>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendParams p, int kv_blocks, int pages_of, int hpt,
                                                          int64_t q_tasks) {
    __shared__ unsigned long long steps[128];
    __shared__ unsigned top_s[2];
    const int tid = threadIdx.x;
    stream_order();
    if (tid < p.rot / 2) steps[tid] = turn_step(__ldg(p.inv_freq + tid * p.if_s));
    __syncthreads();
    int32_t bits = 0;
    if (static_cast<int>(blockIdx.x) >= kv_blocks) {
        const int64_t task = static_cast<int64_t>(blockIdx.x - kv_blocks) * kThreads + tid;
        if (task < q_tasks) q_task<FAST>(p, steps, task, hpt, &bits);
    } else if (THR == 32) {   // a warp a job: (sequence, touched page, head)
        const int64_t job = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + tid / 32;
        const int h = static_cast<int>(job % p.c.H), j = static_cast<int>(job / p.c.H % pages_of);
        const int64_t n = job / p.c.H / pages_of;
        if (n < p.n) kv_job<F8, FAST, 32>(p, steps, nullptr, static_cast<int>(n), j, h, tid % 32, &bits);
    } else {                  // a block a job: sequence n's pages have numbers from cu[n] / page + 2 n on
        const int h = blockIdx.x % p.c.H;
        const int64_t unit = blockIdx.x / p.c.H;
        auto key = [&](int i) { return ld_idx(p.cu, i * p.cu_s, p.cu_dt) / p.c.page + 2 * static_cast<int64_t>(i); };
        const int n = last_at_most(p.n, unit, key);
        const int64_t j = unit - key(n);
        if (j >= 0 && j < (1 << 30)) kv_job<F8, FAST, THR>(p, steps, top_s, n, static_cast<int>(j), h, tid, &bits);
    }
    flag_err(p.dev_err, bits);
}

template <bool F8, bool FAST>
lar_status launch(const AppendParams& p, cudaStream_t stream) {
    const int64_t tokens = p.cu ? p.ntok : static_cast<int64_t>(p.n) * p.T;
    int64_t q_tasks = 0;
    int hpt = 1;
    if (p.q) {
        // heads share their angles where there are threads enough without
        while (hpt < 8 && hpt < p.Hq && tokens * (p.c.D / 16) * p.Hq / (2 * hpt) >= 152 * 2048) hpt *= 2;
        q_tasks = tokens * (p.c.D / 16) * ((p.Hq + hpt - 1) / hpt);
    }
    const int64_t q_blocks = (q_tasks + kThreads - 1) / kThreads;
    int64_t kv_blocks;
    int pages_of = 0;
    if (p.cu) {
        kv_blocks = (p.ntok / p.c.page + 2 * static_cast<int64_t>(p.n)) * p.c.H;
    } else {
        pages_of = p.T == 1 ? 1 : 2;
        kv_blocks = (static_cast<int64_t>(p.n) * pages_of * p.c.H + kThreads / 32 - 1) / (kThreads / 32);
    }
    if (kv_blocks + q_blocks > (int64_t{1} << 31) - 1) return LAR_ERR_SHAPE;
    const dim3 grid(static_cast<unsigned>(kv_blocks + q_blocks));
    return p.cu ? launch_ordered(append_kernel<F8, FAST, kThreads>, grid, kThreads, 0, 1, stream, p, static_cast<int>(kv_blocks), pages_of, hpt, q_tasks)
                : launch_ordered(append_kernel<F8, FAST, 32>, grid, kThreads, 0, 1, stream, p, static_cast<int>(kv_blocks), pages_of, hpt, q_tasks);
}

}  // namespace

lar_status launch_append(const AppendParams& p, void* stream) {
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool fast = p.vec && p.rot % 16 == 0;
    if (p.c.e4m3) return fast ? launch<true, true>(p, s) : launch<true, false>(p, s);
    return fast ? launch<false, true>(p, s) : launch<false, false>(p, s);
}

}  // namespace lar

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
// Steps of T <= 16 tokens: a warp has a job, and the queries are blocks of their own.
// Prompts: a block has the new tokens of a page for some heads and their queries, a thread
// a token's 16 dimensions, whose angles it works out once for all of them; the greatest
// magnitudes come first, and the second look at keys and values finds them in L1 or L2.
#include <cuda_fp8.h>

#include "layer_common.cuh"
#include "serve_params.h"

namespace lar {

namespace {

#ifndef LAR_APPEND_MIN
#define LAR_APPEND_MIN 2
#endif
#ifndef LAR_APPEND_THREADS
#define LAR_APPEND_THREADS 256
#endif
constexpr int kThreads = LAR_APPEND_THREADS;
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

__device__ __forceinline__ void turn(const AppendParams& p, const Unit& un, const Angles& a, float* x) {
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
}

// A unit of a bf16 row as it lies: asked for now, looked at later
struct Raw {
    uint4 a, b;
    __device__ __forceinline__ void load(const void* base, int64_t row, const Unit& un) {
        const unsigned short* p = static_cast<const unsigned short*>(base) + row;
        a = __ldg(reinterpret_cast<const uint4*>(p + un.d0));
        b = __ldg(reinterpret_cast<const uint4*>(p + un.d1));
    }
    __device__ __forceinline__ void widen(float* x) const {
        unpack8(a, x);
        unpack8(b, x + 8);
    }
};

// The unit's values, rotated: x[0..8) at d0, x[8..16) at d1
template <bool FAST>
__device__ __forceinline__ void load_unit(const AppendParams& p, const unsigned long long* steps, const void* base, int64_t row, int64_t ds,
                                          int dt, const Unit& un, const Angles& a, int place, bool rotated, float* x) {
    if constexpr (FAST) {
        ld8<true>(base, row + un.d0, dt, x);
        ld8<true>(base, row + un.d1, dt, x + 8);
        turn(p, un, a, x);
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

template <bool FAST>
__device__ __forceinline__ void put_query(const AppendParams& p, int64_t row, const Unit& un, const float* x) {
    if constexpr (FAST) {
        st8(p.q_out, row + un.d0, p.o_dt, x);
        st8(p.q_out, row + un.d1, p.o_dt, x + 8);
    } else {
        for (int i = 0; i < 16; ++i) st_out(p.q_out, row + (un.d0 + i) * p.os[3], p.o_dt, x[i]);
    }
}

// The new tokens of a call that fall into page `j` (of the touched ones) of sequence n
struct Job {
    int tok, cnt;        // first token's place in the arrays (of a sequence where T is fixed), their number
    int place;           // of the first
    int first;           // its row in the page
    int64_t id;          // the page; -1: none
};

// false: no tokens there
__device__ __forceinline__ bool job_of(const AppendParams& p, int n, int j, Job& job, int32_t* bits) {
    int begin, len;
    span(p, n, &begin, &len, bits);
    const int64_t start = length_of(p, n);
    if (start < 0 || len == 0) return false;
    const int page = p.c.page;
    const int64_t pg = start / page + j;                                // page of the sequence
    const int64_t lo = max(start, pg * page), hi = min(start + len, (pg + 1) * page);
    if (lo >= hi) return false;
    job.tok = begin + static_cast<int>(lo - start);
    job.cnt = static_cast<int>(hi - lo);
    job.place = static_cast<int>(lo);
    job.first = static_cast<int>(lo - pg * page);
    job.id = -1;
    if (pg >= p.c.M) {
        *bits |= LAR_DEVERR_SEQLEN;
    } else {
        job.id = ld_idx(p.c.table, n * p.c.tab_s[0] + pg * p.c.tab_s[1], p.c.tab_dt);
        if (job.id >= p.c.P) {
            *bits |= LAR_DEVERR_PAGE;
            job.id = -1;
        }
    }
    return true;
}

__device__ __forceinline__ void raise(float& top, const float* x) {
#pragma unroll
    for (int e = 0; e < 16; ++e)
        if (fabsf(x[e]) < INFINITY) top = fmaxf(top, fabsf(x[e]));
}

// The scale of a (page, head) whose new values have the greatest magnitude `top`: no less
// than that of `first` tokens that stand before them, whose codes follow it.  Written by
// thread 0 of the THR threads that share the job; returned inverted.
template <int THR>
__device__ __forceinline__ float rescale(const AppendParams& p, bool values, const Job& job, int h, float top, int me) {
    float* at = values ? p.c.v_scale + job.id * p.c.vss[0] + h * p.c.vss[1] : p.c.k_scale + job.id * p.c.kss[0] + h * p.c.kss[1];
    const float was = job.first ? *at : 0.f, need = pow2(scale_exponent(top)), now = was > need ? was : need;
    if (job.first && now > was) {
        const float f = was / now;
        unsigned char* pg = static_cast<unsigned char*>(values ? p.c.v : p.c.k) + job.id * (values ? p.c.vs[0] : p.c.ks[0]) + h * (values ? p.c.vs[2] : p.c.ks[2]);
        const int64_t step = values ? p.c.vs[1] : p.c.ks[1];
        const int UN = p.c.D / 16;
        for (int i = me; i < job.first * UN; i += THR) {
            uint4* to = reinterpret_cast<uint4*>(pg + i / UN * step + i % UN * 16);
            const uint4 old = *to;
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
            *to = make_uint4(out[0], out[1], out[2], out[3]);
        }
    }
    if (THR > 32) __syncthreads();   // all have read the old scale
    else __syncwarp();
    if (me == 0) *at = now;
    return 1.f / now;
}

template <bool F8>
__device__ __forceinline__ void put_unit(const AppendParams& p, bool values, const Job& job, int h, int t, const Unit& un, const float* x, float inv) {
    const int64_t row = values ? job.id * p.c.vs[0] + (job.first + t) * p.c.vs[1] + h * p.c.vs[2]
                               : job.id * p.c.ks[0] + (job.first + t) * p.c.ks[1] + h * p.c.ks[2];
    void* base = values ? p.c.v : p.c.k;
    if constexpr (F8) {
        unsigned char* to = static_cast<unsigned char*>(base) + row;
        const uint2 a = make_uint2(codes4(x, inv), codes4(x + 4, inv)), b = make_uint2(codes4(x + 8, inv), codes4(x + 12, inv));
        if (un.d1 == un.d0 + 8) {
            *reinterpret_cast<uint4*>(to + un.d0) = make_uint4(a.x, a.y, b.x, b.y);
        } else {
            *reinterpret_cast<uint2*>(to + un.d0) = a;
            *reinterpret_cast<uint2*>(to + un.d1) = b;
        }
    } else {
        st8(base, row + un.d0, LAR_BF16, x);
        st8(base, row + un.d1, LAR_BF16, x + 8);
    }
}

// A step's job for one head, by a warp
template <bool F8, bool FAST>
__device__ __forceinline__ void step_job(const AppendParams& p, const unsigned long long* steps, int n, int j, int h, int me, int32_t* bits) {
    Job job;
    if (!job_of(p, n, j, job, bits) || job.id < 0) return;
    const int UN = p.c.D / 16, tasks = job.cnt * UN;
    float kx[16], vx[16];
    auto take = [&](int i) {
        const int t = i / UN, u = i % UN;
        const Unit ku = unit_of<FAST>(p, u, true), vu = {u * 16, u * 16 + 8, -1};
        Angles a;
        angles_of<FAST>(p, steps, ku, job.place + t, a);
        load_unit<FAST>(p, steps, p.k, n * p.ks[0] + (job.tok + t) * p.ks[1] + h * p.ks[2], p.ks[3], p.k_dt, ku, a, job.place + t, true, kx);
        load_unit<FAST>(p, steps, p.v, n * p.vs[0] + (job.tok + t) * p.vs[1] + h * p.vs[2], p.vs[3], p.v_dt, vu, a, job.place + t, false, vx);
    };
    float kinv = 1.f, vinv = 1.f;
    if constexpr (F8) {
        float ktop = 0.f, vtop = 0.f;
        for (int i = me; i < tasks; i += 32) {
            take(i);
            raise(ktop, kx);
            raise(vtop, vx);
        }
        ktop = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(ktop)));
        vtop = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(vtop)));
        kinv = rescale<32>(p, false, job, h, ktop, me);
        vinv = rescale<32>(p, true, job, h, vtop, me);
    }
    const bool kept = F8 && tasks <= 32;   // still in registers
    for (int i = me; i < tasks; i += 32) {
        if (!kept) take(i);
        put_unit<F8>(p, false, job, h, i / UN, unit_of<FAST>(p, i % UN, true), kx, kinv);
        put_unit<F8>(p, true, job, h, i / UN, {i % UN * 16, i % UN * 16 + 8, -1}, vx, vinv);
    }
}

// A prompt's job for heads [h0, h1) and their queries, by a block
constexpr int kJobHeads = 4;   // at most
constexpr int kAtOnce = 4;     // queries' rows that are asked for together

template <bool F8, bool FAST, bool BF>
__device__ __forceinline__ void prompt_job(const AppendParams& p, const unsigned long long* steps, unsigned* top_s, int n, int j, int h0, int h1, int me,
                                           int32_t* bits) {
    Job job;
    if (!job_of(p, n, j, job, bits)) return;
    const int UN = p.c.D / 16, tasks = job.cnt * UN, G = p.q ? p.Hq / p.c.H : 0;
    float inv[2 * kJobHeads];
#pragma unroll
    for (int e = 0; e < 2 * kJobHeads; ++e) inv[e] = 1.f;
    Angles a;
    float x[16];
    // f(head of the job, whether it is the values') with the unit's keys, rotated, and values in x
    auto rows_of = [&](int t, int u, auto f) {
        const Unit ku = unit_of<FAST>(p, u, true), vu = {u * 16, u * 16 + 8, -1};
        const int64_t krow = (job.tok + t) * p.ks[1], vrow = (job.tok + t) * p.vs[1];
        if constexpr (BF) {
#pragma unroll
            for (int e = 0; e < kJobHeads; e += 2) {
                Raw k[2], v[2];
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (h0 + e + i < h1) {
                        k[i].load(p.k, krow + (h0 + e + i) * p.ks[2], ku);
                        v[i].load(p.v, vrow + (h0 + e + i) * p.vs[2], vu);
                    }
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (h0 + e + i < h1) {
                        k[i].widen(x);
                        turn(p, ku, a, x);
                        f(e + i, false);
                        v[i].widen(x);
                        f(e + i, true);
                    }
            }
        } else {
#pragma unroll
            for (int e = 0; e < kJobHeads; ++e)
                if (h0 + e < h1) {
                    load_unit<FAST>(p, steps, p.k, krow + (h0 + e) * p.ks[2], p.ks[3], p.k_dt, ku, a, job.place + t, true, x);
                    f(e, false);
                    load_unit<FAST>(p, steps, p.v, vrow + (h0 + e) * p.vs[2], p.vs[3], p.v_dt, vu, a, job.place + t, false, x);
                    f(e, true);
                }
        }
    };
    const bool one = tasks <= kThreads;   // each thread has one token's unit, and its angles
    if (one && me < tasks) angles_of<FAST>(p, steps, unit_of<FAST>(p, me % UN, true), job.place + me / UN, a);
    if (F8 && job.id >= 0) {
        float top[2 * kJobHeads];
#pragma unroll
        for (int e = 0; e < 2 * kJobHeads; ++e) top[e] = 0.f;
        for (int i = me; i < tasks; i += kThreads) {
            const int t = i / UN, u = i % UN;
            if (!one) angles_of<FAST>(p, steps, unit_of<FAST>(p, u, true), job.place + t, a);
            rows_of(t, u, [&](int e, bool values) { raise(top[2 * e + values], x); });
        }
        if (me < 2 * kJobHeads) top_s[me] = 0u;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 2 * kJobHeads; ++e) {
            const unsigned v = __reduce_max_sync(0xffffffffu, __float_as_uint(top[e]));
            if (me % 32 == 0 && v) atomicMax(&top_s[e], v);
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kJobHeads; ++e)
            if (h0 + e < h1) {
                inv[2 * e] = rescale<kThreads>(p, false, job, h0 + e, __uint_as_float(top_s[2 * e]), me);
                inv[2 * e + 1] = rescale<kThreads>(p, true, job, h0 + e, __uint_as_float(top_s[2 * e + 1]), me);
            }
    }
    for (int i = me; i < tasks; i += kThreads) {
        const int t = i / UN, u = i % UN;
        const Unit un = unit_of<FAST>(p, u, true);
        if (!one) angles_of<FAST>(p, steps, un, job.place + t, a);
        if (job.id >= 0) {
            rows_of(t, u, [&](int e, bool values) {
                put_unit<F8>(p, values, job, h0 + e, t, values ? Unit{u * 16, u * 16 + 8, -1} : un, x, inv[2 * e + values]);
            });
        }
        const int64_t qrow = (job.tok + t) * p.qs[1], orow = (job.tok + t) * p.os[1];
        if constexpr (BF) {
            for (int h = h0 * G; h < h1 * G; h += kAtOnce) {
                Raw r[kAtOnce];
#pragma unroll
                for (int e = 0; e < kAtOnce; ++e)
                    if (h + e < h1 * G) r[e].load(p.q, qrow + (h + e) * p.qs[2], un);
#pragma unroll
                for (int e = 0; e < kAtOnce; ++e)
                    if (h + e < h1 * G) {
                        r[e].widen(x);
                        turn(p, un, a, x);
                        put_query<FAST>(p, orow + (h + e) * p.os[2], un, x);
                    }
            }
        } else {
            for (int h = h0 * G; h < h1 * G; ++h) {
                load_unit<FAST>(p, steps, p.q, qrow + h * p.qs[2], p.qs[3], p.q_dt, un, a, job.place + t, true, x);
                put_query<FAST>(p, orow + h * p.os[2], un, x);
            }
        }
    }
}

// A step's rotated queries: a thread a (token, unit), for `hpt` heads
template <bool FAST>
__device__ __forceinline__ void q_task(const AppendParams& p, const unsigned long long* steps, int64_t task, int hpt) {
    const int UN = p.c.D / 16, chunks = (p.Hq + hpt - 1) / hpt;
    const int u = static_cast<int>(task % UN), ch = static_cast<int>(task / UN % chunks);
    const int64_t tok = task / UN / chunks;
    const int n = static_cast<int>(tok / p.T), t = static_cast<int>(tok % p.T);
    const int64_t start = length_of(p, n);
    if (start < 0) return;
    const int place = static_cast<int>(start) + t;
    const Unit un = unit_of<FAST>(p, u, true);
    Angles a;
    angles_of<FAST>(p, steps, un, place, a);
    const int h1 = min(p.Hq, (ch + 1) * hpt);
    for (int h = ch * hpt; h < h1; ++h) {
        float x[16];
        load_unit<FAST>(p, steps, p.q, n * p.qs[0] + t * p.qs[1] + h * p.qs[2], p.qs[3], p.q_dt, un, a, place, true, x);
        put_query<FAST>(p, n * p.os[0] + t * p.os[1] + h * p.os[2], un, x);
    }
}

__device__ __forceinline__ void load_steps(const AppendParams& p, unsigned long long* steps) {
    if (threadIdx.x < p.rot / 2) steps[threadIdx.x] = turn_step(__ldg(p.inv_freq + threadIdx.x * p.if_s));
    __syncthreads();
}

// Blocks [0, kv_blocks): a warp a job (sequence, touched page, head); the others: queries
template <bool F8, bool FAST>
__global__ void __launch_bounds__(kThreads) append_step(const __grid_constant__ AppendParams p, int kv_blocks, int pages_of, int hpt, int64_t q_tasks) {
    __shared__ unsigned long long steps[128];
    const int tid = threadIdx.x;
    stream_order();
    load_steps(p, steps);
    int32_t bits = 0;
    if (static_cast<int>(blockIdx.x) >= kv_blocks) {
        const int64_t task = static_cast<int64_t>(blockIdx.x - kv_blocks) * kThreads + tid;
        if (task < q_tasks) q_task<FAST>(p, steps, task, hpt);
    } else {
        const int64_t job = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + tid / 32;
        const int h = static_cast<int>(job % p.c.H), j = static_cast<int>(job / p.c.H % pages_of);
        const int64_t n = job / p.c.H / pages_of;
        if (n < p.n) step_job<F8, FAST>(p, steps, static_cast<int>(n), j, h, tid % 32, &bits);
    }
    flag_err(p.dev_err, bits);
}

// A block a job: sequence n's pages have numbers from cu[n] / page + 2 n on
template <bool F8, bool FAST, bool BF>
__global__ void __launch_bounds__(kThreads, LAR_APPEND_MIN) append_prompt(const __grid_constant__ AppendParams p, int groups, int heads) {
    __shared__ unsigned long long steps[128];
    __shared__ unsigned top_s[2 * kJobHeads];
    stream_order();
    load_steps(p, steps);
    int32_t bits = 0;
    const int h0 = static_cast<int>(blockIdx.x % groups) * heads;
    const int64_t unit = blockIdx.x / groups;
    auto key = [&](int i) { return ld_idx(p.cu, i * p.cu_s, p.cu_dt) / p.c.page + 2 * static_cast<int64_t>(i); };
    const int n = last_at_most(p.n, unit, key);
    const int64_t j = unit - key(n);
    if (j >= 0 && j < (1 << 30)) prompt_job<F8, FAST, BF>(p, steps, top_s, n, static_cast<int>(j), h0, min(p.c.H, h0 + heads), threadIdx.x, &bits);
    flag_err(p.dev_err, bits);
}

template <bool F8, bool FAST>
lar_status launch(const AppendParams& p, cudaStream_t stream) {
    const int64_t limit = (int64_t{1} << 31) - 1;
    if (p.cu) {
        const int64_t pages = p.ntok / p.c.page + 2 * static_cast<int64_t>(p.n);
        // heads share their angles where there are blocks enough without
        int heads = 1;
        while (heads < kJobHeads && 2 * heads <= p.c.H && pages * p.c.H >= 152 * 8 * heads) heads *= 2;
        const int64_t groups = (p.c.H + heads - 1) / heads;
        if (pages * groups > limit) return LAR_ERR_SHAPE;
        const dim3 grid(static_cast<unsigned>(pages * groups));
        const bool bf = p.k_dt == LAR_BF16 && p.v_dt == LAR_BF16 && (!p.q || p.q_dt == LAR_BF16);
        if constexpr (FAST) {
            if (bf) return launch_ordered(append_prompt<F8, true, true>, grid, kThreads, 0, 1, stream, p, static_cast<int>(groups), heads);
        }
        return launch_ordered(append_prompt<F8, FAST, false>, grid, kThreads, 0, 1, stream, p, static_cast<int>(groups), heads);
    }
    const int64_t tokens = static_cast<int64_t>(p.n) * p.T;
    int64_t q_tasks = 0;
    int hpt = 1;
    if (p.q) {
        while (hpt < 8 && hpt < p.Hq && tokens * (p.c.D / 16) * p.Hq / (2 * hpt) >= 152 * 2048) hpt *= 2;
        q_tasks = tokens * (p.c.D / 16) * ((p.Hq + hpt - 1) / hpt);
    }
    const int pages_of = p.T == 1 ? 1 : 2;
    const int64_t kv_blocks = (static_cast<int64_t>(p.n) * pages_of * p.c.H + kThreads / 32 - 1) / (kThreads / 32);
    const int64_t blocks = kv_blocks + (q_tasks + kThreads - 1) / kThreads;
    if (blocks > limit) return LAR_ERR_SHAPE;
    return launch_ordered(append_step<F8, FAST>, dim3(static_cast<unsigned>(blocks)), kThreads, 0, 1, stream, p, static_cast<int>(kv_blocks), pages_of, hpt, q_tasks);
}

}  // namespace

lar_status launch_append(const AppendParams& p, void* stream) {
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool fast = p.vec && p.rot % 16 == 0;
    if (p.c.e4m3) return fast ? launch<true, true>(p, s) : launch<true, false>(p, s);
    return fast ? launch<false, true>(p, s) : launch<false, false>(p, s);
}

}  // namespace lar

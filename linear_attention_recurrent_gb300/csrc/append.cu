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
// Steps of T <= 16 tokens: a warp has a job, and the queries are blocks of their own.  Steps whose
// rows a warp's lanes can hold (T D / 16 up to 64, bf16) ask for them before length and page are known;
// the queries' do in any case.
// Prompts: a block has the new tokens of a page, with their angles in a table, and a warp a
// head (or warps share one where heads are few); after the greatest magnitudes it comes for
// keys and values again, which L2 still has.  The queries are blocks of their own here
// too, a thread a token's unit, whose angles it works out once for several heads.
//
// Bound: bytes for prompts (16384 tokens, 32 + 8 heads of 128, e4m3: 80 us where the copy rate
// admits 54; the keys and values alone 43 of 15, the queries beside them 37 of 40; into bf16 pages 70
// of 59; from fp32 rows, angles worked out for each, 174 of 104), latency for steps (256 tokens 6.6
// us, one 4.2: a launch, frequencies, length, page, old scale; 256 of fp32 8.3).  The table holds
// 4096 angles, 32 KB: pages of 128 tokens, whose angles every thread works out, take 113 us.  Keys
// and values kept in registers instead of asked for again: 88 to 120 (they spill).
#include <cuda_fp8.h>

#include "layer_common.cuh"
#include "serve_params.h"

namespace lar {

int cached_occupancy(const void* kern, int threads, size_t smem, size_t smem_max, int* sms_out);

namespace {

constexpr int kThreads = 256;
constexpr int kAtOnce = 4;   // queries' rows that are asked for together
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

// the same of values that are known to be finite, or NaN
__device__ __forceinline__ unsigned codes4_finite(const float* x, float inv) {
    const f32x2 m = pack2(inv, inv);
    float a, b, c, d;
    unpack2(mul2(pack2(x[0], x[1]), m), a, b);
    unpack2(mul2(pack2(x[2], x[3]), m), c, d);
    unsigned r;
    asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
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
        for (int i = 0; i < 8; i += 2) {   // two pairs at once
            const f32x2 u = pack2(x[i], x[i + 1]), v = pack2(x[i + 8], x[i + 9]);
            const f32x2 c = pack2(a.c[i], a.c[i + 1]), s = pack2(a.s[i], a.s[i + 1]), m = pack2(-a.s[i], -a.s[i + 1]);
            unpack2(fma2(u, c, mul2(v, m)), x[i], x[i + 1]);
            unpack2(fma2(v, c, mul2(u, s)), x[i + 8], x[i + 9]);
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
    // the greatest magnitude's bits (bf16 magnitudes are ordered as whole numbers), NaN apart
    __device__ __forceinline__ unsigned top() const {
        const unsigned m = 0x7fff7fffu;
        unsigned t = __vmaxu2(__vmaxu2(__vmaxu2(a.x & m, a.y & m), __vmaxu2(a.z & m, a.w & m)),
                              __vmaxu2(__vmaxu2(b.x & m, b.y & m), __vmaxu2(b.z & m, b.w & m)));
        return max(t >> 16, t & 0xffffu) << 16;
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
__device__ __forceinline__ bool job_of(const AppendParams& p, int n, int j, int64_t start, Job& job, int32_t* bits) {
    int begin, len;
    span(p, n, &begin, &len, bits);
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
// than that of `first` tokens that stand before them, whose codes follow it, by `count`
// threads of which this is `me`.  The caller stores it once all of them have come here.
__device__ __forceinline__ float rescale(const AppendParams& p, bool values, const Job& job, int h, float top, int me, int count) {
    const float* at = values ? p.c.v_scale + job.id * p.c.vss[0] + h * p.c.vss[1] : p.c.k_scale + job.id * p.c.kss[0] + h * p.c.kss[1];
    const float was = job.first ? *at : 0.f, need = pow2(scale_exponent(top)), now = was > need ? was : need;
    if (job.first && now > was) {
        const float f = was / now;
        unsigned char* pg = static_cast<unsigned char*>(values ? p.c.v : p.c.k) + job.id * (values ? p.c.vs[0] : p.c.ks[0]) + h * (values ? p.c.vs[2] : p.c.ks[2]);
        const int64_t step = values ? p.c.vs[1] : p.c.ks[1];
        const int UN = p.c.D / 16;
        for (int i = me; i < job.first * UN; i += count) {
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
    return now;
}

__device__ __forceinline__ void store_scales(const AppendParams& p, const Job& job, int h, float k, float v) {
    p.c.k_scale[job.id * p.c.kss[0] + h * p.c.kss[1]] = k;
    p.c.v_scale[job.id * p.c.vss[0] + h * p.c.vss[1]] = v;
}

template <bool F8, bool FINITE = false>
__device__ __forceinline__ void put_unit(const AppendParams& p, bool values, const Job& job, int h, int t, const Unit& un, const float* x, float inv) {
    const int64_t row = values ? job.id * p.c.vs[0] + (job.first + t) * p.c.vs[1] + h * p.c.vs[2]
                               : job.id * p.c.ks[0] + (job.first + t) * p.c.ks[1] + h * p.c.ks[2];
    void* base = values ? p.c.v : p.c.k;
    if constexpr (F8) {
        unsigned char* to = static_cast<unsigned char*>(base) + row;
        auto code = [&](const float* v) { return FINITE ? codes4_finite(v, inv) : codes4(v, inv); };
        const uint2 a = make_uint2(code(x), code(x + 4)), b = make_uint2(code(x + 8), code(x + 12));
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

// A step's job for one head, by a warp, where its lanes can hold all of the step's tokens: the
// rows are asked for before the sequence's length and the page are known
constexpr int kStepUnits = 2;   // of a lane

struct StepRows {
    Raw k[kStepUnits], v[kStepUnits];
    int64_t start;   // the sequence's length

    __device__ __forceinline__ void load(const AppendParams& p, int n, int h, int me) {
        const int UN = p.c.D / 16, tasks = p.T * UN;
        start = length_of(p, n);
#pragma unroll
        for (int e = 0; e < kStepUnits; ++e) {
            const int i = me + e * 32, t = i / UN, u = i % UN;
            if (i >= tasks) continue;
            k[e].load(p.k, n * p.ks[0] + t * p.ks[1] + h * p.ks[2], unit_of<true>(p, u, true));
            v[e].load(p.v, n * p.vs[0] + t * p.vs[1] + h * p.vs[2], {u * 16, u * 16 + 8, -1});
        }
    }
};

template <bool F8>
__device__ __forceinline__ void step_job_bf16(const AppendParams& p, const unsigned long long* steps, const StepRows& rows, int n, int j, int h, int me,
                                              int32_t* bits) {
    const int UN = p.c.D / 16, tasks = p.T * UN;
    const Raw (&k)[kStepUnits] = rows.k, (&v)[kStepUnits] = rows.v;
    Job job;
    if (!job_of(p, n, j, rows.start, job, bits) || job.id < 0) return;
    float x[kStepUnits][16];
    float ktop = 0.f, vtop = 0.f;
#pragma unroll
    for (int e = 0; e < kStepUnits; ++e) {
        const int i = me + e * 32, t = i / UN - job.tok;   // among the page's tokens
        if (i >= tasks || t < 0 || t >= job.cnt) continue;
        const Unit un = unit_of<true>(p, i % UN, true);
        Angles a;
        angles_of<true>(p, steps, un, job.place + t, a);
        k[e].widen(x[e]);
        turn(p, un, a, x[e]);
        if (F8) {
            raise(ktop, x[e]);
            float y[16];
            v[e].widen(y);
            raise(vtop, y);
        }
    }
    float kinv = 1.f, vinv = 1.f;
    if constexpr (F8) {
        ktop = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(ktop)));
        vtop = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(vtop)));
        const float ks = rescale(p, false, job, h, ktop, me, 32), vs = rescale(p, true, job, h, vtop, me, 32);
        __syncwarp();   // all have read the old ones
        if (me == 0) store_scales(p, job, h, ks, vs);
        kinv = 1.f / ks;
        vinv = 1.f / vs;
    }
#pragma unroll
    for (int e = 0; e < kStepUnits; ++e) {
        const int i = me + e * 32, t = i / UN - job.tok, u = i % UN;
        if (i >= tasks || t < 0 || t >= job.cnt) continue;
        put_unit<F8>(p, false, job, h, t, unit_of<true>(p, u, true), x[e], kinv);
        float y[16];
        v[e].widen(y);
        put_unit<F8>(p, true, job, h, t, {u * 16, u * 16 + 8, -1}, y, vinv);
    }
}

// A step's job for one head, by a warp
template <bool F8, bool FAST>
__device__ __forceinline__ void step_job(const AppendParams& p, const unsigned long long* steps, int n, int j, int h, int me, int32_t* bits) {
    Job job;
    if (!job_of(p, n, j, length_of(p, n), job, bits) || job.id < 0) return;
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
        const float ks = rescale(p, false, job, h, ktop, me, 32), vs = rescale(p, true, job, h, vtop, me, 32);
        __syncwarp();   // all have read the old ones
        if (me == 0) store_scales(p, job, h, ks, vs);
        kinv = 1.f / ks;
        vinv = 1.f / vs;
    }
    const bool kept = F8 && tasks <= 32;   // still in registers
    for (int i = me; i < tasks; i += 32) {
        if (!kept) take(i);
        put_unit<F8>(p, false, job, h, i / UN, unit_of<FAST>(p, i % UN, true), kx, kinv);
        put_unit<F8>(p, true, job, h, i / UN, {i % UN * 16, i % UN * 16 + 8, -1}, vx, vinv);
    }
}

// A prompt's job for heads [h0, h1), by a block
constexpr int kTable = 4096;   // angles of a table: 64 tokens of 64 pairs
constexpr int kBatch = 4;      // units that a thread asks for together
constexpr int kJobWarps = kThreads / 32;

// Where a token's pairs 8 u + 2 i and 8 u + 2 i + 1 lie, in pairs of cosine and sine: neighbouring units side by side
__device__ __forceinline__ int table_at(const AppendParams& p, int t, int u, int i) { return ((t * 4 + i) * (p.rot / 16) + u) * 2; }

__device__ __forceinline__ void fill_table(const AppendParams& p, const unsigned long long* steps, float2* table, const Job& job, int me) {
    const int half = p.rot / 2;
    for (int i = me; i < job.cnt * half; i += kThreads) {
        const int t = i / half, pair = i % half;
        float c, s;
        cos_sin(steps[pair] * static_cast<unsigned long long>(job.place + t), c, s);
        table[table_at(p, t, pair / 8, pair % 8 / 2) + pair % 2] = make_float2(c * p.rope_scale, s * p.rope_scale);
    }
    __syncthreads();
}

__device__ __forceinline__ void from_table(const AppendParams& p, const float2* table, const Unit& un, int t, Angles& a) {
    if (un.pair < 0) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(table + table_at(p, t, un.pair / 8, i));
        a.c[2 * i] = v.x;
        a.s[2 * i] = v.y;
        a.c[2 * i + 1] = v.z;
        a.s[2 * i + 1] = v.w;
    }
}

// Rows of any type and layout, one unit after another: f(values, t, unit, x) for `mine` of
// `count` threads that share a head.
template <bool FAST, typename F>
__device__ __forceinline__ void any_rows(const AppendParams& p, const unsigned long long* steps, const Job& job, int h, int mine, int count, F f) {
    const int UN = p.c.D / 16, tasks = job.cnt * UN;
#pragma unroll 1
    for (int i = mine; i < tasks; i += count) {
        const int t = i / UN, u = i % UN;
        const Unit ku = unit_of<FAST>(p, u, true), vu = {u * 16, u * 16 + 8, -1};
        Angles a;
        angles_of<FAST>(p, steps, ku, job.place + t, a);
        float x[16];
        load_unit<FAST>(p, steps, p.k, (job.tok + t) * p.ks[1] + h * p.ks[2], p.ks[3], p.k_dt, ku, a, job.place + t, true, x);
        f(false, t, ku, x);
        load_unit<FAST>(p, steps, p.v, (job.tok + t) * p.vs[1] + h * p.vs[2], p.vs[3], p.v_dt, vu, a, job.place + t, false, x);
        f(true, t, vu, x);
    }
}

template <bool FAST>
__device__ __noinline__ void any_tops(const AppendParams& p, const unsigned long long* steps, const Job& job, int h, int mine, int count, float* top) {
    any_rows<FAST>(p, steps, job, h, mine, count, [&](bool values, int, const Unit&, const float* x) { raise(top[values], x); });
}

template <bool F8, bool FAST>
__device__ __noinline__ void any_put(const AppendParams& p, const unsigned long long* steps, const Job& job, int h, int mine, int count, float kinv, float vinv) {
    any_rows<FAST>(p, steps, job, h, mine, count,
                   [&](bool values, int t, const Unit& un, const float* x) { put_unit<F8>(p, values, job, h, t, un, x, values ? vinv : kinv); });
}

// bf16 rows that 16-byte loads fit, several asked for at once: f(t, unit, x) with keys rotated,
// or g(raw) alone where RAW
template <bool VALUES, bool RAW, typename A, typename F>
__device__ __forceinline__ void rows(const AppendParams& p, const Job& job, int h, int mine, int count, A angles, F f) {
    const int UN = p.c.D / 16, tasks = job.cnt * UN;
    const unsigned short* base = static_cast<const unsigned short*>(VALUES ? p.v : p.k) + (VALUES ? job.tok * p.vs[1] + h * p.vs[2] : job.tok * p.ks[1] + h * p.ks[2]);
    const int64_t step = VALUES ? p.vs[1] : p.ks[1];
#pragma unroll 1
    for (int i0 = mine; i0 < tasks; i0 += count * kBatch) {
        Raw r[kBatch];
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
            const int i = min(i0 + e * count, tasks - 1);   // the last ones again, to no effect
            r[e].load(base, i / UN * step, unit_of<true>(p, i % UN, !VALUES));
        }
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
            const int i = min(i0 + e * count, tasks - 1), t = i / UN;
            if constexpr (RAW) {
                f(r[e]);
            } else {
                const Unit un = unit_of<true>(p, i % UN, !VALUES);
                float x[16];
                r[e].widen(x);
                if (!VALUES) {
                    Angles a;
                    angles(un, t, a);
                    turn(p, un, a, x);
                }
                f(t, un, x);
            }
        }
    }
}

template <bool F8, bool FAST, bool BF>
__device__ __forceinline__ void prompt_job(const AppendParams& p, const unsigned long long* steps, float2* table, unsigned (*top_s)[2], int n, int j, int h0,
                                           int h1, int me, int32_t* bits) {
    Job job;
    if (!job_of(p, n, j, length_of(p, n), job, bits) || job.id < 0) return;   // the whole block
    const int lane = me % 32, warp = me / 32;
    const bool tab = BF && job.cnt * (p.rot / 2) <= kTable;
    if (tab) fill_table(p, steps, table, job, me);
    int side = kJobWarps;   // heads side by side
    while (side / 2 >= h1 - h0) side /= 2;
    const int slot = warp % side, part = warp / side, count = kJobWarps / side * 32, mine = part * 32 + lane;   // this thread's place among a head's
    auto angles = [&](const Unit& un, int t, Angles& a) {
        if (tab) from_table(p, table, un, t, a);
        else angles_of<FAST>(p, steps, un, job.place + t, a);
    };
#pragma unroll 1
    for (int base = h0; base < h1; base += side) {
        const int h = base + slot;
        const bool on = h < h1;
        float kinv = 1.f, vinv = 1.f;
        bool finite = true;
        if constexpr (F8) {
            auto share = [&](unsigned k, unsigned v) {   // the head's greatest, in top_s
                __syncthreads();   // it is read no more
                if (me < 2 * kJobWarps) top_s[me / 2][me % 2] = 0u;
                __syncthreads();
                k = __reduce_max_sync(0xffffffffu, k);
                v = __reduce_max_sync(0xffffffffu, v);
                if (lane == 0) {
                    atomicMax(&top_s[slot][0], k);
                    atomicMax(&top_s[slot][1], v);
                }
                __syncthreads();
            };
            if constexpr (BF) {
                // infinities and NaN show as the greatest bits; where there are any, once more without them
                float top = 0.f;
                bool nan = false;
                unsigned vtop = 0;
                if (on) {
                    rows<false, false>(p, job, h, mine, count, angles, [&](int, const Unit&, const float* x) {
#pragma unroll
                        for (int q = 0; q < 16; ++q) {
                            top = fmaxf(top, fabsf(x[q]));
                            nan |= x[q] != x[q];
                        }
                    });
                    rows<true, true>(p, job, h, mine, count, angles, [&](const Raw& r) { vtop = max(vtop, r.top()); });
                }
                share(nan ? 0x7fffffffu : __float_as_uint(top), vtop);
#pragma unroll
                for (int e = 0; e < kJobWarps; ++e) finite &= max(top_s[e][0], top_s[e][1]) < 0x7f800000u;
            }
            if (!BF || !finite) {
                float top[2] = {0.f, 0.f};
                if (on) any_tops<FAST>(p, steps, job, h, mine, count, top);
                share(__float_as_uint(top[0]), __float_as_uint(top[1]));
            }
            if (on) {
                kinv = rescale(p, false, job, h, __uint_as_float(top_s[slot][0]), mine, count);
                vinv = rescale(p, true, job, h, __uint_as_float(top_s[slot][1]), mine, count);
            }
            __syncthreads();   // all have read the old scales
            if (on && mine == 0) store_scales(p, job, h, kinv, vinv);
            kinv = 1.f / kinv;
            vinv = 1.f / vinv;
        }
        if (!on) continue;
        if (BF && finite) {
            rows<false, false>(p, job, h, mine, count, angles, [&](int t, const Unit& un, const float* x) { put_unit<F8, true>(p, false, job, h, t, un, x, kinv); });
            rows<true, false>(p, job, h, mine, count, angles, [&](int t, const Unit& un, const float* x) { put_unit<F8, true>(p, true, job, h, t, un, x, vinv); });
        } else {
            any_put<F8, FAST>(p, steps, job, h, mine, count, kinv, vinv);
        }
    }
}

// Rotated queries: a thread a (token, unit), for `hpt` heads
template <bool FAST, bool BF>
__device__ __forceinline__ void q_task(const AppendParams& p, const unsigned long long* steps, int64_t task, int hpt) {
    const int UN = p.c.D / 16, chunks = (p.Hq + hpt - 1) / hpt;
    const int u = static_cast<int>(task % UN), ch = static_cast<int>(task / UN % chunks);
    const int64_t tok = task / UN / chunks;
    int n, t;
    int64_t qrow, orow;
    if (p.cu) {
        n = last_at_most(p.n, tok, [&](int i) { return ld_idx(p.cu, i * p.cu_s, p.cu_dt); });
        int begin, len;
        int32_t bits = 0;   // flagged by the jobs
        span(p, n, &begin, &len, &bits);
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
    const Unit un = unit_of<FAST>(p, u, true);
    const int h1 = min(p.Hq, (ch + 1) * hpt);
    Raw r[BF ? kAtOnce : 1];
    if constexpr (BF) {   // the first rows are asked for before the length is known
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e)
            if (ch * hpt + e < h1) r[e].load(p.q, qrow + (ch * hpt + e) * p.qs[2], un);
    }
    const int64_t start = length_of(p, n);
    if (start < 0) return;
    const int place = static_cast<int>(start) + t;
    Angles a;
    angles_of<FAST>(p, steps, un, place, a);
    float x[16];
    if constexpr (BF) {
        for (int h = ch * hpt; h < h1; h += kAtOnce) {
            if (h > ch * hpt) {
#pragma unroll
                for (int e = 0; e < kAtOnce; ++e)
                    if (h + e < h1) r[e].load(p.q, qrow + (h + e) * p.qs[2], un);
            }
#pragma unroll
            for (int e = 0; e < kAtOnce; ++e)
                if (h + e < h1) {
                    r[e].widen(x);
                    turn(p, un, a, x);
                    put_query<FAST>(p, orow + (h + e) * p.os[2], un, x);
                }
        }
    } else {
        for (int h = ch * hpt; h < h1; ++h) {
            load_unit<FAST>(p, steps, p.q, qrow + h * p.qs[2], p.qs[3], p.q_dt, un, a, place, true, x);
            put_query<FAST>(p, orow + h * p.os[2], un, x);
        }
    }
}

__device__ __forceinline__ void load_steps(const AppendParams& p, unsigned long long* steps) {
    if (threadIdx.x < p.rot / 2) steps[threadIdx.x] = turn_step(__ldg(p.inv_freq + threadIdx.x * p.if_s));
    __syncthreads();
}

// Blocks [0, kv_blocks): a warp a job (sequence, touched page, head); the others: queries
template <bool F8, bool FAST, bool BF>
__global__ void __launch_bounds__(kThreads, 2) append_step(const __grid_constant__ AppendParams p, int kv_blocks, int pages_of, int hpt, int64_t q_tasks) {
    __shared__ unsigned long long steps[128];
    const int tid = threadIdx.x;
    stream_order();
    int32_t bits = 0;
    if (static_cast<int>(blockIdx.x) >= kv_blocks) {
        const int64_t task = static_cast<int64_t>(blockIdx.x - kv_blocks) * kThreads + tid;
        load_steps(p, steps);
        if (task < q_tasks) q_task<FAST, BF>(p, steps, task, hpt);
    } else {
        const int64_t job = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + tid / 32;
        const int h = static_cast<int>(job % p.c.H), j = static_cast<int>(job / p.c.H % pages_of);
        const int64_t n = job / p.c.H / pages_of;
        const bool held = BF && p.T * (p.c.D / 16) <= 32 * kStepUnits;
        StepRows rows;
        if (held && n < p.n) rows.load(p, static_cast<int>(n), h, tid % 32);
        load_steps(p, steps);
        if (n < p.n) {
            if constexpr (BF) {
                if (held) step_job_bf16<F8>(p, steps, rows, static_cast<int>(n), j, h, tid % 32, &bits);
            }
            if (!held) step_job<F8, FAST>(p, steps, static_cast<int>(n), j, h, tid % 32, &bits);
        }
    }
    flag_err(p.dev_err, bits);
}

// Blocks [0, kv_blocks): jobs, where sequence n's pages have numbers from cu[n] / page + 2 n
// on; the others: queries
template <bool F8, bool FAST, bool BF>
__global__ void __launch_bounds__(kThreads, 2) append_prompt(const __grid_constant__ AppendParams p, int kv_blocks, int groups, int heads, int hpt,
                                                                          int64_t q_tasks) {
    __shared__ unsigned long long steps[128];
    __shared__ unsigned top_s[kJobWarps][2];
    __shared__ alignas(16) float2 table[FAST ? kTable : 1];
    stream_order();
    load_steps(p, steps);
    int32_t bits = 0;
    if (static_cast<int>(blockIdx.x) >= kv_blocks) {
        const int64_t task = static_cast<int64_t>(blockIdx.x - kv_blocks) * kThreads + threadIdx.x;
        if (task < q_tasks) q_task<FAST, BF>(p, steps, task, hpt);
        return;
    }
    const int h0 = static_cast<int>(blockIdx.x % groups) * heads;
    const int64_t unit = blockIdx.x / groups;
    auto key = [&](int i) { return ld_idx(p.cu, i * p.cu_s, p.cu_dt) / p.c.page + 2 * static_cast<int64_t>(i); };
    // The search finds no span that offsets fall back behind: each is looked at once besides, by
    // the block of its number (blocks are two a span at least).
    if (static_cast<int>(blockIdx.x) < p.n && threadIdx.x == 0) {
        int begin, len;
        span(p, static_cast<int>(blockIdx.x), &begin, &len, &bits);
    }
    const int n = last_at_most(p.n, unit, key);
    const int64_t j = unit - key(n);
    if (j >= 0 && j < (1 << 30)) prompt_job<F8, FAST, BF>(p, steps, table, top_s, n, static_cast<int>(j), h0, min(p.c.H, h0 + heads), threadIdx.x, &bits);
    flag_err(p.dev_err, bits);
}

template <bool F8, bool FAST>
lar_status launch(const AppendParams& p, cudaStream_t stream) {
    const int64_t limit = (int64_t{1} << 31) - 1;
    const bool bf = p.k_dt == LAR_BF16 && p.v_dt == LAR_BF16 && (!p.q || p.q_dt == LAR_BF16);
    const int64_t tokens = p.cu ? p.ntok : static_cast<int64_t>(p.n) * p.T;
    // asked for where it decides anything: the smallest steps are as long as their launch takes
    int sms = 1;
    if ((p.cu || tokens * (p.c.D / 16) * p.Hq >= 2048) &&
        cached_occupancy(reinterpret_cast<const void*>(append_prompt<F8, FAST, false>), kThreads, 0, 0, &sms) < 1)
        return LAR_ERR_LAUNCH;
    int64_t q_tasks = 0;
    int hpt = 1;   // heads share their angles where there are threads enough without
    if (p.q) {
        const int64_t units = tokens * (p.c.D / 16) * p.Hq;
        if (FAST && bf) hpt = kAtOnce;   // rows that are asked for together take no longer than one
        while (hpt < 32 && hpt < p.Hq && units / (2 * hpt) >= static_cast<int64_t>(sms) * 1024) hpt *= 2;
        q_tasks = tokens * (p.c.D / 16) * ((p.Hq + hpt - 1) / hpt);
    }
    const int64_t q_blocks = (q_tasks + kThreads - 1) / kThreads;
    if (p.cu) {
        const int64_t pages = p.ntok / p.c.page + 2 * static_cast<int64_t>(p.n);
        int heads = 1;   // likewise
        while (heads < 8 && heads < p.c.H && pages * p.c.H >= static_cast<int64_t>(sms) * 2 * heads) heads *= 2;
        const int64_t groups = (p.c.H + heads - 1) / heads;
        if (pages * groups + q_blocks > limit) return LAR_ERR_SHAPE;
        const dim3 grid(static_cast<unsigned>(pages * groups + q_blocks));
        const int kv = static_cast<int>(pages * groups), gr = static_cast<int>(groups);
        if constexpr (FAST) {
            if (bf) return launch_ordered(append_prompt<F8, true, true>, grid, kThreads, 0, 1, stream, p, kv, gr, heads, hpt, q_tasks);
        }
        return launch_ordered(append_prompt<F8, FAST, false>, grid, kThreads, 0, 1, stream, p, kv, gr, heads, hpt, q_tasks);
    }
    const int pages_of = p.T == 1 ? 1 : 2;
    const int64_t kv_blocks = (static_cast<int64_t>(p.n) * pages_of * p.c.H + kThreads / 32 - 1) / (kThreads / 32);
    if (kv_blocks + q_blocks > limit) return LAR_ERR_SHAPE;
    const dim3 grid(static_cast<unsigned>(kv_blocks + q_blocks));
    const int kv = static_cast<int>(kv_blocks);
    if constexpr (FAST) {
        if (bf) return launch_ordered(append_step<F8, true, true>, grid, kThreads, 0, 1, stream, p, kv, pages_of, hpt, q_tasks);
    }
    return launch_ordered(append_step<F8, FAST, false>, grid, kThreads, 0, 1, stream, p, kv, pages_of, hpt, q_tasks);
}

}  // namespace

lar_status launch_append(const AppendParams& p, void* stream) {
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool fast = p.vec && p.rot % 16 == 0;
    if (p.c.e4m3) return fast ? launch<true, true>(p, s) : launch<true, false>(p, s);
    return fast ? launch<false, true>(p, s) : launch<false, false>(p, s);
}

}  // namespace lar

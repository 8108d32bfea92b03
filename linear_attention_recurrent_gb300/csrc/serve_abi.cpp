// serve_abi.cpp -- C entry points of the paged key/value cache (append, attention)
// and of the draw of tokens.  As in lar_abi.cpp every descriptor is validated on the
// host and nothing is launched (and nothing written) unless every check passes.
#include <math.h>
#include <stdint.h>

#include "abi_checks.h"
#include "lar.h"
#include "serve_params.h"

using namespace lar;

namespace {

struct CacheIn {
    const lar_tensor *k_cache, *v_cache, *k_scale, *v_scale, *block_table, *seq_lens;
};

lar_status check_pages(const lar_tensor* t) {
    if (!t) return LAR_ERR_NULL;
    if (t->dtype == LAR_E4M3) {   // the one type that check() does not take
        lar_tensor b = *t;
        b.dtype = LAR_BF16;
        b.data = reinterpret_cast<void*>(reinterpret_cast<uintptr_t>(t->data) & ~uintptr_t{1});
        if (!b.data) b.data = t->data;
        LAR_TRY(check(&b, 4, 4, false));
    } else {
        if (t->dtype != LAR_BF16) return LAR_ERR_DTYPE;
        LAR_TRY(check(t, 4, 4, false));
    }
    const int64_t es = elem_size(t->dtype);
    if (t->shape[3] > 1 && t->stride[3] != 1) return LAR_ERR_STRIDE;
    if (reinterpret_cast<uintptr_t>(t->data) % 16) return LAR_ERR_ALIGN;
    for (int i = 0; i < 3; ++i)
        if ((t->stride[i] * es) % 16) return LAR_ERR_ALIGN;
    return LAR_OK;
}

lar_status check_scale(const lar_tensor* t, int64_t P, int64_t H, float** data, int64_t* st) {
    LAR_TRY(check(t, 2, 2, false));
    if (t->dtype != LAR_F32) return LAR_ERR_DTYPE;
    if (t->shape[0] != P || t->shape[1] != H) return LAR_ERR_SHAPE;
    *data = static_cast<float*>(t->data);
    st[0] = t->stride[0];
    st[1] = t->stride[1];
    return LAR_OK;
}

lar_status check_cache(const CacheIn& in, int64_t n, CacheParams& c) {
    LAR_TRY(check_pages(in.k_cache));
    LAR_TRY(check_pages(in.v_cache));
    if (in.k_cache->dtype != in.v_cache->dtype) return LAR_ERR_DTYPE;
    for (int i = 0; i < 4; ++i)
        if (in.k_cache->shape[i] != in.v_cache->shape[i]) return LAR_ERR_SHAPE;
    const int64_t P = in.k_cache->shape[0], page = in.k_cache->shape[1], H = in.k_cache->shape[2],
                  D = in.k_cache->shape[3];
    if (D != 64 && D != 128 && D != 256) return LAR_ERR_SHAPE;
    if (page < 16 || page > 1024 || page % 16 || H < 1 || H > 1024 || P > (int64_t{1} << 31) - 1) return LAR_ERR_SHAPE;
    c.e4m3 = in.k_cache->dtype == LAR_E4M3;
    if (c.e4m3) {
        LAR_TRY(check_scale(in.k_scale, P, H, &c.k_scale, c.kss));
        LAR_TRY(check_scale(in.v_scale, P, H, &c.v_scale, c.vss));
    } else if (in.k_scale || in.v_scale) {
        return LAR_ERR_ARG;   // 16-bit pages have no scales
    }
    LAR_TRY(check(in.block_table, 2, 2, true));
    const int64_t M = in.block_table->shape[1];
    if (in.block_table->shape[0] != n || M > (1 << 30) / page) return LAR_ERR_SHAPE;
    LAR_TRY(vec_view(in.seq_lens, n, true, &c.lens, &c.len_s, &c.len_dt));
    c.k = in.k_cache->data;
    c.v = in.v_cache->data;
    for (int i = 0; i < 3; ++i) {
        c.ks[i] = in.k_cache->stride[i];
        c.vs[i] = in.v_cache->stride[i];
    }
    c.P = P;
    c.page = static_cast<int>(page);
    c.H = static_cast<int>(H);
    c.D = static_cast<int>(D);
    c.M = static_cast<int>(M);
    c.table = in.block_table->data;
    c.tab_s[0] = in.block_table->stride[0];
    c.tab_s[1] = in.block_table->stride[1];
    c.tab_dt = in.block_table->dtype;
    return LAR_OK;
}

// Two views of one shape whose address ranges meet may still be apart, as the keys'
// and the values' halves of one buffer are: with equal strides they form one view with
// one more dimension, which must not overlap itself.
bool apart(const lar_tensor* a, const lar_tensor* b) {
    if (!meet(range_of(a), range_of(b))) return true;
    if (a->ndim != b->ndim || a->ndim > 4 || a->dtype != b->dtype) return false;
    for (int i = 0; i < a->ndim; ++i)
        if (a->stride[i] != b->stride[i] || a->shape[i] != b->shape[i]) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a->data), y = reinterpret_cast<uintptr_t>(b->data);
    const uintptr_t off = x < y ? y - x : x - y;
    const int64_t es = elem_size(a->dtype);
    if (off % es) return false;
    lar_tensor both = *a;
    both.shape[both.ndim] = 2;
    both.stride[both.ndim] = static_cast<int64_t>(off) / es;
    both.ndim++;
    return !overlaps_itself(&both);
}

bool vec_rows(const void* data, int dt, const int64_t st[4]) { return vec8(data, dt, st, 3, st[3]); }

}  // namespace

extern "C" {

lar_status kv_append(const lar_tensor* q, const lar_tensor* k, const lar_tensor* v, const lar_tensor* q_out,
                     const lar_tensor* k_cache, const lar_tensor* v_cache, const lar_tensor* k_scale,
                     const lar_tensor* v_scale, const lar_tensor* block_table, const lar_tensor* seq_lens,
                     const lar_tensor* cu_seqlens, const lar_tensor* inv_freq, float rope_scale, uint32_t flags,
                     int32_t* dev_err, void* stream) {
    AppendParams p{};
    if (flags & ~static_cast<uint32_t>(LAR_ROPE_INTERLEAVED)) return LAR_ERR_ARG;
    const bool packed = cu_seqlens != nullptr;
    LAR_TRY(check(k, 3, packed ? 3 : 4, false));
    const int nd = k->ndim;
    LAR_TRY(check(v, nd, nd, false));
    if ((q == nullptr) != (q_out == nullptr)) return LAR_ERR_ARG;
    if (q) {
        LAR_TRY(check(q, nd, nd, false));
        LAR_TRY(check(q_out, nd, nd, false));
    }
    int64_t n, T;
    if (packed) {
        LAR_TRY(check(cu_seqlens, 1, 1, true));
        n = cu_seqlens->shape[0] - 1;
        p.ntok = k->shape[0];
        if (n < 0 || n > 65535 || p.ntok > (1 << 30)) return LAR_ERR_SHAPE;
        T = p.ntok;
        p.T = 0;
        p.cu = cu_seqlens->data;
        p.cu_s = cu_seqlens->stride[0];
        p.cu_dt = cu_seqlens->dtype;
    } else {
        n = k->shape[0];
        T = nd == 3 ? 1 : k->shape[1];
        if (n > 65535 || T < 1 || T > 16) return LAR_ERR_SHAPE;
        p.T = static_cast<int>(T);
    }
    LAR_TRY(check_cache({k_cache, v_cache, k_scale, v_scale, block_table, seq_lens}, n, p.c));
    const int64_t hd[2] = {p.c.H, p.c.D};
    LAR_TRY(token_view(k, packed, n, T, hd, 2, p.ks));
    LAR_TRY(token_view(v, packed, n, T, hd, 2, p.vs));
    if (q) {
        const int64_t hq[2] = {q->shape[nd - 2], p.c.D};
        if (hq[0] < 1 || hq[0] > 65535 || hq[0] % p.c.H) return LAR_ERR_SHAPE;
        LAR_TRY(token_view(q, packed, n, T, hq, 2, p.qs));
        LAR_TRY(token_view(q_out, packed, n, T, hq, 2, p.os));
        if (overlaps_itself(q_out)) return LAR_ERR_STRIDE;
        p.Hq = static_cast<int>(hq[0]);
        p.q = q->data; p.q_dt = q->dtype;
        p.q_out = q_out->data; p.o_dt = q_out->dtype;
    }
    if (inv_freq) {
        LAR_TRY(check(inv_freq, 1, 1, false));
        if (inv_freq->dtype != LAR_F32) return LAR_ERR_DTYPE;
        if (inv_freq->shape[0] < 1 || 2 * inv_freq->shape[0] > p.c.D) return LAR_ERR_SHAPE;
        p.inv_freq = static_cast<const float*>(inv_freq->data);
        p.if_s = inv_freq->stride[0];
        p.rot = static_cast<int>(2 * inv_freq->shape[0]);
        if (!isfinite(rope_scale)) return LAR_ERR_ARG;
    } else if (flags || rope_scale != 1.f) {
        return LAR_ERR_ARG;   // a way to rotate without frequencies
    }
    p.interleaved = (flags & LAR_ROPE_INTERLEAVED) != 0;
    p.rope_scale = rope_scale;
    if (overlaps_itself(k_cache) || overlaps_itself(v_cache) ||
        (p.c.e4m3 && (overlaps_itself(k_scale) || overlaps_itself(v_scale))))
        return LAR_ERR_STRIDE;
    p.n = static_cast<int>(n);
    p.k = k->data; p.k_dt = k->dtype;
    p.v = v->data; p.v_dt = v->dtype;
    p.dev_err = dev_err;
    // keys against values may lie between one another; everything else may not
    if (!apart(k_cache, v_cache) || (p.c.e4m3 && !apart(k_scale, v_scale))) return LAR_ERR_ALIAS;
    const lar_tensor* ins[] = {q, k, v, block_table, seq_lens, cu_seqlens, inv_freq};
    for (int i = 0; i < 2; ++i) {
        const lar_tensor* outs[] = {i ? v_cache : k_cache, i ? v_scale : k_scale, q_out};
        LAR_TRY(check_aliasing(outs, 3, ins, 7, dev_err));
    }
    const lar_tensor* a[] = {k_cache, v_scale};
    const lar_tensor* b[] = {v_cache, k_scale};
    LAR_TRY(check_aliasing(a, 2, nullptr, 0, dev_err));
    LAR_TRY(check_aliasing(b, 2, nullptr, 0, dev_err));
    p.vec = vec_rows(p.k, p.k_dt, p.ks) && vec_rows(p.v, p.v_dt, p.vs) &&
            (!q || (vec_rows(p.q, p.q_dt, p.qs) && vec_rows(p.q_out, p.o_dt, p.os)));
    if (n == 0 || T == 0) return LAR_OK;
    return launch_append(p, stream);
}

int64_t attn_workspace(int32_t T, int32_t Hq, int32_t H, int32_t D) {
    if (T < 1 || T > 16 || H < 1 || H > 1024 || Hq < H || Hq % H || Hq / H > 256 || (D != 64 && D != 128 && D != 256)) return -1;
    return attn_workspace_floats(T, Hq / H, D);
}

lar_status attn_decode(const lar_tensor* q, const lar_tensor* k_cache, const lar_tensor* v_cache,
                       const lar_tensor* k_scale, const lar_tensor* v_scale, const lar_tensor* block_table,
                       const lar_tensor* seq_lens, const lar_tensor* out, const lar_tensor* lse,
                       const lar_tensor* workspace, float scale, int32_t window, int32_t* dev_err, void* stream) {
    AttnParams p{};
    LAR_TRY(check(q, 3, 4, false));
    const int nd = q->ndim;
    LAR_TRY(check(out, nd, nd, false));
    if (q->dtype != LAR_BF16) return LAR_ERR_DTYPE;
    const int64_t n = q->shape[0], T = nd == 3 ? 1 : q->shape[1], Hq = q->shape[nd - 2];
    if (n > 65535 || T < 1 || T > 16) return LAR_ERR_SHAPE;
    LAR_TRY(check_cache({k_cache, v_cache, k_scale, v_scale, block_table, seq_lens}, n, p.c));
    if (Hq < 1 || Hq % p.c.H || Hq / p.c.H > 256) return LAR_ERR_SHAPE;
    if (window < 0 || !isfinite(scale)) return LAR_ERR_ARG;
    const int64_t hd[2] = {Hq, p.c.D};
    LAR_TRY(token_view(q, false, n, T, hd, 2, p.qs));
    LAR_TRY(token_view(out, false, n, T, hd, 2, p.os));
    if (overlaps_itself(out)) return LAR_ERR_STRIDE;
    p.B = static_cast<int>(n);
    p.T = static_cast<int>(T);
    p.Hq = static_cast<int>(Hq);
    p.G = static_cast<int>(Hq / p.c.H);
    if (lse) {
        LAR_TRY(check(lse, nd - 1, nd - 1, false));
        if (lse->dtype != LAR_F32) return LAR_ERR_DTYPE;
        LAR_TRY(token_view(lse, false, n, T, hd, 1, p.ls));
        if (overlaps_itself(lse)) return LAR_ERR_STRIDE;
        p.lse = static_cast<float*>(lse->data);
    }
    LAR_TRY(check(workspace, 1, 1, false));
    if (workspace->dtype != LAR_F32) return LAR_ERR_DTYPE;
    if (workspace->shape[0] < attn_workspace_floats(p.T, p.G, p.c.D)) return LAR_ERR_SHAPE;
    if (workspace->stride[0] != 1) return LAR_ERR_STRIDE;
    if (reinterpret_cast<uintptr_t>(workspace->data) % 16) return LAR_ERR_ALIGN;
    p.ws = static_cast<float*>(workspace->data);
    p.q = q->data;
    p.q_pairs = p.qs[3] == 1 && reinterpret_cast<uintptr_t>(q->data) % 4 == 0 && !((p.qs[0] | p.qs[1] | p.qs[2]) & 1);
    p.out = out->data; p.o_dt = out->dtype;
    p.scale = scale;
    p.window = window;
    p.dev_err = dev_err;
    const lar_tensor* outs[] = {out, lse, workspace};
    const lar_tensor* ins[] = {q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens};
    LAR_TRY(check_aliasing(outs, 3, ins, 7, dev_err));
    if (n == 0) return LAR_OK;
    return launch_attn(p, stream);
}

lar_status sample_tokens(const lar_tensor* logits, const lar_tensor* u, const lar_tensor* temperature,
                         const lar_tensor* top_k, const lar_tensor* top_p, const lar_tensor* min_p,
                         const lar_tensor* tokens, const lar_tensor* probs, int32_t* dev_err, void* stream) {
    SampleParams p{};
    LAR_TRY(check(logits, 2, 3, false));
    const int nd = logits->ndim;
    const int64_t B = logits->shape[0], T = nd == 3 ? logits->shape[1] : 1, V = logits->shape[nd - 1];
    if (B > 65535 || T < 1 || T > 16 || V < 1 || V > (1 << 24)) return LAR_ERR_SHAPE;
    LAR_TRY(token_view(logits, false, B, T, &V, 1, p.xs));
    int64_t st[2];
    LAR_TRY(check(u, nd - 1, nd - 1, false));
    if (u->dtype != LAR_F32) return LAR_ERR_DTYPE;
    LAR_TRY(token_view(u, false, B, T, nullptr, 0, st));
    p.us[0] = st[0]; p.us[1] = st[1];
    LAR_TRY(check(tokens, nd - 1, nd - 1, true));
    LAR_TRY(token_view(tokens, false, B, T, nullptr, 0, p.ts));
    if (overlaps_itself(tokens)) return LAR_ERR_STRIDE;
    if (temperature) LAR_TRY(f32_vec(temperature, B, &p.temp, &p.temp_s));
    if (top_p) LAR_TRY(f32_vec(top_p, B, &p.top_p, &p.tp_s));
    if (min_p) LAR_TRY(f32_vec(min_p, B, &p.min_p, &p.mp_s));
    if (top_k) LAR_TRY(vec_view(top_k, B, true, &p.top_k, &p.tk_s, &p.tk_dt));
    if (probs) {
        LAR_TRY(check(probs, nd, nd, false));
        if (probs->dtype != LAR_F32) return LAR_ERR_DTYPE;
        LAR_TRY(token_view(probs, false, B, T, &V, 1, p.ps));
        if (overlaps_itself(probs)) return LAR_ERR_STRIDE;
        p.probs = static_cast<float*>(probs->data);
    }
    p.B = static_cast<int>(B);
    p.T = static_cast<int>(T);
    p.V = V;
    p.x = logits->data; p.x_dt = logits->dtype;
    p.u = static_cast<const float*>(u->data);
    p.tok = tokens->data; p.tok_dt = tokens->dtype;
    p.dev_err = dev_err;
    const lar_tensor* outs[] = {tokens, probs};
    const lar_tensor* ins[] = {logits, u, temperature, top_k, top_p, min_p};
    LAR_TRY(check_aliasing(outs, 2, ins, 6, dev_err));
    if (B == 0) return LAR_OK;
    return launch_sample(p, stream);
}

}  // extern "C"

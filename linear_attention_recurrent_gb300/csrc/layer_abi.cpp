// layer_abi.cpp -- C entry points of the calls around the recurrent state decode:
// the causal convolution, the selective scan and the verification of drafted
// tokens.  As in lar_abi.cpp every descriptor is validated on the host and
// nothing is launched (and nothing written) unless every check passes.
#include <stdint.h>

#include "abi_checks.h"
#include "lar.h"
#include "layer_params.h"

using namespace lar;

namespace {

// How a call names its slots and tokens.
struct Where {
    const lar_tensor *read_idx, *write_idx, *num_accepted, *state_idx, *cu_seqlens;
    bool tokens;   // per-token slots
    bool packed;   // cu_seqlens
};

// lead: x, whose leading sizes are [B, T] (`rest` trailing ones) or [tokens].
lar_status check_where(const Where& w, const lar_tensor* lead, int rest, SlotParams& s) {
    int64_t n;
    if (w.packed) {
        LAR_TRY(check(w.cu_seqlens, 1, 1, true));
        n = w.cu_seqlens->shape[0] - 1;
        if (lead->ndim != 1 + rest) return LAR_ERR_RANK;
        // places in the token arrays, and a part's end past them, fit 32 bits in the kernels
        if (n < 0 || n > 65535 || lead->shape[0] > (1 << 30)) return LAR_ERR_SHAPE;
        s.cu = w.cu_seqlens->data;
        s.cu_s = w.cu_seqlens->stride[0];
        s.cu_dt = w.cu_seqlens->dtype;
        s.ntok = lead->shape[0];
        s.T = 1;
    } else {
        n = lead->shape[0];
        const int64_t T = lead->ndim == 1 + rest ? 1 : lead->shape[1];
        if (n > 65535 || T < 1 || T > 16) return LAR_ERR_SHAPE;
        s.T = static_cast<int>(T);
    }
    s.n = static_cast<int>(n);
    if (w.tokens) {
        if (!w.state_idx) return LAR_ERR_NULL;
        if ((w.read_idx == nullptr) == (w.num_accepted == nullptr)) return LAR_ERR_ARG;
        LAR_TRY(check(w.state_idx, 2, 2, true));
        if (w.state_idx->shape[0] != n || w.state_idx->shape[1] != s.T) return LAR_ERR_SHAPE;
        s.tslot = w.state_idx->data;
        s.tsl_s[0] = w.state_idx->stride[0];
        s.tsl_s[1] = w.state_idx->stride[1];
        s.tsl_dt = w.state_idx->dtype;
        if (w.num_accepted) return vec_view(w.num_accepted, n, true, &s.nacc, &s.na_s, &s.na_dt);
    }
    LAR_TRY(vec_view(w.read_idx, n, true, &s.ridx, &s.ri_s, &s.ri_dt));
    if (w.write_idx) LAR_TRY(vec_view(w.write_idx, n, true, &s.widx, &s.wi_s, &s.wi_dt));
    return LAR_OK;
}

// pool [P, rows, cols]: innermost stride 1, 16-byte aligned rows.
lar_status check_pool(const lar_tensor* t, int64_t rows, int64_t cols, bool aligned, int64_t ps[2], int64_t* P) {
    LAR_TRY(check(t, 3, 3, false));
    if (t->shape[1] != rows || t->shape[2] != cols) return LAR_ERR_SHAPE;
    if (t->stride[2] != 1 && cols > 1) return LAR_ERR_STRIDE;
    const int64_t es = elem_size(t->dtype);
    if (aligned && (reinterpret_cast<uintptr_t>(t->data) % 16 || (t->stride[0] * es) % 16 || (t->stride[1] * es) % 16))
        return LAR_ERR_ALIGN;
    ps[0] = t->stride[0];
    ps[1] = t->stride[1];
    *P = t->shape[0];
    return LAR_OK;
}

lar_status conv(const Where& where, const lar_tensor* x, const lar_tensor* weight, const lar_tensor* bias,
                const lar_tensor* pool, const lar_tensor* out, uint32_t flags, int32_t* dev_err, void* stream) {
    ConvParams p{};
    if (flags & ~static_cast<uint32_t>(LAR_SILU)) return LAR_ERR_ARG;
    LAR_TRY(check(x, 2, where.packed ? 2 : 3, false));
    LAR_TRY(check(weight, 2, 2, false));
    LAR_TRY(check(out, x->ndim, x->ndim, false));
    const int64_t C = x->shape[x->ndim - 1], W = weight->shape[1];
    if (C < 1 || C > (1 << 24) || W < 2 || W > 4 || weight->shape[0] != C) return LAR_ERR_SHAPE;
    LAR_TRY(check_where(where, x, 1, p.s));
    const int64_t T = where.packed ? p.s.ntok : p.s.T;
    LAR_TRY(token_view(x, where.packed, p.s.n, T, &C, 1, p.xs));
    LAR_TRY(token_view(out, where.packed, p.s.n, T, &C, 1, p.os));
    LAR_TRY(check_pool(pool, W - 1, C, false, p.ps, &p.s.P));
    if (overlaps_itself(out) || overlaps_itself(pool)) return LAR_ERR_STRIDE;
    if (bias) LAR_TRY(vec_view(bias, C, false, &p.bias, &p.b_s, &p.bias_dt));
    p.C = static_cast<int>(C);
    p.W = static_cast<int>(W);
    p.x = x->data; p.x_dt = x->dtype;
    p.w = weight->data; p.w_dt = weight->dtype;
    p.ws[0] = weight->stride[0]; p.ws[1] = weight->stride[1];
    p.pool = pool->data; p.pool_dt = pool->dtype;
    p.out = out->data; p.out_dt = out->dtype;
    p.silu = (flags & LAR_SILU) != 0;
    p.s.dev_err = dev_err;
    const lar_tensor* outs[] = {pool, out};
    const lar_tensor* ins[] = {x, weight, bias, where.read_idx, where.write_idx, where.num_accepted, where.state_idx,
                               where.cu_seqlens};
    LAR_TRY(check_aliasing(outs, 2, ins, 8, dev_err));
    p.vec = C % 8 == 0 && vec8(p.x, p.x_dt, p.xs, 2, p.xs[2]) && vec8(p.out, p.out_dt, p.os, 2, p.os[2]) &&
            vec8(p.pool, p.pool_dt, p.ps, 2, 1);
    p.vec_w = p.ws[0] == W && vec8(p.w, p.w_dt, nullptr, 0, p.ws[1]);
    p.vec_b = bias && vec8(p.bias, p.bias_dt, nullptr, 0, p.b_s);
    if (p.s.n == 0) return LAR_OK;
    return where.packed ? lar::launch_conv_prefill(p, stream) : lar::launch_conv_step(p, stream);
}

struct SsmIn {
    const lar_tensor *x, *dt, *A, *B, *C, *D, *z, *dt_bias;
};

lar_status ssm(const Where& where, const SsmIn& in, const lar_tensor* pool, const lar_tensor* out, uint32_t flags,
               int32_t* dev_err, void* stream) {
    SsmParams p{};
    if (flags & ~static_cast<uint32_t>(LAR_DT_SOFTPLUS)) return LAR_ERR_ARG;
    const bool raw = (flags & LAR_DT_SOFTPLUS) != 0;
    if (!raw && in.dt_bias) return LAR_ERR_ARG;   // a bias without its softplus is a caller's mistake
    const int hi = where.packed ? 2 : 3;
    LAR_TRY(check(in.x, 2, hi, false));
    const int nd = in.x->ndim;
    LAR_TRY(check(in.dt, nd, nd, false));
    LAR_TRY(check(out, nd, nd, false));
    LAR_TRY(check(in.A, 2, 2, false));
    LAR_TRY(check(in.B, nd + 1, nd + 1, false));
    LAR_TRY(check(in.C, nd + 1, nd + 1, false));
    if (in.z) LAR_TRY(check(in.z, nd, nd, false));
    if (in.A->dtype != LAR_F32) return LAR_ERR_DTYPE;
    const int64_t D = in.x->shape[nd - 1], N = in.A->shape[1], G = in.B->shape[nd - 1];
    if (N != 16 && N != 32 && N != 64 && N != 128) return LAR_ERR_SHAPE;
    if (D < 1 || D > (1 << 24) || G < 1 || D % G != 0 || in.A->shape[0] != D) return LAR_ERR_SHAPE;
    LAR_TRY(check_where(where, in.x, 1, p.s));
    const int64_t T = where.packed ? p.s.ntok : p.s.T;
    const int64_t gn[2] = {G, N};
    LAR_TRY(token_view(in.x, where.packed, p.s.n, T, &D, 1, p.xs));
    LAR_TRY(token_view(in.dt, where.packed, p.s.n, T, &D, 1, p.ds));
    LAR_TRY(token_view(out, where.packed, p.s.n, T, &D, 1, p.os));
    if (in.z) LAR_TRY(token_view(in.z, where.packed, p.s.n, T, &D, 1, p.zs));
    LAR_TRY(token_view(in.B, where.packed, p.s.n, T, gn, 2, p.bs));
    LAR_TRY(token_view(in.C, where.packed, p.s.n, T, gn, 2, p.cs));
    LAR_TRY(check_pool(pool, D, N, true, p.ps, &p.s.P));
    if (overlaps_itself(out) || overlaps_itself(pool)) return LAR_ERR_STRIDE;
    if (in.D) LAR_TRY(f32_vec(in.D, D, &p.skip, &p.skip_s));
    if (in.dt_bias) LAR_TRY(f32_vec(in.dt_bias, D, &p.dt_bias, &p.dtb_s));
    p.D = static_cast<int>(D);
    p.N = static_cast<int>(N);
    p.G = static_cast<int>(G);
    p.per_group = static_cast<int>(D / G);
    p.x = in.x->data; p.x_dt = in.x->dtype;
    p.dt = in.dt->data; p.dt_dt = in.dt->dtype;
    if (in.z) { p.z = in.z->data; p.z_dt = in.z->dtype; }
    p.B = in.B->data; p.B_dt = in.B->dtype;
    p.C = in.C->data; p.C_dt = in.C->dtype;
    p.A = static_cast<const float*>(in.A->data);
    p.as[0] = in.A->stride[0]; p.as[1] = in.A->stride[1];
    p.pool = pool->data; p.pool_dt = pool->dtype;
    p.out = out->data; p.out_dt = out->dtype;
    p.softplus = raw;
    p.s.dev_err = dev_err;
    const lar_tensor* outs[] = {pool, out};
    const lar_tensor* ins[] = {in.x, in.dt, in.A, in.B, in.C, in.D, in.z, in.dt_bias, where.read_idx, where.write_idx,
                               where.num_accepted, where.state_idx, where.cu_seqlens};
    LAR_TRY(check_aliasing(outs, 2, ins, 13, dev_err));
    p.vec = p.per_group % 8 == 0 && vec8(p.x, p.x_dt, p.xs, 2, p.xs[2]) && vec8(p.dt, p.dt_dt, p.ds, 2, p.ds[2]) &&
            vec8(p.out, p.out_dt, p.os, 2, p.os[2]) && (!in.z || vec8(p.z, p.z_dt, p.zs, 2, p.zs[2]));
    p.vec_bc = vec8(p.B, p.B_dt, p.bs, 3, p.bs[3]) && vec8(p.C, p.C_dt, p.cs, 3, p.cs[3]);
    if (p.s.n == 0) return LAR_OK;
    return where.packed ? lar::launch_ssm_prefill(p, stream) : lar::launch_ssm_step(p, stream);
}

}  // namespace

extern "C" {

lar_status conv_decode(const lar_tensor* x, const lar_tensor* weight, const lar_tensor* bias, const lar_tensor* pool,
                       const lar_tensor* read_idx, const lar_tensor* write_idx, const lar_tensor* out, uint32_t flags,
                       int32_t* dev_err, void* stream) {
    return conv(Where{read_idx, write_idx, nullptr, nullptr, nullptr, false, false}, x, weight, bias, pool, out, flags,
                dev_err, stream);
}

lar_status conv_decode_tokens(const lar_tensor* x, const lar_tensor* weight, const lar_tensor* bias,
                              const lar_tensor* pool, const lar_tensor* read_idx, const lar_tensor* num_accepted,
                              const lar_tensor* state_idx, const lar_tensor* out, uint32_t flags, int32_t* dev_err,
                              void* stream) {
    return conv(Where{read_idx, nullptr, num_accepted, state_idx, nullptr, true, false}, x, weight, bias, pool, out,
                flags, dev_err, stream);
}

lar_status conv_prefill(const lar_tensor* x, const lar_tensor* weight, const lar_tensor* bias, const lar_tensor* pool,
                        const lar_tensor* cu_seqlens, const lar_tensor* read_idx, const lar_tensor* write_idx,
                        const lar_tensor* out, uint32_t flags, int32_t* dev_err, void* stream) {
    return conv(Where{read_idx, write_idx, nullptr, nullptr, cu_seqlens, false, true}, x, weight, bias, pool, out,
                flags, dev_err, stream);
}

lar_status ssm_decode(const lar_tensor* x, const lar_tensor* dt, const lar_tensor* A, const lar_tensor* B,
                      const lar_tensor* C, const lar_tensor* D, const lar_tensor* z, const lar_tensor* dt_bias,
                      const lar_tensor* pool, const lar_tensor* read_idx, const lar_tensor* write_idx,
                      const lar_tensor* out, uint32_t flags, int32_t* dev_err, void* stream) {
    return ssm(Where{read_idx, write_idx, nullptr, nullptr, nullptr, false, false},
               SsmIn{x, dt, A, B, C, D, z, dt_bias}, pool, out, flags, dev_err, stream);
}

lar_status ssm_decode_tokens(const lar_tensor* x, const lar_tensor* dt, const lar_tensor* A, const lar_tensor* B,
                             const lar_tensor* C, const lar_tensor* D, const lar_tensor* z, const lar_tensor* dt_bias,
                             const lar_tensor* pool, const lar_tensor* read_idx, const lar_tensor* num_accepted,
                             const lar_tensor* state_idx, const lar_tensor* out, uint32_t flags, int32_t* dev_err,
                             void* stream) {
    return ssm(Where{read_idx, nullptr, num_accepted, state_idx, nullptr, true, false},
               SsmIn{x, dt, A, B, C, D, z, dt_bias}, pool, out, flags, dev_err, stream);
}

lar_status ssm_prefill(const lar_tensor* x, const lar_tensor* dt, const lar_tensor* A, const lar_tensor* B,
                       const lar_tensor* C, const lar_tensor* D, const lar_tensor* z, const lar_tensor* dt_bias,
                       const lar_tensor* pool, const lar_tensor* cu_seqlens, const lar_tensor* read_idx,
                       const lar_tensor* write_idx, const lar_tensor* out, uint32_t flags, int32_t* dev_err,
                       void* stream) {
    return ssm(Where{read_idx, write_idx, nullptr, nullptr, cu_seqlens, false, true},
               SsmIn{x, dt, A, B, C, D, z, dt_bias}, pool, out, flags, dev_err, stream);
}

lar_status spec_verify(const lar_tensor* draft_tokens, const lar_tensor* draft_probs, const lar_tensor* target_probs,
                       const lar_tensor* u_accept, const lar_tensor* u_sample, const lar_tensor* num_draft,
                       const lar_tensor* num_accepted, const lar_tensor* tokens, int32_t* dev_err, void* stream) {
    VerifyParams p{};
    LAR_TRY(check(target_probs, 3, 3, false));
    const int64_t B = target_probs->shape[0], T = target_probs->shape[1], V = target_probs->shape[2];
    if (B > 65535 || T < 1 || T > 16 || V < 1 || V > (1 << 24)) return LAR_ERR_SHAPE;
    LAR_TRY(check(draft_tokens, 2, 2, true));
    LAR_TRY(check(u_accept, 2, 2, false));
    LAR_TRY(check(u_sample, 1, 1, false));
    LAR_TRY(check(num_accepted, 1, 1, true));
    LAR_TRY(check(tokens, 2, 2, true));
    if (u_accept->dtype != LAR_F32 || u_sample->dtype != LAR_F32) return LAR_ERR_DTYPE;
    if (draft_tokens->shape[0] != B || draft_tokens->shape[1] != T - 1 || u_accept->shape[0] != B ||
        u_accept->shape[1] != T - 1 || u_sample->shape[0] != B || num_accepted->shape[0] != B ||
        tokens->shape[0] != B || tokens->shape[1] != T)
        return LAR_ERR_SHAPE;
    if (overlaps_itself(num_accepted) || overlaps_itself(tokens)) return LAR_ERR_STRIDE;
    if (draft_probs) {
        LAR_TRY(check(draft_probs, 3, 3, false));
        if (draft_probs->shape[0] != B || draft_probs->shape[1] != T - 1 || draft_probs->shape[2] != V)
            return LAR_ERR_SHAPE;
        p.q = draft_probs->data;
        p.q_dt = draft_probs->dtype;
        for (int i = 0; i < 3; ++i) p.qs[i] = draft_probs->stride[i];
    }
    if (num_draft) LAR_TRY(vec_view(num_draft, B, true, &p.nd, &p.nd_s, &p.nd_dt));
    p.B = static_cast<int>(B);
    p.T = static_cast<int>(T);
    p.V = V;
    p.tok = draft_tokens->data; p.tok_dt = draft_tokens->dtype;
    p.p = target_probs->data; p.p_dt = target_probs->dtype;
    p.ua = static_cast<const float*>(u_accept->data);
    p.us = static_cast<const float*>(u_sample->data);
    p.us_s = u_sample->stride[0];
    p.acc = num_accepted->data; p.acc_s = num_accepted->stride[0]; p.acc_dt = num_accepted->dtype;
    p.out = tokens->data; p.out_dt = tokens->dtype;
    for (int i = 0; i < 2; ++i) {
        p.tk_s[i] = draft_tokens->stride[i];
        p.ua_s[i] = u_accept->stride[i];
        p.os[i] = tokens->stride[i];
    }
    for (int i = 0; i < 3; ++i) p.ps[i] = target_probs->stride[i];
    p.dev_err = dev_err;
    const lar_tensor* outs[] = {num_accepted, tokens};
    const lar_tensor* ins[] = {draft_tokens, draft_probs, target_probs, u_accept, u_sample, num_draft};
    LAR_TRY(check_aliasing(outs, 2, ins, 6, dev_err));
    if (B == 0) return LAR_OK;
    return lar::launch_verify(p, stream);
}

}  // extern "C"

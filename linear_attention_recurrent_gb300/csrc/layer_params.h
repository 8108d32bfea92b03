// layer_params.h -- the validated, flattened argument blocks of the calls around
// the recurrent state decode (causal convolution, selective scan, verification
// of drafted tokens), handed from layer_abi.cpp to the launchers.
#pragma once

#include <stdint.h>

#include "lar.h"

namespace lar {

// Which pool slots a call reads and writes, as in the decode calls.  Every
// stride is in elements.
struct SlotParams {
    int n;                                          // sequences
    int T;                                          // tokens per sequence (1 for packed spans)
    int64_t P;                                      // pool slots
    const void* ridx;  int64_t ri_s; int ri_dt;     // [n], NULL with nacc
    const void* widx;  int64_t wi_s; int wi_dt;     // [n] or NULL: write to the read slot
    const void* nacc;  int64_t na_s; int na_dt;     // accepted counts [n] or NULL
    const void* tslot; int64_t tsl_s[2]; int tsl_dt;  // per-token slots [n, T] or NULL
    const void* cu;    int64_t cu_s; int cu_dt;     // span offsets [n + 1] or NULL (fixed T)
    int64_t ntok;                                   // packed: tokens in the arrays
    int32_t* dev_err;
};

// y[t, c] = bias[c] + sum_j w[c, j] x[t - (W - 1) + j, c]
struct ConvParams {
    SlotParams s;
    int C, W;
    const void* x;    int64_t xs[3]; int x_dt;      // sequence, token, channel (packed: sequence stride 0)
    const void* w;    int64_t ws[2]; int w_dt;      // channel, tap
    const void* bias; int64_t b_s; int bias_dt;     // [C] or NULL
    void* pool;       int64_t ps[2]; int pool_dt;   // slot, row (channel stride 1)
    void* out;        int64_t os[3]; int out_dt;
    int silu;
    int vec;                                        // 16-byte accesses of 8 channels fit x, out and the pool
    int vec_w, vec_b;                               // and the weights of 8 channels lie in one piece, and the bias
};

// h[d, n] <- exp(dt[d] A[d, n]) h[d, n] + dt[d] x[d] B[g, n];  y[d] = sum_n C[g, n] h[d, n] + D[d] x[d]
struct SsmParams {
    SlotParams s;
    int D, N, G, per_group;                         // per_group = D / G
    const void* x;  int64_t xs[3]; int x_dt;
    const void* dt; int64_t ds[3]; int dt_dt;
    const void* z;  int64_t zs[3]; int z_dt;        // or NULL
    const void* B;  int64_t bs[4]; int B_dt;        // sequence, token, group, state
    const void* C;  int64_t cs[4]; int C_dt;
    const float* A; int64_t as[2];                  // channel, state
    const float* skip;    int64_t skip_s;           // D of the formula, [D] or NULL
    const float* dt_bias; int64_t dtb_s;            // [D] or NULL
    void* pool; int64_t ps[2]; int pool_dt;         // slot, channel (state stride 1)
    void* out;  int64_t os[3]; int out_dt;
    int softplus;
    int vec;                                        // 16-byte accesses of 8 channels fit x, dt, z and out
    int vec_bc;                                     // 16-byte accesses of rows of states fit B and C
};

struct VerifyParams {
    int B, T;
    int64_t V;
    const void* tok;    int64_t tk_s[2]; int tok_dt;     // [B, T - 1]
    const void* q;      int64_t qs[3]; int q_dt;         // [B, T - 1, V] or NULL: one-hot at the drafted token
    const void* p;      int64_t ps[3]; int p_dt;         // [B, T, V]
    const float* ua;    int64_t ua_s[2];                 // [B, T - 1]
    const float* us;    int64_t us_s;                    // [B]
    const void* nd;     int64_t nd_s; int nd_dt;         // drafted tokens [B] or NULL: T - 1
    void* acc;          int64_t acc_s; int acc_dt;       // [B]
    void* out;          int64_t os[2]; int out_dt;       // [B, T]
    int32_t* dev_err;
};

lar_status launch_conv_step(const ConvParams& p, void* stream);      // fixed T (conv_decode, conv_decode_tokens)
lar_status launch_conv_prefill(const ConvParams& p, void* stream);
lar_status launch_ssm_step(const SsmParams& p, void* stream);        // fixed T (ssm_decode, ssm_decode_tokens)
lar_status launch_ssm_prefill(const SsmParams& p, void* stream);
lar_status launch_verify(const VerifyParams& p, void* stream);

}  // namespace lar

// serve_params.h -- the validated, flattened argument blocks of the paged
// key/value cache's calls and of the draw of tokens, handed from serve_abi.cpp to
// the launchers.  Every stride is in elements.
#pragma once

#include <stdint.h>

#include "lar.h"

namespace lar {

// A paged cache of keys and values: [P, page, H, D], dimension stride 1, and the
// table that names each sequence's pages.
struct CacheParams {
    void *k, *v;
    int64_t ks[3], vs[3];                           // page, token, head
    float *k_scale, *v_scale;                       // [P, H] for e4m3, else NULL
    int64_t kss[2], vss[2];
    int e4m3;                                       // else bf16
    int64_t P;
    int page, H, D;
    const void* table; int64_t tab_s[2]; int tab_dt;  // [B, M]
    int M;
    const void* lens;  int64_t len_s; int len_dt;     // [B]: tokens before the call
};

struct AppendParams {
    CacheParams c;
    int n, T, Hq;                                   // sequences, tokens a sequence (fixed form), query heads
    const void* cu; int64_t cu_s; int cu_dt;        // span offsets [n + 1] or NULL
    int64_t ntok;                                   // packed: tokens in the arrays
    const void* q; int64_t qs[4]; int q_dt;         // sequence, token, head, dimension; or NULL
    const void* k; int64_t ks[4]; int k_dt;
    const void* v; int64_t vs[4]; int v_dt;
    void* q_out;   int64_t os[4]; int o_dt;
    const float* inv_freq; int64_t if_s;            // [rot / 2] or NULL
    int rot, interleaved;
    float rope_scale;
    int vec;                                        // 16-byte accesses of 8 dimensions fit q, k, v and q_out
    int32_t* dev_err;
};

struct AttnParams {
    CacheParams c;
    int B, T, Hq, G;                                // G = Hq / H
    const void* q; int64_t qs[4];                   // bf16
    int q_pairs;                                    // 4-byte accesses of two dimensions fit q
    void* out; int64_t os[4]; int o_dt;
    float* lse; int64_t ls[3];                      // [B, T, Hq] or NULL
    float* ws;                                      // partial sums of blocks that share a pair
    float scale;
    int window;                                     // 0: none
    int32_t* dev_err;
};

struct SampleParams {
    int B, T;
    int64_t V;
    const void* x; int64_t xs[3]; int x_dt;         // [B, T, V]
    const float* u; int64_t us[2];                  // [B, T]
    const float* temp; int64_t temp_s;              // [B] or NULL, as the next three
    const void* top_k; int64_t tk_s; int tk_dt;
    const float* top_p; int64_t tp_s;
    const float* min_p; int64_t mp_s;
    void* tok; int64_t ts[2]; int tok_dt;           // [B, T]
    float* probs; int64_t ps[3];                    // [B, T, V] or NULL
    int32_t* dev_err;
};

// floats of workspace that a call of this shape may use
int64_t attn_workspace_floats(int T, int G, int D);

lar_status launch_append(const AppendParams& p, void* stream);
lar_status launch_attn(const AttnParams& p, void* stream);
lar_status launch_sample(const SampleParams& p, void* stream);

}  // namespace lar

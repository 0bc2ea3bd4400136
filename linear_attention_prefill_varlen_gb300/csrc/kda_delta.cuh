// The gated delta rule: what its kernels share.
#pragma once

#include "kda_layer.cuh"

namespace kda_layer {

struct DeltaParams {
    const void *q, *k, *v, *gate, *beta;
    const float *a_log, *dt_bias;
    float *states;
    void *out;
    const int32_t *cache_indices, *query_start_loc;  // query_start_loc NULL: token i is sequence i
    const uint8_t *has_initial_state;                // NULL: all set
    int64_t qs[2], ks[2], vs[2], gs[2], bs[2], os[2], ss[2];
    int64_t ci_stride, null_block_id, tokens;
    int num_seqs, heads;
    int gate_dtype, gate_kind, beta_dtype, beta_kind;
    float scale;
};

// softplus in the form that neither overflows nor cancels.
__device__ __forceinline__ float softplus_f(float x) {
    return fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x)));
}

// The decay exp(g) of one channel from the stored gate value.
__device__ __forceinline__ float decay_of(float raw, int kind, float neg_a, float bias) {
    const float g = kind == KDA_GATE_SOFTPLUS ? neg_a * softplus_f(raw + bias) : raw;
    return expf(g);
}

__device__ __forceinline__ float beta_of(float raw, int kind) {
    return kind == KDA_BETA_SIGMOID ? sigmoid_f(raw) : raw;
}

// Sequence s: its rows [start, end) clamped to the tokens, its state line (-1:
// the null block), and whether it reads the line.
struct Seq {
    int64_t start, end, line;
    bool reads;
};

__device__ __forceinline__ Seq load_seq(const DeltaParams &p, int s) {
    Seq q;
    if (p.query_start_loc == nullptr) {
        q.start = s, q.end = s + 1;
    } else {
        q.start = max((int64_t)p.query_start_loc[s], (int64_t)0);
        q.end = min((int64_t)p.query_start_loc[s + 1], p.tokens);
    }
    const int64_t line = p.cache_indices[s * p.ci_stride];
    const bool null = line == p.null_block_id;
    q.line = null ? -1 : line;
    q.reads = !null && (p.has_initial_state == nullptr || p.has_initial_state[s] != 0);
    return q;
}

}  // namespace kda_layer

// The gated delta rule, token by token (include/kda_layer.h, kda_delta_t).
//
// The rows v of a state are independent: row v needs only v_t[v], and k, q,
// beta and the decays that all rows share.  A warp keeps 4 * kGroups rows of
// one head's state in registers for a whole sequence: 8 lanes per row, each
// with D / 8 of its columns, so one 16-byte load covers a quarter of four rows
// and a dot product is D / 8 FMAs and 3 shuffles.  Per token
//     S' = S a,  p = S' k,  r = S' q,  u = beta (v - p),  S = S' + u k,
//     o = scale (r + u (k.q)),
// so that both dot products run on S' together and o needs no second pass.
// The block's warps prepare kBatch tokens at a time in shared memory (decays,
// k, q, v, k.q, beta): a warp per token, once for all rows of the block.
//
// Bound: for one token the state, read and written once, in HBM.
#include "kda_delta_chunk.cuh"

namespace kda_layer {
namespace {

constexpr int kWarps = 8;
constexpr int kBatch = kWarps;  // tokens prepared together

template <int D>
struct Token {
    float a[D], k[D], q[D], v[D];
    float beta, kq, pad[2];
};

template <typename T, int D, int kGroups, bool kChannelGate, typename G>
__global__ void __launch_bounds__(kWarps * 32)
    delta_recurrent_kernel(const __grid_constant__ DeltaParams p, int max_len, int *head) {
    constexpr int kRows = kWarps * 4 * kGroups;  // rows of a block
    constexpr int C = D / 32;                    // channels of a lane in the preparation
    constexpr int NV = D / 32;                   // 4-column pieces of a lane's part of a row
    __shared__ Token<D> tok[kBatch];
    dependency_wait();
    // The head of the chunked path's workspace, before its kernels use it.
    if (head != nullptr && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 64) head[threadIdx.x] = 0;
    const int s = blockIdx.x / p.heads, h = blockIdx.x % p.heads;
    const Seq seq = load_seq(p, s);
    if (seq.start >= seq.end || seq.end - seq.start > max_len) return;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int sub = lane / 8, col = lane % 8;
    const int row0 = blockIdx.y * kRows + warp * 4 * kGroups;
    float *state = p.states + (seq.line < 0 ? 0 : seq.line) * p.ss[0] + h * p.ss[1];

    float S[kGroups][NV][4];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        const float *row = state + (row0 + g * 4 + sub) * D;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (seq.reads) f = *reinterpret_cast<const float4 *>(row + i * 32 + col * 4);
            S[g][i][0] = f.x, S[g][i][1] = f.y, S[g][i][2] = f.z, S[g][i][3] = f.w;
        }
    }
    const float factor = gate_factor(p.a_log, h, p.gate_kind);
    float bias[C] = {};
    if (p.dt_bias != nullptr)
#pragma unroll
        for (int c = 0; c < C; ++c)
            bias[c] = kChannelGate ? p.dt_bias[h * D + lane * C + c] : p.dt_bias[h];
    for (int64_t base = seq.start; base < seq.end; base += kBatch) {
        const int n = (int)min((int64_t)kBatch, seq.end - base);
        if (base != seq.start) __syncthreads();
        if (warp < n) {
            const int64_t t = base + warp;
            Token<D> &to = tok[warp];
            const auto qv = ld_vec<T, C>(static_cast<const T *>(p.q) + t * p.qs[0] + h * p.qs[1] + lane * C);
            const auto kv = ld_vec<T, C>(static_cast<const T *>(p.k) + t * p.ks[0] + h * p.ks[1] + lane * C);
            const auto vv = ld_vec<T, C>(static_cast<const T *>(p.v) + t * p.vs[0] + h * p.vs[1] + lane * C);
            float a[C];
            if constexpr (kChannelGate) {
                const auto gv = ld_vec<G, C>(static_cast<const G *>(p.gate) + t * p.gs[0] + h * p.gs[1] + lane * C);
#pragma unroll
                for (int c = 0; c < C; ++c) a[c] = decay_of(to_f<G>(gv.v[c]), p.gate_kind, factor, bias[c]);
            } else {
                const float one = decay_of(ld_dyn(p.gate, t * p.gs[0] + h * p.gs[1], p.gate_dtype),
                                           p.gate_kind, factor, bias[0]);
#pragma unroll
                for (int c = 0; c < C; ++c) a[c] = one;
            }
            float kq = 0.0f;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const float kf = to_f<T>(kv.v[c]), qf = to_f<T>(qv.v[c]);
                to.a[lane * C + c] = a[c];
                to.k[lane * C + c] = kf;
                to.q[lane * C + c] = qf;
                to.v[lane * C + c] = to_f<T>(vv.v[c]);
                kq = fmaf(kf, qf, kq);
            }
#pragma unroll
            for (int m = 16; m > 0; m /= 2) kq += __shfl_xor_sync(0xffffffffu, kq, m);
            if (lane == 0) {
                to.kq = kq;
                to.beta = beta_of(ld_dyn(p.beta, t * p.bs[0] + h * p.bs[1], p.beta_dtype), p.beta_kind);
            }
        }
        __syncthreads();
        for (int j = 0; j < n; ++j) {
            const Token<D> &to = tok[j];
            float pk[kGroups] = {}, rq[kGroups] = {};
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const float4 a = *reinterpret_cast<const float4 *>(to.a + i * 32 + col * 4);
                const float4 k = *reinterpret_cast<const float4 *>(to.k + i * 32 + col * 4);
                const float4 q = *reinterpret_cast<const float4 *>(to.q + i * 32 + col * 4);
                const float av[4] = {a.x, a.y, a.z, a.w}, kv[4] = {k.x, k.y, k.z, k.w},
                            qv[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int g = 0; g < kGroups; ++g)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        S[g][i][c] *= av[c];
                        pk[g] = fmaf(S[g][i][c], kv[c], pk[g]);
                        rq[g] = fmaf(S[g][i][c], qv[c], rq[g]);
                    }
            }
#pragma unroll
            for (int m = 4; m > 0; m /= 2)
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    pk[g] += __shfl_xor_sync(0xffffffffu, pk[g], m);
                    rq[g] += __shfl_xor_sync(0xffffffffu, rq[g], m);
                }
            const float beta = to.beta, kq = to.kq;
            float o = 0.0f;
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                const float u = beta * (to.v[row0 + g * 4 + sub] - pk[g]);
                if (col == g) o = p.scale * fmaf(u, kq, rq[g]);
                pk[g] = u;
            }
            if (col < kGroups) {
                T *out = static_cast<T *>(p.out) + (base + j) * p.os[0] + h * p.os[1];
                out[row0 + col * 4 + sub] = from_f<T>(o);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const float4 k = *reinterpret_cast<const float4 *>(to.k + i * 32 + col * 4);
                const float kv[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
                for (int g = 0; g < kGroups; ++g)
#pragma unroll
                    for (int c = 0; c < 4; ++c) S[g][i][c] = fmaf(pk[g], kv[c], S[g][i][c]);
            }
        }
    }
    if (seq.line < 0) return;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        float *row = state + (row0 + g * 4 + sub) * D;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            *reinterpret_cast<float4 *>(row + i * 32 + col * 4) =
                make_float4(S[g][i][0], S[g][i][1], S[g][i][2], S[g][i][3]);
    }
}

template <typename T, int D, int kGroups, bool kChannelGate, typename G>
cudaError_t launch_groups(const DeltaParams &p, int max_len, int *head, kda_stream_t stream) {
    const dim3 grid((unsigned)((int64_t)p.num_seqs * p.heads), D / (kWarps * 4 * kGroups));
    return launch(delta_recurrent_kernel<T, D, kGroups, kChannelGate, G>, grid, kWarps * 32, 0, stream,
                  p, max_len, head);
}

template <typename T, int D, bool kChannelGate, typename G>
cudaError_t launch_rows(const DeltaParams &p, int max_len, int *head, kda_stream_t stream) {
    // A block of all rows shares one preparation of the tokens; blocks of 32
    // rows spread few (sequence, head) pairs over more SMs.
    if ((int64_t)p.num_seqs * p.heads < 2 * current_sms())
        return launch_groups<T, D, 1, kChannelGate, G>(p, max_len, head, stream);
    return launch_groups<T, D, D / 32, kChannelGate, G>(p, max_len, head, stream);
}

template <typename T, int D>
cudaError_t launch_gate(const DeltaParams &p, bool channel, int max_len, int *head, kda_stream_t stream) {
    if (!channel) return launch_rows<T, D, false, float>(p, max_len, head, stream);
    if (p.gate_dtype == KDA_DTYPE_F32) return launch_rows<T, D, true, float>(p, max_len, head, stream);
    if (p.gate_dtype == KDA_DTYPE_BF16) return launch_rows<T, D, true, __nv_bfloat16>(p, max_len, head, stream);
    return launch_rows<T, D, true, __half>(p, max_len, head, stream);
}

template <typename T>
cudaError_t launch_dim(const DeltaParams &p, int head_dim, bool channel, int max_len, int *head, kda_stream_t stream) {
    if (head_dim == 64) return launch_gate<T, 64>(p, channel, max_len, head, stream);
    return launch_gate<T, 128>(p, channel, max_len, head, stream);
}

// Token by token, sequences of at most max_len tokens.
cudaError_t run_recurrent(const DeltaParams &p, const kda_delta_t *d, int max_len, int *head, kda_stream_t stream) {
    const bool channel = d->gate_per_channel != 0;
    if (d->x_dtype == KDA_DTYPE_BF16)
        return launch_dim<__nv_bfloat16>(p, d->head_dim, channel, max_len, head, stream);
    if (d->x_dtype == KDA_DTYPE_F16) return launch_dim<__half>(p, d->head_dim, channel, max_len, head, stream);
    return launch_dim<float>(p, d->head_dim, channel, max_len, head, stream);
}

bool strides_ok(const int64_t *s, int64_t quantum) {
    return s[0] >= 0 && s[1] >= 0 && s[0] % quantum == 0 && s[1] % quantum == 0;
}

kda_status_t check(const kda_delta_t *d) {
    if (d == nullptr || d->version != 0 || d->reserved != 0 || !dtype_ok(d->x_dtype) ||
        !dtype_ok(d->gate_dtype) || !dtype_ok(d->beta_dtype))
        return KDA_ERR_INVALID_ARG;
    if ((d->gate_kind != KDA_GATE_LOG && d->gate_kind != KDA_GATE_SOFTPLUS) ||
        (d->beta_kind != KDA_BETA_PLAIN && d->beta_kind != KDA_BETA_SIGMOID) ||
        (d->gate_per_channel != 0 && d->gate_per_channel != 1) || d->heads <= 0 ||
        !isfinite(d->scale) || d->cache_index_stride < 0)
        return KDA_ERR_INVALID_ARG;
    if ((d->head_dim != 64 && d->head_dim != 128) || d->heads > 65535) return KDA_ERR_UNSUPPORTED;
    if (d->q == nullptr || d->k == nullptr || d->v == nullptr || d->gate == nullptr || d->beta == nullptr ||
        d->states == nullptr || d->out == nullptr)
        return KDA_ERR_INVALID_ARG;
    if ((d->a_log != nullptr) != (d->gate_kind == KDA_GATE_SOFTPLUS) ||
        (d->dt_bias != nullptr && d->gate_kind != KDA_GATE_SOFTPLUS))
        return KDA_ERR_INVALID_ARG;
    if (d->beta_stride[0] < 0 || d->beta_stride[1] < 0 || d->gate_stride[0] < 0 || d->gate_stride[1] < 0)
        return KDA_ERR_INVALID_ARG;
    const int64_t quantum = 16 / dtype_bytes(d->x_dtype), gq = 16 / dtype_bytes(d->gate_dtype);
    if (!aligned(d->q, 16) || !aligned(d->k, 16) || !aligned(d->v, 16) || !aligned(d->out, 16) ||
        !aligned(d->states, 16) || !strides_ok(d->q_stride, quantum) || !strides_ok(d->k_stride, quantum) ||
        !strides_ok(d->v_stride, quantum) || !strides_ok(d->out_stride, quantum) ||
        !strides_ok(d->state_stride, 4))
        return KDA_ERR_MISALIGNED;
    if (d->gate_per_channel && (!aligned(d->gate, 16) || !strides_ok(d->gate_stride, gq)))
        return KDA_ERR_MISALIGNED;
    if (!aligned(d->gate, (uintptr_t)dtype_bytes(d->gate_dtype)) ||
        !aligned(d->beta, (uintptr_t)dtype_bytes(d->beta_dtype)) || !aligned(d->a_log, 4) ||
        !aligned(d->dt_bias, 4))
        return KDA_ERR_MISALIGNED;
    return KDA_OK;
}

DeltaParams params_of(const kda_delta_t *d) {
    DeltaParams p = {};
    p.q = d->q, p.k = d->k, p.v = d->v, p.gate = d->gate, p.beta = d->beta;
    p.a_log = d->a_log, p.dt_bias = d->dt_bias, p.states = d->states, p.out = d->out;
    for (int i = 0; i < 2; ++i) {
        p.qs[i] = d->q_stride[i], p.ks[i] = d->k_stride[i], p.vs[i] = d->v_stride[i];
        p.gs[i] = d->gate_stride[i], p.bs[i] = d->beta_stride[i], p.os[i] = d->out_stride[i];
        p.ss[i] = d->state_stride[i];
    }
    p.ci_stride = d->cache_index_stride ? d->cache_index_stride : 1;
    p.heads = (int)d->heads;
    p.gate_dtype = d->gate_dtype, p.gate_kind = d->gate_kind;
    p.beta_dtype = d->beta_dtype, p.beta_kind = d->beta_kind;
    p.scale = d->scale;
    return p;
}

// Sequences up to this length go token by token, longer ones in chunks.
constexpr int kShortLen = 16;

// Whether a packed call uses the chunked path: 16-bit x and sequences that can be long.
bool uses_chunks(int64_t tokens, int x_dtype) { return x_dtype != KDA_DTYPE_F32 && tokens > kShortLen; }

// Grids of (sequences x heads) blocks, and token rows, stay below 2^31.
bool sizes_ok(int64_t tokens, int64_t num_seqs, int64_t heads) {
    return tokens >= 0 && num_seqs >= 0 && tokens <= INT32_MAX && num_seqs <= INT32_MAX &&
           heads > 0 && num_seqs <= INT32_MAX / heads;
}

}  // namespace
}  // namespace kda_layer

using namespace kda_layer;

extern "C" {

kda_status_t kda_delta_check(const kda_delta_t *d) { return check(d); }

kda_status_t kda_packed_delta_rule_workspace(int64_t tokens, int64_t num_seqs, int64_t heads,
                                             int32_t head_dim, int32_t x_dtype, int32_t sm_count,
                                             int64_t *bytes) {
    if (bytes == nullptr || !sizes_ok(tokens, num_seqs, heads) || !dtype_ok(x_dtype) || sm_count < 0)
        return KDA_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128) return KDA_ERR_UNSUPPORTED;
    *bytes = 0;
    if (tokens > 0 && num_seqs > 0 && uses_chunks(tokens, x_dtype))
        *bytes = chunk_plan(tokens, num_seqs, heads, head_dim, sm_count ? sm_count : current_sms()).bytes;
    return KDA_OK;
}

kda_status_t kda_packed_delta_rule(const kda_delta_t *d, int64_t tokens,
                                   const int32_t *cache_indices, const uint8_t *has_initial_state,
                                   const int32_t *query_start_loc, int64_t num_seqs,
                                   int64_t null_block_id, void *workspace, int64_t workspace_bytes,
                                   kda_stream_t stream) {
    if (d == nullptr || !sizes_ok(tokens, num_seqs, d->heads)) return KDA_ERR_INVALID_ARG;
    if (tokens == 0 || num_seqs == 0) return KDA_OK;
    const kda_status_t st = check(d);
    if (st != KDA_OK) return st;
    if (cache_indices == nullptr || has_initial_state == nullptr || query_start_loc == nullptr)
        return KDA_ERR_INVALID_ARG;
    DeltaParams p = params_of(d);
    p.cache_indices = cache_indices, p.has_initial_state = has_initial_state;
    p.query_start_loc = query_start_loc;
    p.null_block_id = null_block_id;
    p.num_seqs = (int)num_seqs;
    p.tokens = tokens;
    if (!uses_chunks(tokens, d->x_dtype)) return cuda_status(run_recurrent(p, d, INT32_MAX, nullptr, stream));
    const ChunkPlan plan = chunk_plan(tokens, num_seqs, d->heads, d->head_dim, current_sms());
    if (workspace == nullptr || workspace_bytes < plan.bytes || plan.slots * d->heads > INT32_MAX)
        return KDA_ERR_INVALID_ARG;
    if (!aligned(workspace, 256)) return KDA_ERR_MISALIGNED;
    // The short sequences first: that kernel also zeroes the workspace's head.
    cudaError_t e = run_recurrent(p, d, kShortLen, static_cast<int *>(workspace), stream);
    if (e == cudaSuccess) e = run_chunked(p, d, plan, kShortLen, workspace, stream);
    return cuda_status(e);
}

kda_status_t kda_delta_rule_update(const kda_delta_t *d, int64_t batch, const int32_t *cache_indices,
                                   int64_t null_block_id, kda_stream_t stream) {
    if (d == nullptr || !sizes_ok(batch, batch, d->heads)) return KDA_ERR_INVALID_ARG;
    if (batch == 0) return KDA_OK;
    const kda_status_t st = check(d);
    if (st != KDA_OK) return st;
    if (cache_indices == nullptr) return KDA_ERR_INVALID_ARG;
    DeltaParams p = params_of(d);
    p.cache_indices = cache_indices;
    p.null_block_id = null_block_id;
    p.num_seqs = (int)batch;
    p.tokens = batch;
    return cuda_status(run_recurrent(p, d, 1, nullptr, stream));
}

}  // extern "C"

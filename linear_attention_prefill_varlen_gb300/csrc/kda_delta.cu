// The gated delta rule on the state's rows in registers (include/kda_layer.h,
// kda_delta_t): one token per sequence, and whole sequences.
//
// The rows v of a state are independent: row v needs only v_t[v], and k, q, beta
// and the decays that all rows share. A warp keeps rows of one head's state in
// registers, a row spread over 8 or 16 lanes. Per token
//     S' = S a,  p = S' k,  r = S' q,  u = beta (v - p),  S = S' + u k,
//     o = scale (r + u (k.q)),
// so that both dot products run on S' together and o needs no second pass.
//
// Bound: for one token the state, read and written once, in HBM (1024 tokens of
// 12 heads: 250 us, 6.49 TB/s, 97% of a device copy's rate).
#include "kda_delta_chunk.cuh"

namespace kda_layer {
namespace {

constexpr int kWarps = 8;

// ------------------------------------------------------------------ one token

template <int D>
struct Token {
    float a[D], k[D], q[D], v[D];
    float beta, kq, pad[2];
};

template <typename T, int D, int kGroups, bool kChannelGate, typename G>
__global__ void __launch_bounds__(kWarps * 32) delta_update_kernel(const __grid_constant__ DeltaParams p) {
    constexpr int kRows = kWarps * 4 * kGroups;  // rows of a block
    constexpr int C = D / 32;                    // channels of a lane in the preparation
    constexpr int NV = D / 32;                   // 4-column pieces of a lane's part of a row
    __shared__ Token<D> to;
    dependency_wait();
    const int s = blockIdx.x / p.heads, h = blockIdx.x % p.heads;
    const Seq seq = load_seq(p, s);
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
    if (warp == 0) {
        const int64_t t = s;
        const float factor = gate_factor(p.a_log, h, p.gate_kind);
        float bias[C] = {};
        if (p.dt_bias != nullptr)
#pragma unroll
            for (int c = 0; c < C; ++c)
                bias[c] = kChannelGate ? p.dt_bias[h * D + lane * C + c] : p.dt_bias[h];
        const auto qv = ld_vec<T, C>(static_cast<const T *>(p.q) + t * p.qs[0] + h * p.qs[1] + lane * C);
        const auto kv = ld_vec<T, C>(static_cast<const T *>(p.k) + t * p.ks[0] + h * p.ks[1] + lane * C);
        const auto vv = ld_vec<T, C>(static_cast<const T *>(p.v) + t * p.vs[0] + h * p.vs[1] + lane * C);
        float a[C];
        if constexpr (kChannelGate) {
            const auto gv = ld_vec<G, C>(static_cast<const G *>(p.gate) + t * p.gs[0] + h * p.gs[1] + lane * C);
#pragma unroll
            for (int c = 0; c < C; ++c) a[c] = decay_of(to_f<G>(gv.v[c]), p.gate_kind, factor, bias[c]);
        } else {
            const float one = decay_of(ld_dyn(p.gate, t * p.gs[0] + h * p.gs[1], p.gate_dtype), p.gate_kind, factor, bias[0]);
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
    float pk[kGroups] = {}, rq[kGroups] = {};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const float4 a = *reinterpret_cast<const float4 *>(to.a + i * 32 + col * 4);
        const float4 k = *reinterpret_cast<const float4 *>(to.k + i * 32 + col * 4);
        const float4 q = *reinterpret_cast<const float4 *>(to.q + i * 32 + col * 4);
        const float av[4] = {a.x, a.y, a.z, a.w}, kv[4] = {k.x, k.y, k.z, k.w}, qv[4] = {q.x, q.y, q.z, q.w};
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
    float o = 0.0f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        const float u = to.beta * (to.v[row0 + g * 4 + sub] - pk[g]);
        if (col == g) o = p.scale * fmaf(u, to.kq, rq[g]);
        pk[g] = u;
    }
    if (col < kGroups)
        static_cast<T *>(p.out)[(int64_t)s * p.os[0] + h * p.os[1] + row0 + col * 4 + sub] = from_f<T>(o);
    if (seq.line < 0) return;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        float *row = state + (row0 + g * 4 + sub) * D;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const float4 k = *reinterpret_cast<const float4 *>(to.k + i * 32 + col * 4);
            *reinterpret_cast<float4 *>(row + i * 32 + col * 4) =
                make_float4(fmaf(pk[g], k.x, S[g][i][0]), fmaf(pk[g], k.y, S[g][i][1]),
                            fmaf(pk[g], k.z, S[g][i][2]), fmaf(pk[g], k.w, S[g][i][3]));
        }
    }
}

// ------------------------------------------------------------------ sequences, four tokens at a time

// With G_j the decays of a block's tokens up to j and H_j those after j,
//     p_j = S (k_j G_j),  r_j = S (q_j G_j)              all from the block's first S
//     u_j = beta_j (v_j - p_j - sum_{i<j} u_i M_ji),     M_ji = k_j . (k_i G_j / G_i)
//     o_j = scale (r_j + sum_{i<=j} u_i N_ji),           N_ji = q_j . (k_i G_j / G_i)
//     S   = S G_3 + sum_j u_j (k_j H_j)
// (the quotients are products of the decays between). The state is touched 13
// times for 4 tokens instead of 16, and one reduction over lanes, not four, stands
// between a block and the next. The block's threads prepare two such groups at a
// time in shared memory, a thread per channel. A row belongs to 16 lanes: with 8,
// shared memory would be read twice as often per product, and it, not the FP32
// pipe, would bound the loop.
constexpr int kTokens = 4, kBlocks = 2, kRound = kTokens * kBlocks;

template <int D>
struct Round {
    float kd[kRound][D], qd[kRound][D], ku[kRound][D], v[kRound][D], a[kBlocks][D];
    float part[kBlocks][4][16];  // per warp: M (k) and N (q) sums, pairs in pair_at's order
    float coef[kBlocks][16];
    float beta[kRound];
};

// Order of the 16 sums: N_ji for i <= j, then M_ji for i < j.
__host__ __device__ constexpr int n_at(int j, int i) { return j * (j + 1) / 2 + i; }
__host__ __device__ constexpr int m_at(int j, int i) { return 10 + j * (j - 1) / 2 + i; }

// m tokens of group b of the round.
template <typename T, int D, int kGroups, int m>
__device__ __forceinline__ void group(const DeltaParams &p, const Round<D> &sm, int b, float2 (&S)[kGroups][D / 64][2],
                                      int64_t base, int h, int row0, int lane) {
    constexpr int NV = D / 64, kDup = 16 / kGroups;
    const int sub = lane / 16, col = lane % 16;
    float sums[2][m];
#pragma unroll
    for (int j = 0; j < m; ++j)
#pragma unroll
        for (int what = 0; what < 2; ++what) {
            const float *x = (what ? sm.qd : sm.kd)[b * kTokens + j];
            float2 acc[kGroups];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const float4 f = *reinterpret_cast<const float4 *>(x + i * 64 + col * 4);
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    acc[g] = i == 0 ? __fmul2_rn(S[g][i][0], make_float2(f.x, f.y))
                                    : __ffma2_rn(S[g][i][0], make_float2(f.x, f.y), acc[g]);
                    acc[g] = __ffma2_rn(S[g][i][1], make_float2(f.z, f.w), acc[g]);
                }
            }
            float v[kGroups];
#pragma unroll
            for (int g = 0; g < kGroups; ++g) v[g] = acc[g].x + acc[g].y;
            // Sums over the 16 lanes of a row, group g to lanes kDup g ...
#pragma unroll
            for (int w = 8, left = kGroups; w > 0; w /= 2, left = left > 1 ? left / 2 : 1) {
                if (left > 1) {
                    const bool up = col & w;
#pragma unroll
                    for (int g = 0; g < left / 2; ++g) {
                        const float send = up ? v[g] : v[g + left / 2], keep = up ? v[g + left / 2] : v[g];
                        v[g] = keep + __shfl_xor_sync(0xffffffffu, send, w);
                    }
                } else {
                    v[0] += __shfl_xor_sync(0xffffffffu, v[0], w);
                }
            }
            sums[what][j] = v[0];
        }
    // The lane's row: its u and o
    const int row = row0 + col / kDup * 2 + sub;
    float c[16], u[m];
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
        const float4 f = *reinterpret_cast<const float4 *>(&sm.coef[b][i]);
        c[i] = f.x, c[i + 1] = f.y, c[i + 2] = f.z, c[i + 3] = f.w;
    }
    T *out = static_cast<T *>(p.out) + (base + b * kTokens) * p.os[0] + h * p.os[1] + row;
#pragma unroll
    for (int j = 0; j < m; ++j) {
        float x = sm.v[b * kTokens + j][row] - sums[0][j];
#pragma unroll
        for (int i = 0; i < j; ++i) x = fmaf(-u[i], c[m_at(j, i)], x);
        u[j] = sm.beta[b * kTokens + j] * x;
        float o = sums[1][j];
#pragma unroll
        for (int i = 0; i <= j; ++i) o = fmaf(u[i], c[n_at(j, i)], o);
        if (col % kDup == j % kDup) out[j * p.os[0]] = from_f<T>(p.scale * o);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const float4 f = *reinterpret_cast<const float4 *>(sm.a[b] + i * 64 + col * 4);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            S[g][i][0] = __fmul2_rn(S[g][i][0], make_float2(f.x, f.y));
            S[g][i][1] = __fmul2_rn(S[g][i][1], make_float2(f.z, f.w));
        }
    }
#pragma unroll
    for (int j = 0; j < m; ++j) {
        float uj[kGroups];
#pragma unroll
        for (int g = 0; g < kGroups; ++g) uj[g] = __shfl_sync(0xffffffffu, u[j], sub * 16 + g * kDup);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const float4 f = *reinterpret_cast<const float4 *>(sm.ku[b * kTokens + j] + i * 64 + col * 4);
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                S[g][i][0] = __ffma2_rn(make_float2(uj[g], uj[g]), make_float2(f.x, f.y), S[g][i][0]);
                S[g][i][1] = __ffma2_rn(make_float2(uj[g], uj[g]), make_float2(f.z, f.w), S[g][i][1]);
            }
        }
    }
}

template <typename T, int D, int kGroups, bool kChannelGate, typename G>
__global__ void __launch_bounds__(kWarps * 32, 2)
    delta_recurrent_kernel(const __grid_constant__ DeltaParams p, int max_len, int *head) {
    constexpr int kRows = kWarps * 2 * kGroups;  // rows of a block
    constexpr int NV = D / 64;                   // 4-column pieces of a lane's part of a row
    __shared__ Round<D> sm;
    dependency_wait();
    // The head of the chunked path's workspace, before its kernels use it.
    if (head != nullptr && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 64) head[threadIdx.x] = 0;
    const int s = blockIdx.x / p.heads, h = blockIdx.x % p.heads;
    const Seq seq = load_seq(p, s);
    const int64_t len = seq.end - seq.start;
    if (len <= 0 || len > max_len) return;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int sub = lane / 16, col = lane % 16;
    const int row0 = blockIdx.y * kRows + warp * 2 * kGroups;
    float *state = p.states + (seq.line < 0 ? 0 : seq.line) * p.ss[0] + h * p.ss[1];

    // Preparation: channel d of group blk of the round. Rows past the end read the
    // last row instead and are masked.
    const int d = threadIdx.x % D, blk = threadIdx.x / D;
    const bool prepares = D * kBlocks == kWarps * 32 || blk < kBlocks;
    T qr[kTokens], kr[kTokens], vr[kTokens];
    G gr[kTokens];
    float one[kTokens], br = 0.0f;
    auto load = [&](int64_t first) {
#pragma unroll
        for (int j = 0; j < kTokens; ++j) {
            const int64_t t = seq.start + min(first + blk * kTokens + j, len - 1);
            qr[j] = static_cast<const T *>(p.q)[t * p.qs[0] + h * p.qs[1] + d];
            kr[j] = static_cast<const T *>(p.k)[t * p.ks[0] + h * p.ks[1] + d];
            vr[j] = static_cast<const T *>(p.v)[t * p.vs[0] + h * p.vs[1] + d];
            if constexpr (kChannelGate) gr[j] = static_cast<const G *>(p.gate)[t * p.gs[0] + h * p.gs[1] + d];
            else one[j] = ld_dyn(p.gate, t * p.gs[0] + h * p.gs[1], p.gate_dtype);
        }
        const int64_t t = seq.start + min(first + (int)(threadIdx.x % kRound), len - 1);
        br = ld_dyn(p.beta, t * p.bs[0] + h * p.bs[1], p.beta_dtype);
    };
    load(0);
    float2 S[kGroups][NV][2];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        const float *row = state + (row0 + g * 2 + sub) * D;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (seq.reads) f = *reinterpret_cast<const float4 *>(row + i * 64 + col * 4);
            S[g][i][0] = make_float2(f.x, f.y), S[g][i][1] = make_float2(f.z, f.w);
        }
    }
    const float factor = gate_factor(p.a_log, h, p.gate_kind);
    const float bias = p.dt_bias == nullptr ? 0.0f : kChannelGate ? p.dt_bias[h * D + d] : p.dt_bias[h];

    for (int64_t base = 0; base < len; base += kRound) {
        const int n = (int)min((int64_t)kRound, len - base);
        if (base != 0) __syncthreads();
        if (prepares) {
            float a[kTokens], k[kTokens], q[kTokens];
            float run = 1.0f, f[16];
#pragma unroll
            for (int j = 0; j < kTokens; ++j) {
                const int at = blk * kTokens + j;
                const bool in = at < n;
                const float decay = decay_of(kChannelGate ? to_f<G>(gr[j]) : one[j], p.gate_kind, factor, bias);
                a[j] = in ? decay : 1.0f;
                k[j] = in ? to_f<T>(kr[j]) : 0.0f;
                q[j] = in ? to_f<T>(qr[j]) : 0.0f;
                run *= a[j];
                sm.kd[at][d] = k[j] * run;
                sm.qd[at][d] = q[j] * run;
                sm.v[at][d] = in ? to_f<T>(vr[j]) : 0.0f;
            }
            sm.a[blk][d] = run;
            run = 1.0f;
#pragma unroll
            for (int j = kTokens - 1; j >= 0; --j) {
                sm.ku[blk * kTokens + j][d] = k[j] * run;
                run *= a[j];
            }
#pragma unroll
            for (int i = 0; i < kTokens; ++i) {
                float w = k[i];
                f[n_at(i, i)] = q[i] * w;
#pragma unroll
                for (int j = i + 1; j < kTokens; ++j) {
                    w *= a[j];
                    f[n_at(j, i)] = q[j] * w;
                    f[m_at(j, i)] = k[j] * w;
                }
            }
            const float sum = scatter_sum(f, lane);
            if (lane % 2 == 0) sm.part[blk][warp % (D / 32)][lane / 2] = sum;
            if (threadIdx.x < kRound) sm.beta[threadIdx.x] = (int)threadIdx.x < n ? beta_of(br, p.beta_kind) : 0.0f;
        }
        // The next round's tokens, while these are worked on (without a branch, at whose
        // end the loaded registers would be waited for; past the end, the last row again).
        load(base + kRound);
        __syncthreads();
        if (threadIdx.x < kBlocks * 16) {
            float sum = 0.0f;
#pragma unroll
            for (int x = 0; x < D / 32; ++x) sum += sm.part[threadIdx.x / 16][x][threadIdx.x % 16];
            sm.coef[threadIdx.x / 16][threadIdx.x % 16] = sum;
        }
        __syncthreads();
        for (int b = 0; b * kTokens < n; ++b) {
            const int m = min(kTokens, n - b * kTokens);
            // Whole groups in straight line, so that the sums of all tokens overlap.
            if (m == kTokens) group<T, D, kGroups, kTokens>(p, sm, b, S, seq.start + base, h, row0, lane);
            else if (m == 1) group<T, D, kGroups, 1>(p, sm, b, S, seq.start + base, h, row0, lane);
            else if (m == 2) group<T, D, kGroups, 2>(p, sm, b, S, seq.start + base, h, row0, lane);
            else group<T, D, kGroups, 3>(p, sm, b, S, seq.start + base, h, row0, lane);
        }
    }
    if (seq.line < 0) return;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        float *row = state + (row0 + g * 2 + sub) * D;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            *reinterpret_cast<float4 *>(row + i * 64 + col * 4) =
                make_float4(S[g][i][0].x, S[g][i][0].y, S[g][i][1].x, S[g][i][1].y);
    }
}

// ------------------------------------------------------------------ host

// A block of all of a head's rows shares one preparation of the tokens; blocks of
// 32 rows spread few (sequence, head) pairs over more SMs.
bool few_pairs(const DeltaParams &p) { return (int64_t)p.num_seqs * p.heads < 2 * current_sms(); }

template <typename T, int D, bool kChannelGate, typename G>
struct Update {
    static cudaError_t run(const DeltaParams &p, int, int *, kda_stream_t stream) {
        const unsigned pairs = (unsigned)((int64_t)p.num_seqs * p.heads);
        if (few_pairs(p))
            return launch(delta_update_kernel<T, D, 1, kChannelGate, G>, dim3(pairs, D / 32), kWarps * 32, 0, stream, p);
        return launch(delta_update_kernel<T, D, D / 32, kChannelGate, G>, dim3(pairs), kWarps * 32, 0, stream, p);
    }
};

template <typename T, int D, bool kChannelGate, typename G>
struct Recurrent {
    static cudaError_t run(const DeltaParams &p, int max_len, int *head, kda_stream_t stream) {
        const unsigned pairs = (unsigned)((int64_t)p.num_seqs * p.heads);
        if (few_pairs(p))
            return launch(delta_recurrent_kernel<T, D, 2, kChannelGate, G>, dim3(pairs, D / 32), kWarps * 32, 0, stream,
                          p, max_len, head);
        return launch(delta_recurrent_kernel<T, D, D / 16, kChannelGate, G>, dim3(pairs), kWarps * 32, 0, stream, p,
                      max_len, head);
    }
};

template <template <typename, int, bool, typename> class Op, typename T, int D>
cudaError_t run_gate(const DeltaParams &p, bool channel, int max_len, int *head, kda_stream_t stream) {
    if (!channel) return Op<T, D, false, float>::run(p, max_len, head, stream);
    if (p.gate_dtype == KDA_DTYPE_F32) return Op<T, D, true, float>::run(p, max_len, head, stream);
    if (p.gate_dtype == KDA_DTYPE_BF16) return Op<T, D, true, __nv_bfloat16>::run(p, max_len, head, stream);
    return Op<T, D, true, __half>::run(p, max_len, head, stream);
}

template <template <typename, int, bool, typename> class Op, typename T>
cudaError_t run_dim(const DeltaParams &p, const kda_delta_t *d, int max_len, int *head, kda_stream_t stream) {
    const bool channel = d->gate_per_channel != 0;
    return d->head_dim == 64 ? run_gate<Op, T, 64>(p, channel, max_len, head, stream)
                             : run_gate<Op, T, 128>(p, channel, max_len, head, stream);
}

// Sequences of at most max_len tokens; head: 256 bytes to zero, or NULL.
template <template <typename, int, bool, typename> class Op>
cudaError_t run_op(const DeltaParams &p, const kda_delta_t *d, int max_len, int *head, kda_stream_t stream) {
    if (d->x_dtype == KDA_DTYPE_BF16) return run_dim<Op, __nv_bfloat16>(p, d, max_len, head, stream);
    if (d->x_dtype == KDA_DTYPE_F16) return run_dim<Op, __half>(p, d, max_len, head, stream);
    return run_dim<Op, float>(p, d, max_len, head, stream);
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

// Sequences up to this length go four tokens at a time through FP32, longer ones in
// chunks. Where all (sequence, head) pairs run at once (four blocks of 32 rows each,
// two per SM) the chunked path's launches cost as much as about 80 tokens; a full
// GPU does 40 tokens for the price of a chunk (bf16, 12 heads of 128, us: one
// sequence of 64 tokens 22 against 33, of 128 42 against 36; 256 sequences of 32 362
// against 494, of 64 682 against 507).
int short_len(int64_t num_seqs, int64_t heads) {
    return num_seqs * heads * 4 <= 2 * (int64_t)current_sms() ? 80 : 40;
}

// Whether a packed call uses the chunked path: 16-bit x and sequences that can be long.
bool uses_chunks(int64_t tokens, int x_dtype, int short_tokens) { return x_dtype != KDA_DTYPE_F32 && tokens > short_tokens; }

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
    if (tokens > 0 && num_seqs > 0 && uses_chunks(tokens, x_dtype, 40))  // the shorter of the two lengths
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
    const int short_tokens = short_len(num_seqs, d->heads);
    if (!uses_chunks(tokens, d->x_dtype, short_tokens)) return cuda_status(run_op<Recurrent>(p, d, INT32_MAX, nullptr, stream));
    const ChunkPlan plan = chunk_plan(tokens, num_seqs, d->heads, d->head_dim, current_sms());
    if (workspace == nullptr || workspace_bytes < plan.bytes || plan.slots * d->heads > INT32_MAX)
        return KDA_ERR_INVALID_ARG;
    if (!aligned(workspace, 256)) return KDA_ERR_MISALIGNED;
    // The short sequences first: that kernel also zeroes the workspace's head.
    cudaError_t e = run_op<Recurrent>(p, d, short_tokens, static_cast<int *>(workspace), stream);
    if (e == cudaSuccess) e = run_chunked(p, d, plan, short_tokens, workspace, stream);
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
    return cuda_status(run_op<Update>(p, d, 1, nullptr, stream));
}

}  // extern "C"

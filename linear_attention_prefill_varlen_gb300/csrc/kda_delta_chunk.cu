// The gated delta rule in chunks of 64 tokens (include/kda_layer.h, kda_delta_t).
//
// Inside a chunk that starts from the state S0 (rows v, columns k), with
// G_i = the product of the decays of its tokens up to i (per channel):
//     L_ij = beta_i sum_k k_i k_j G_i / G_j          (i > j)
//     A_ij =        sum_k q_i k_j G_i / G_j          (i >= j)
//     T    = (I + L)^-1,  W = T diag(beta) (k G),  U = T diag(beta) v
//     V'   = U - W S0^T                              (the rows u of the recurrence)
//     o    = scale * ((q G) S0^T + A V')
//     S1   = S0 diag(G_63) + V'^T (k G_63 / G)
// The quotients of decays are never formed: a product over the tokens between
// j and i is built from the decays themselves, with a reference point between
// the two tokens, so every factor is in [0, 1] and nothing overflows (levels
// of 8, 16, 32 and 64 tokens; pairs inside 8 tokens by running products).
//
// 1. prepare: a block per (chunk, head), all in parallel, computes T, W, U, A
//    and the decayed q and k, and writes them as the shared-memory images the
//    walk needs.
// 2. walk: a block per (segment, head) goes through its chunks in order with the
//    state in registers; three products per chunk on tcgen05 with the state
//    and V' as TMEM operands.
// 3. A sequence longer than a segment is first walked without outputs: from
//    zero (B) and from the identity (M), per segment; since a segment maps a
//    state S to S M + B, a small kernel then finds every segment's first state.
//
// Precision: the state path is FP32. Tensor-core operands on it are pairs of
// halves, x 2^s = hi + lo with 22 bits, s taken from the largest value of the
// tile (of the row for S and V'), and three products hi hi, hi lo, lo hi summed
// in FP32. What feeds only o (q G, A, and S and V' there) is one half: 11 bits
// against the 8 or 11 of the output's type.
#include "kda_delta_chunk.cuh"

namespace kda_layer {
namespace {

// ------------------------------------------------------------------ layout

// Workspace of one (chunk slot, head), in bytes. Operand images are what the
// tensor core reads: rows of 128 bytes (64 halves), 16-byte pieces of row r at
// piece ^ (r % 8), column blocks of 64 one after another.
template <int D>
struct Slot {
    static constexpr int kW = kChunk * D * 2;                 // one W image (hi or lo)
    static constexpr int w_hi = 0, w_lo = kW;                 // [token][k]
    static constexpr int k_hi = 2 * kW, k_lo = 3 * kW;        // [k][token]
    static constexpr int q = 4 * kW;                          // [token][k]
    static constexpr int a = 5 * kW;                          // [i][j], 64 x 64
    static constexpr int u = a + kChunk * kChunk * 2;         // fp32 [token][v]
    static constexpr int decay = u + kChunk * D * 4;          // fp32 [k]: G_63
    static constexpr int scales = decay + D * 4;              // fp32: W, k, q, A unscaling
    static constexpr int bytes = scales + 64;
};

constexpr int kHeader = 256;  // workspace: first word set when a wait ran out

__host__ __device__ constexpr int64_t slot_bytes(int D) { return D == 64 ? Slot<64>::bytes : Slot<128>::bytes; }

// Byte offset of half (row, col) in an operand image of `rows` rows.
__device__ __forceinline__ int image_at(int row, int col, int rows) {
    return (col >> 6) * rows * 128 + row * 128 + ((((col >> 3) & 7) ^ (row & 7)) << 4) + (col & 7) * 2;
}

// ------------------------------------------------------------------ scaling

// Power-of-two scaling of a group of values with the largest magnitude m: up
// brings them below 2^15, down undoes it. The exponent is kept where both are
// normal numbers.
__device__ __forceinline__ float scale_up(float m) {
    const int e = min(max((int)(__float_as_uint(m) >> 23) & 255, 20), 254);
    return __uint_as_float((uint32_t)(268 - e) << 23);
}
__device__ __forceinline__ float scale_down(float m) {
    const int e = min(max((int)(__float_as_uint(m) >> 23) & 255, 20), 254);
    return __uint_as_float((uint32_t)(e - 14) << 23);
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// hi and lo halves of two values.
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = pack2(a - f.x, b - f.y);
}

// ------------------------------------------------------------------ mma.sync

__device__ __forceinline__ uint32_t smem_u32(const void *p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
}
__device__ __forceinline__ void ldsm2(uint32_t (&r)[2], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];"
                 : "=r"(r[0]), "=r"(r[1]) : "r"(at));
}
__device__ __forceinline__ void ldsm2t(uint32_t (&r)[2], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];"
                 : "=r"(r[0]), "=r"(r[1]) : "r"(at));
}
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
                 "{%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// ------------------------------------------------------------------ prepare

// The sequence that owns slot j of a map f(s) = floor(qsl[s] / unit) + s (the
// largest s with f(s) <= j), and j - f(s).
__device__ __forceinline__ int find_seq(const DeltaParams &p, int64_t j, int64_t unit, int64_t &rest) {
    int lo = 0, hi = p.num_seqs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        const int64_t at = max((int64_t)p.query_start_loc[mid], (int64_t)0);
        if (at / unit + mid <= j) lo = mid;
        else hi = mid - 1;
    }
    rest = j - (max((int64_t)p.query_start_loc[lo], (int64_t)0) / unit + lo);
    return lo;
}

template <int D>
struct PrepSmem {
    static constexpr int kRow = D + 8;  // halves: rows 16 bytes past a multiple of 128 bytes
    union {
        struct { __half lk_hi[32][kRow], lk_lo[32][kRow], lq[32][kRow], rk_hi[32][kRow], rk_lo[32][kRow]; } lv;
        struct { __half k_hi[64][kRow], k_lo[64][kRow]; } kg;
    } x;
    __half v[64][kRow];
    union {
        float L[64][68];
        struct { __half hi[64][72], lo[64][72]; } t;
    } l;
    float T[64][68];
    float tmp[3][16][20];
    __half A[64][72];
    float block_decay[8][D];
    float beta[64];
    uint32_t top[4][8];  // per warp: largest |k|, |q|, |v|, then T', W
};

template <int C>
__device__ __forceinline__ void store_row(__half *at, const float (&f)[C]) {
    if constexpr (C == 4) {
        *reinterpret_cast<uint2 *>(at) = make_uint2(pack2(f[0], f[1]), pack2(f[2], f[3]));
    } else {
        *reinterpret_cast<uint32_t *>(at) = pack2(f[0], f[1]);
    }
}

template <int C>
__device__ __forceinline__ void store_split(__half *hi, __half *lo, const float (&f)[C]) {
    uint32_t h[2], l[2];
    split2(f[0], f[1], h[0], l[0]);
    if constexpr (C == 4) {
        split2(f[2], f[3], h[1], l[1]);
        *reinterpret_cast<uint2 *>(hi) = make_uint2(h[0], h[1]);
        *reinterpret_cast<uint2 *>(lo) = make_uint2(l[0], l[1]);
    } else {
        *reinterpret_cast<uint32_t *>(hi) = h[0];
        *reinterpret_cast<uint32_t *>(lo) = l[0];
    }
}

// The sums over the warp of 32 values, value i to lane i.
__device__ __forceinline__ float scatter_sum(float (&v)[32], int lane) {
#pragma unroll
    for (int m = 16; m > 0; m /= 2) {
        const bool up = lane & m;
#pragma unroll
        for (int i = 0; i < m; ++i) {
            const float send = up ? v[i] : v[i + m];
            const float keep = up ? v[i + m] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
        }
    }
    return v[0];
}

// The larger of 8 warps' bit patterns of magnitudes, as a float.
__device__ __forceinline__ float top_of(const uint32_t (&t)[8]) {
    uint32_t m = t[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max(m, t[i]);
    return __uint_as_float(m);
}

__device__ __forceinline__ uint32_t mag(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// One (chunk, head). Warp b holds tokens 8b .. 8b + 7 in registers, a lane C
// channels of each.
template <typename T, int D, bool kChannelGate, typename G>
__global__ void __launch_bounds__(256, 2)
    delta_prepare_kernel(const __grid_constant__ DeltaParams p, char *ws, int short_len) {
    constexpr int C = D / 32;
    extern __shared__ __align__(1024) char raw_smem[];
    PrepSmem<D> &sm = *reinterpret_cast<PrepSmem<D> *>(raw_smem);
    dependency_wait();
    const int64_t slot = blockIdx.x / p.heads;
    const int h = blockIdx.x % p.heads;
    int64_t chunk;
    const int s = find_seq(p, slot, kChunk, chunk);
    const Seq seq = load_seq(p, s);
    const int64_t len = seq.end - seq.start;
    if (len <= short_len || chunk < 0 || chunk * kChunk >= len) return;
    const int64_t t0 = seq.start + chunk * kChunk;
    const int n = (int)min((int64_t)kChunk, seq.end - t0);
    const int b = threadIdx.x / 32, lane = threadIdx.x % 32;
    char *out = ws + kHeader + (slot * p.heads + h) * slot_bytes(D);

    // ---- load; rows past the sequence's end are k = q = v = beta = 0, decay 1
    float k[8][C], q[8][C], a[8][C];
    Vec<T, C> vraw[8];
    {
        float neg_a = 0.0f, bias[C] = {};
        if (p.gate_kind == KDA_GATE_SOFTPLUS) {
            neg_a = -expf(p.a_log[h]);
            if (p.dt_bias != nullptr)
#pragma unroll
                for (int c = 0; c < C; ++c)
                    bias[c] = kChannelGate ? p.dt_bias[h * D + lane * C + c] : p.dt_bias[h];
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const int64_t t = t0 + b * 8 + r;
            const bool in = b * 8 + r < n;
            if (in) {
                const auto kv = ld_vec<T, C>(static_cast<const T *>(p.k) + t * p.ks[0] + h * p.ks[1] + lane * C);
                const auto qv = ld_vec<T, C>(static_cast<const T *>(p.q) + t * p.qs[0] + h * p.qs[1] + lane * C);
                vraw[r] = ld_vec<T, C>(static_cast<const T *>(p.v) + t * p.vs[0] + h * p.vs[1] + lane * C);
                if constexpr (kChannelGate) {
                    const auto gv = ld_vec<G, C>(static_cast<const G *>(p.gate) + t * p.gs[0] + h * p.gs[1] + lane * C);
#pragma unroll
                    for (int c = 0; c < C; ++c) a[r][c] = to_f<G>(gv.v[c]);
                } else {
                    const float one = ld_dyn(p.gate, t * p.gs[0] + h * p.gs[1], p.gate_dtype);
#pragma unroll
                    for (int c = 0; c < C; ++c) a[r][c] = one;
                }
#pragma unroll
                for (int c = 0; c < C; ++c) k[r][c] = to_f<T>(kv.v[c]), q[r][c] = to_f<T>(qv.v[c]);
            } else {
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    k[r][c] = q[r][c] = a[r][c] = 0.0f;
                    vraw[r].v[c] = from_f<T>(0.0f);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < 8; ++r)
#pragma unroll
            for (int c = 0; c < C; ++c)
                a[r][c] = b * 8 + r < n ? decay_of(a[r][c], p.gate_kind, neg_a, bias[c]) : 1.0f;
    }
    if (lane < 8) {
        const int64_t t = t0 + b * 8 + lane;
        sm.beta[b * 8 + lane] =
            b * 8 + lane < n ? beta_of(ld_dyn(p.beta, t * p.bs[0] + h * p.bs[1], p.beta_dtype), p.beta_kind) : 0.0f;
    }
    {
        uint32_t mk = 0, mq = 0, mv = 0;
        float whole[C];
#pragma unroll
        for (int c = 0; c < C; ++c) whole[c] = 1.0f;
#pragma unroll
        for (int r = 0; r < 8; ++r)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                mk = max(mk, mag(k[r][c])), mq = max(mq, mag(q[r][c]));
                mv = max(mv, mag(to_f<T>(vraw[r].v[c])));
                whole[c] *= a[r][c];
            }
        mk = __reduce_max_sync(0xffffffffu, mk);
        mq = __reduce_max_sync(0xffffffffu, mq);
        mv = __reduce_max_sync(0xffffffffu, mv);
        if (lane == 0) sm.top[0][b] = mk, sm.top[1][b] = mq, sm.top[2][b] = mv;
#pragma unroll
        for (int c = 0; c < C; ++c) sm.block_decay[b][lane * C + c] = whole[c];
    }
    // L and A start as zeros (L's upper part is read by the block products).
    for (int i = threadIdx.x; i < 64 * 68; i += 256) (&sm.l.L[0][0])[i] = 0.0f, (&sm.T[0][0])[i] = 0.0f;
    for (int i = threadIdx.x; i < 64 * 72 / 2; i += 256) reinterpret_cast<uint32_t *>(&sm.A[0][0])[i] = 0;
    __syncthreads();
    const float top_k = top_of(sm.top[0]), top_q = top_of(sm.top[1]), top_v = top_of(sm.top[2]);
    const float up_k = scale_up(top_k), up_q = scale_up(top_q), up_v = scale_up(top_v);
    const float down_k = scale_down(top_k), down_q = scale_down(top_q), down_v = scale_down(top_v);
    // |A| < 2^(e_q + e_k + 9), so A up_q up_k 2^-22 is below 2^15.
    const float up_a = up_q * 0x1p-11f, up_a2 = up_k * 0x1p-11f;

    // ---- pairs inside 8 tokens: running products of decays, FP32
    {
        const int at = lane;
        const int i = 1 + (at >= 1) + (at >= 3) + (at >= 6) + (at >= 10) + (at >= 15) + (at >= 21);
        const int j = at - i * (i - 1) / 2;
        float f[32];
#pragma unroll
        for (int jj = 0; jj < 8; ++jj) {
            float w[C];
#pragma unroll
            for (int c = 0; c < C; ++c) w[c] = k[jj][c];
#pragma unroll
            for (int ii = jj + 1; ii < 8; ++ii) {
                float sum = 0.0f;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    w[c] *= a[ii][c];
                    sum = fmaf(k[ii][c], w[c], sum);
                }
                f[ii * (ii - 1) / 2 + jj] = sum;
            }
        }
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            f[28 + d] = 0.0f;
#pragma unroll
            for (int c = 0; c < C; ++c) f[28 + d] = fmaf(q[d][c], k[d][c], f[28 + d]);
        }
        float got = scatter_sum(f, lane);
        if (lane < 28) sm.l.L[b * 8 + i][b * 8 + j] = got * sm.beta[b * 8 + i];
        else sm.A[b * 8 + lane - 28][b * 8 + lane - 28] = __float2half_rn(got * up_a * up_a2);
#pragma unroll
        for (int jj = 0; jj < 8; ++jj) {
            float w[C];
#pragma unroll
            for (int c = 0; c < C; ++c) w[c] = k[jj][c];
#pragma unroll
            for (int ii = jj + 1; ii < 8; ++ii) {
                float sum = 0.0f;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    w[c] *= a[ii][c];
                    sum = fmaf(q[ii][c], w[c], sum);
                }
                f[ii * (ii - 1) / 2 + jj] = sum;
            }
        }
#pragma unroll
        for (int d = 4; d < 8; ++d) {
            f[24 + d] = 0.0f;
#pragma unroll
            for (int c = 0; c < C; ++c) f[24 + d] = fmaf(q[d][c], k[d][c], f[24 + d]);
        }
        got = scatter_sum(f, lane) * up_a * up_a2;
        if (lane < 28) sm.A[b * 8 + i][b * 8 + j] = __float2half_rn(got);
        else sm.A[b * 8 + lane - 24][b * 8 + lane - 24] = __float2half_rn(got);
    }

#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
        for (int c = 0; c < C; ++c) k[r][c] *= up_k, q[r][c] *= up_q;

    // ---- pairs of blocks: per level, the later half's tokens carry the decays
    // from the middle to them, the earlier half's those from them to the middle
    const int g = lane / 4, cc = lane % 4 * 2;
#pragma unroll 1
    for (int half = 1; half <= 4; half *= 2) {  // blocks of 8 in half a level: 1, 2, 4
        const int pos = b % (2 * half);         // block's place in its level group
        const int row0 = b / (2 * half) * (half * 8) + (pos % half) * 8;
        float run[C];
#pragma unroll
        for (int c = 0; c < C; ++c) run[c] = 1.0f;
        if (pos >= half) {
            for (int o = half; o < pos; ++o)
#pragma unroll
                for (int c = 0; c < C; ++c) run[c] *= sm.block_decay[b - pos + o][lane * C + c];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                float f[C], fq[C];
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    run[c] *= a[r][c];
                    f[c] = k[r][c] * run[c];
                    fq[c] = q[r][c] * run[c];
                }
                store_split<C>(&sm.x.lv.lk_hi[row0 + r][lane * C], &sm.x.lv.lk_lo[row0 + r][lane * C], f);
                store_row<C>(&sm.x.lv.lq[row0 + r][lane * C], fq);
            }
        } else {
            for (int o = pos + 1; o < half; ++o)
#pragma unroll
                for (int c = 0; c < C; ++c) run[c] *= sm.block_decay[b - pos + o][lane * C + c];
#pragma unroll
            for (int r = 7; r >= 0; --r) {
                float f[C];
#pragma unroll
                for (int c = 0; c < C; ++c) f[c] = k[r][c] * run[c], run[c] *= a[r][c];
                store_split<C>(&sm.x.lv.rk_hi[row0 + r][lane * C], &sm.x.lv.rk_lo[row0 + r][lane * C], f);
            }
        }
        __syncthreads();
        // kk by hi hi + hi lo + lo hi, qk by hi hi
        if (half == 1) {
            if (b < 4) {  // pair b: rows of k in the tile's first 8 rows, of q in the others
                float c[4] = {};
                const int lr = lane % 8, piece = lane / 8;
                const __half *top = (piece & 1) ? sm.x.lv.lq[b * 8 + lr] : sm.x.lv.lk_hi[b * 8 + lr];
                const __half *low = sm.x.lv.lk_lo[b * 8 + lr];
                const int br = b * 8 + lane % 8, bk = (lane / 8 % 2) * 8;
#pragma unroll
                for (int kk = 0; kk < D; kk += 16) {
                    uint32_t ah[4], al[4], bh[2], bl[2];
                    ldsm4(ah, smem_u32(top + kk + (piece >> 1) * 8));
                    ldsm4(al, smem_u32(low + kk + (piece >> 1) * 8));
                    ldsm2(bh, smem_u32(&sm.x.lv.rk_hi[br][kk + bk]));
                    ldsm2(bl, smem_u32(&sm.x.lv.rk_lo[br][kk + bk]));
                    al[1] = al[3] = 0;
                    mma16(c, ah, bh);
                    mma16(c, al, bh);
                    ah[1] = ah[3] = 0;
                    mma16(c, ah, bl);
                }
                const int i = b * 16 + 8 + g, j = b * 16 + cc;
                const float f = sm.beta[i];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    sm.l.L[i][j + e] = c[e] * down_k * down_k * f;
                    sm.A[i][j + e] = __float2half_rn(c[2 + e] * 0x1p-22f);
                }
            }
        } else {
            const bool wide = half == 4;
            const int m = wide ? b / 4 : b / 4;               // 16-row tile of the left operand
            const int nt = wide ? b % 4 : m * 2 + b / 2 % 2;  // 8-row tile of the right operand
            const bool do_k = wide || b % 2 == 0, do_q = wide || b % 2 == 1;
            float ck[4] = {}, cq[4] = {};
            const int ar = m * 16 + lane % 16, ak = lane / 16 * 8;
            const int br = nt * 8 + lane % 8, bk = (lane / 8 % 2) * 8;
#pragma unroll
            for (int kk = 0; kk < D; kk += 16) {
                uint32_t ah[4], bh[2];
                ldsm2(bh, smem_u32(&sm.x.lv.rk_hi[br][kk + bk]));
                if (do_k) {
                    uint32_t al[4], bl[2];
                    ldsm4(ah, smem_u32(&sm.x.lv.lk_hi[ar][kk + ak]));
                    ldsm4(al, smem_u32(&sm.x.lv.lk_lo[ar][kk + ak]));
                    ldsm2(bl, smem_u32(&sm.x.lv.rk_lo[br][kk + bk]));
                    mma16(ck, ah, bh);
                    mma16(ck, al, bh);
                    mma16(ck, ah, bl);
                }
                if (do_q) {
                    ldsm4(ah, smem_u32(&sm.x.lv.lq[ar][kk + ak]));
                    mma16(cq, ah, bh);
                }
            }
            // token rows and columns of the tile
            const int i0 = wide ? 32 + m * 16 : m * 32 + 16;
            const int j0 = wide ? nt * 8 : m * 32 + nt % 2 * 8;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = i0 + g + e / 2 * 8, j = j0 + cc + e % 2;
                if (do_k) sm.l.L[i][j] = ck[e] * down_k * down_k * sm.beta[i];
                if (do_q) sm.A[i][j] = __float2half_rn(cq[e] * 0x1p-22f);
            }
        }
        __syncthreads();
    }

    // ---- decays from the chunk's start (k G, q G) and to its end (k G_63 / G)
    {
        float run[C];
#pragma unroll
        for (int c = 0; c < C; ++c) run[c] = 1.0f;
        for (int o = 0; o < b; ++o)
#pragma unroll
            for (int c = 0; c < C; ++c) run[c] *= sm.block_decay[o][lane * C + c];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            float f[C], fq[C], fv[C];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                run[c] *= a[r][c];
                f[c] = k[r][c] * run[c];
                fq[c] = q[r][c] * run[c];
                fv[c] = to_f<T>(vraw[r].v[c]) * up_v;
            }
            const int row = b * 8 + r;
            store_split<C>(&sm.x.kg.k_hi[row][lane * C], &sm.x.kg.k_lo[row][lane * C], f);
            store_row<C>(&sm.v[row][lane * C], fv);
            store_row<C>(reinterpret_cast<__half *>(out + Slot<D>::q + image_at(row, lane * C, 64)), fq);
        }
#pragma unroll
        for (int c = 0; c < C; ++c) run[c] = 1.0f;
        for (int o = b + 1; o < 8; ++o)
#pragma unroll
            for (int c = 0; c < C; ++c) run[c] *= sm.block_decay[o][lane * C + c];
        uint32_t kh[C][4], kl[C][4];
#pragma unroll
        for (int r = 6; r >= 0; r -= 2)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const float later = k[r + 1][c] * run[c];
                run[c] *= a[r + 1][c];
                const float earlier = k[r][c] * run[c];
                run[c] *= a[r][c];
                split2(earlier, later, kh[c][r / 2], kl[c][r / 2]);
            }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int at = image_at(lane * C + c, b * 8, D);
            *reinterpret_cast<uint4 *>(out + Slot<D>::k_hi + at) = make_uint4(kh[c][0], kh[c][1], kh[c][2], kh[c][3]);
            *reinterpret_cast<uint4 *>(out + Slot<D>::k_lo + at) = make_uint4(kl[c][0], kl[c][1], kl[c][2], kl[c][3]);
        }
        if (b == 0)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float whole = 1.0f;
                for (int o = 0; o < 8; ++o) whole *= sm.block_decay[o][lane * C + c];
                reinterpret_cast<float *>(out + Slot<D>::decay)[lane * C + c] = whole;
            }
        // A: 64 x 64 halves, two 16-byte pieces per thread
        for (int i = threadIdx.x; i < 64 * 8; i += 256)
            *reinterpret_cast<uint4 *>(out + Slot<D>::a + image_at(i / 8, i % 8 * 8, 64)) =
                *reinterpret_cast<const uint4 *>(&sm.A[i / 8][i % 8 * 8]);
    }

    // ---- T = (I + L)^-1: 16 x 16 diagonal blocks by forward substitution (a
    // column per lane), the others from T_IJ = -T_II sum_M L_IM T_MJ
    if (b < 4 && lane < 16) {
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float sum = 0.0f;
#pragma unroll
            for (int m = 0; m < i; ++m) sum = fmaf(sm.l.L[b * 16 + i][b * 16 + m], x[m], sum);
            x[i] = (i == lane ? 1.0f : 0.0f) - sum;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) sm.T[b * 16 + i][b * 16 + lane] = x[i];
    }
    __syncthreads();
    {
        const int i = threadIdx.x / 16, j = threadIdx.x % 16;
#pragma unroll 1
        for (int dist = 1; dist < 4; ++dist) {
            for (int J = 0; J + dist < 4; ++J) {
                const int I = J + dist;
                float sum = 0.0f;
                for (int m = J * 16; m < I * 16; ++m) sum = fmaf(sm.l.L[I * 16 + i][m], sm.T[m][J * 16 + j], sum);
                sm.tmp[J][i][j] = sum;
            }
            __syncthreads();
            for (int J = 0; J + dist < 4; ++J) {
                const int I = J + dist;
                float sum = 0.0f;
#pragma unroll
                for (int m = 0; m < 16; ++m) sum = fmaf(sm.T[I * 16 + i][I * 16 + m], sm.tmp[J][m][j], sum);
                sm.T[I * 16 + i][J * 16 + j] = -sum;
            }
            __syncthreads();
        }
    }

    // ---- W = T diag(beta) k G and U = T diag(beta) v
    {
        float t[16];
        uint32_t m = 0;
        const int row = threadIdx.x / 4, col = threadIdx.x % 4 * 16;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            t[i] = sm.T[row][col + i] * sm.beta[col + i];
            m = max(m, mag(t[i]));
        }
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) sm.top[3][b] = m;
        __syncthreads();  // also: nobody reads L any more
        const float up_t = scale_up(top_of(sm.top[3]));
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            uint32_t hi, lo;
            split2(t[i] * up_t, t[i + 1] * up_t, hi, lo);
            *reinterpret_cast<uint32_t *>(&sm.l.t.hi[row][col + i]) = hi;
            *reinterpret_cast<uint32_t *>(&sm.l.t.lo[row][col + i]) = lo;
        }
    }
    __syncthreads();
    const float down_t = scale_down(top_of(sm.top[3]));
    constexpr int NT = D / 64;  // 8-column tiles of a warp
    const int ar = lane % 16, ak = lane / 16 * 8;
    float acc[4][NT][4] = {};
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
        uint32_t bh[NT][2], bl[NT][2];
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            ldsm2t(bh[x], smem_u32(&sm.x.kg.k_hi[ks * 16 + ar][(b * NT + x) * 8]));
            ldsm2t(bl[x], smem_u32(&sm.x.kg.k_lo[ks * 16 + ar][(b * NT + x) * 8]));
        }
#pragma unroll
        for (int m = ks; m < 4; ++m) {
            uint32_t ah[4], al[4];
            ldsm4(ah, smem_u32(&sm.l.t.hi[m * 16 + ar][ks * 16 + ak]));
            ldsm4(al, smem_u32(&sm.l.t.lo[m * 16 + ar][ks * 16 + ak]));
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                mma16(acc[m][x], ah, bh[x]);
                mma16(acc[m][x], al, bh[x]);
                mma16(acc[m][x], ah, bl[x]);
            }
        }
    }
    {
        uint32_t top = 0;
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int x = 0; x < NT; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    acc[m][x][e] = acc[m][x][e] * down_t * down_k;
                    top = max(top, mag(acc[m][x][e]));
                }
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) sm.top[0][b] = top;
    }
    float acu[4][NT][4] = {};
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
        uint32_t bh[NT][2];
#pragma unroll
        for (int x = 0; x < NT; ++x) ldsm2t(bh[x], smem_u32(&sm.v[ks * 16 + ar][(b * NT + x) * 8]));
#pragma unroll
        for (int m = ks; m < 4; ++m) {
            uint32_t ah[4], al[4];
            ldsm4(ah, smem_u32(&sm.l.t.hi[m * 16 + ar][ks * 16 + ak]));
            ldsm4(al, smem_u32(&sm.l.t.lo[m * 16 + ar][ks * 16 + ak]));
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                mma16(acu[m][x], ah, bh[x]);
                mma16(acu[m][x], al, bh[x]);
            }
        }
    }
    __syncthreads();
    const float top_w = top_of(sm.top[0]);
    const float up_w = scale_up(top_w);
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const int row = m * 16 + g + e * 4, col = (b * NT + x) * 8 + cc;
                uint32_t hi, lo;
                split2(acc[m][x][e] * up_w, acc[m][x][e + 1] * up_w, hi, lo);
                const int at = image_at(row, col, 64);
                *reinterpret_cast<uint32_t *>(out + Slot<D>::w_hi + at) = hi;
                *reinterpret_cast<uint32_t *>(out + Slot<D>::w_lo + at) = lo;
                *reinterpret_cast<float2 *>(out + Slot<D>::u + (row * D + col) * 4) =
                    make_float2(acu[m][x][e] * down_t * down_v, acu[m][x][e + 1] * down_t * down_v);
            }
    if (threadIdx.x == 0) {
        float *f = reinterpret_cast<float *>(out + Slot<D>::scales);
        f[0] = scale_down(top_w);
        f[1] = down_k;
        f[2] = down_q;
        f[3] = 0x1p11f * down_q;  // A: times 2^11 down_k
        f[4] = 0x1p11f * down_k;
    }
}

// ------------------------------------------------------------------ barriers

// Every wait ends: after kWaitTries polls it gives up and sets `abort`, which
// ends the other waits of the block too.
constexpr int kWaitTries = 1 << 20;

__device__ __forceinline__ void bar_init(uint32_t bar, int count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
                 "selp.u32 %0, 1, 0, p;\n}" : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int *abort) {
    for (int i = 0; i < kWaitTries; ++i) {
        if (bar_test(bar, parity)) return true;
        if ((i & 63) == 63 && *abort != 0) return false;
    }
    *abort = 1;
    return false;
}
// The 256 threads of the compute warps meet; true if any of them brings true.
__device__ __forceinline__ bool meet_any(bool bad) {
    uint32_t r;
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbarrier.cta.red.or.pred q, 1, 256, p;\n"
                 "selp.u32 %0, 1, 0, q;\n}" : "=r"(r) : "r"((uint32_t)bad) : "memory");
    return r != 0;
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

// ------------------------------------------------------------------ tcgen05

__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// 16 consecutive 32-bit columns of the warp's 32 lanes.
__device__ __forceinline__ void tc_ld16(uint32_t (&r)[16], uint32_t at) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(at));
}
__device__ __forceinline__ void tc_st16(uint32_t at, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                   "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}

// Descriptor of an operand image in shared memory: K-major, 128-byte swizzle,
// 8-row groups 1024 bytes apart (bit 46: the descriptor's version).
__device__ __forceinline__ uint64_t operand_desc(uint32_t at) {
    return (uint64_t)((at & 0x3ffff) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// fp16 x fp16 -> fp32, both K-major, 128 x N.
__host__ __device__ constexpr uint32_t instr_desc(int N) {
    return 1u << 4 | (uint32_t)(N >> 3) << 17 | (uint32_t)(128 >> 4) << 24;
}
// D[128 x N] (+)= A[128 x 16] B[N x 16]^T, A in TMEM.
__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile("{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
                 ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add) : "memory");
}

// ------------------------------------------------------------------ walk

// What a walk does: write outputs and final states, or the two summaries of a
// segment (its end state from zero or from the cached state, and from the identity).
enum { kWalkOut = 0, kWalkSummary = 1 };

template <int D, int kMode>
struct WalkSmem {
    static constexpr int kStages = 2;
    static constexpr bool kOut = kMode == kWalkOut;
    static constexpr int kKStages = kOut ? 1 : 2;
    alignas(1024) char w[kStages][2 * Slot<D>::kW];  // hi, lo
    char kk[kKStages][2 * Slot<D>::kW];
    char q[kOut ? kStages : 1][kOut ? Slot<D>::kW : 1024];
    char a[kOut ? 8192 : 1024];
    float u[kStages][kChunk * D];
    float meta[kStages][D + 16];  // G_63 and the scales of the chunk
    float top[2][2][128];         // row maxima of the two halves: of S, of V'
    float row_scale[2][2][128];   // unscaling of S and V' rows, for the outputs
    uint64_t bars[24];
    int abort;
    uint32_t tmem;
};

enum {
    kWFull = 0, kWEmpty = 2, kKFull = 4, kKEmpty = 6, kQFull = 8, kQEmpty = 10, kUFull = 12, kUEmpty = 14,
    kAFull = 16, kAEmpty = 17, kSReady = 18, kPDone = 19, kVReady = 20, kDDone = 21, kODone = 22, kOFree = 23
};

// TMEM columns (D = 128): hi and lo of S, P, o's two parts, hi and lo of V', the state's update.
template <int D>
struct Cols {
    static constexpr int s_hi = 0, s_lo = D / 2, p = D, o1 = D + 64, v_hi = D + 128, v_lo = D + 160,
                         d = D + 192, o2 = 2 * D + 192;  // + 64 = 2 D + 256 <= 512
};

struct WalkArgs {
    char *ws;
    float *summary;        // [segment slot][head][2][D][D]: B, M
    float *first;          // [segment slot][head][D][D]: the state a later segment starts from
    int64_t seg_tokens;    // tokens of a segment (a multiple of 64)
    int short_len;
    int split;             // segments are searched for; 0: item = sequence
};

constexpr int kWalkThreads = 448;  // 8 compute warps, 4 output warps, a tensor-core warp, a copy warp

// Rows of `values` of one group scaled to halves: hi and lo packed pairs.
template <int N>
__device__ __forceinline__ float max_abs(const float (&f)[N]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, fabsf(f[i]));
    return m;
}

template <typename T, int D, int kMode>
__global__ void __launch_bounds__(kWalkThreads, 1)
    delta_walk_kernel(const __grid_constant__ DeltaParams p, const __grid_constant__ WalkArgs w) {
    using Sm = WalkSmem<D, kMode>;
    using Col = Cols<D>;
    constexpr bool kOut = kMode == kWalkOut;
    constexpr int H = D / 2;  // state columns of a thread
    extern __shared__ __align__(1024) char raw_smem[];
    // The operand images start on 1024 bytes (the swizzle's period).
    Sm &sm = *reinterpret_cast<Sm *>(raw_smem + ((1024 - (smem_u32(raw_smem) & 1023)) & 1023));
    dependency_wait();

    // ---- the segment
    const int which = kOut ? 0 : blockIdx.x % 2;  // summary: 0 the state's part (B), 1 the identity's (M)
    const int64_t item = blockIdx.x / (kOut ? 1 : 2);
    const int64_t seg_slot = item / p.heads;
    const int h = item % p.heads;
    int64_t seg = 0;
    const int s = w.split ? find_seq(p, seg_slot, w.seg_tokens, seg) : (int)seg_slot;
    const Seq seq = load_seq(p, s);
    const int64_t len = seq.end - seq.start;
    if (len <= w.short_len || seg < 0 || seg * w.seg_tokens >= len) return;
    const bool last_seg = (seg + 1) * w.seg_tokens >= len;
    // A sequence's last segment is never summarised, its first has no use for M.
    if (!kOut && (last_seg || (which == 1 && seg == 0))) return;
    const int64_t begin = seq.start + seg * w.seg_tokens;
    const int64_t stop = last_seg ? seq.end : begin + w.seg_tokens;
    const int chunks = (int)((stop - begin + kChunk - 1) / kChunk);
    const char *slots = w.ws + kHeader +
        ((seq.start / kChunk + s + seg * (w.seg_tokens / kChunk)) * p.heads + h) * slot_bytes(D);
    const int64_t slot_step = (int64_t)p.heads * slot_bytes(D);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t bars = smem_u32(sm.bars);
    volatile int *abort = &sm.abort;
    auto bar = [&](int i) { return bars + i * 8; };

    if (threadIdx.x == 0) {
        for (int i = 0; i < 24; ++i) {
            int count = 1;
            if (i == kSReady || i == kVReady) count = 8;
            if (i == kUEmpty || i == kUEmpty + 1) count = kOut ? 12 : 8;
            if (i == kOFree) count = 4;
            bar_init(bar(i), count);
        }
        sm.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sm.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = sm.tmem;

    if (warp < 8) {
        // ---- compute warps: row v of the state, columns [half * H, half * H + H)
        const int half = warp / 4, v = warp % 4 * 32 + lane;
        const uint32_t mine = tmem + ((uint32_t)(warp % 4 * 32) << 16);
        const bool row_in = v < D;
        float S[H];
#pragma unroll
        for (int i = 0; i < H; ++i) S[i] = 0.0f;
        if (row_in) {
            const float *from = nullptr;
            if (kOut && !(seg == 0 && last_seg)) from = w.first + ((seg_slot * p.heads + h) * D + v) * D;
            else if (which == 0 && seg == 0 && seq.reads) from = p.states + seq.line * p.ss[0] + h * p.ss[1] + v * D;
            if (from != nullptr) {
#pragma unroll
                for (int i = 0; i < H; i += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(from + half * H + i);
                    S[i] = f.x, S[i + 1] = f.y, S[i + 2] = f.z, S[i + 3] = f.w;
                }
            } else if (which == 1) {
#pragma unroll
                for (int i = 0; i < H; ++i) S[i] = half * H + i == v ? 1.0f : 0.0f;
            }
        }
        bool bad = false;
        for (int c = 0; c < chunks; ++c) {
            const uint32_t par = c & 1, ring = c >> 1 & 1;
            // S as halves
            sm.top[0][half][v] = max_abs(S);
            if (meet_any(bad)) { bad = true; break; }
            const float top_s = fmaxf(sm.top[0][0][v], sm.top[0][1][v]);
            const float up_s = scale_up(top_s), down_s = scale_down(top_s);
#pragma unroll
            for (int i = 0; i < H; i += 32) {
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) split2(S[i + 2 * j] * up_s, S[i + 2 * j + 1] * up_s, hi[j], lo[j]);
                tc_st16(mine + Col::s_hi + (half * H + i) / 2, hi);
                tc_st16(mine + Col::s_lo + (half * H + i) / 2, lo);
            }
            if (kOut && half == 0) sm.row_scale[0][par][v] = down_s;
            tc_wait_st();
            tc_before();
            __syncwarp();
            if (lane == 0) bar_arrive(bar(kSReady));
            // V' = U - W S^T: this thread's 32 tokens
            bad = !bar_wait(bar(kUFull + par), ring, abort) || !bar_wait(bar(kPDone), par, abort);
            tc_after();
            const float *meta = sm.meta[par];
            const float down_p = meta[D], down_k = meta[D + 1];
            float V[32];
            {
                uint32_t r0[16], r1[16];
                tc_ld16(r0, mine + Col::p + half * 32);
                tc_ld16(r1, mine + Col::p + half * 32 + 16);
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    V[j] = __uint_as_float(r0[j]) * down_p * down_s;
                    V[16 + j] = __uint_as_float(r1[j]) * down_p * down_s;
                }
            }
            const bool uses_u = (kOut || which == 0) && row_in;
#pragma unroll
            for (int j = 0; j < 32; ++j) V[j] = (uses_u ? sm.u[par][(half * 32 + j) * D + v] : 0.0f) - V[j];
            sm.top[1][half][v] = max_abs(V);
            if (kOut && c > 0) bad |= !bar_wait(bar(kODone), (c - 1) & 1, abort);  // V' of the last chunk is still read
            if (meet_any(bad)) { bad = true; break; }
            const float top_v = fmaxf(sm.top[1][0][v], sm.top[1][1][v]);
            const float up_v = scale_up(top_v), down_v = scale_down(top_v);
            {
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) split2(V[2 * j] * up_v, V[2 * j + 1] * up_v, hi[j], lo[j]);
                tc_st16(mine + Col::v_hi + half * 16, hi);
                tc_st16(mine + Col::v_lo + half * 16, lo);
            }
            if (kOut && half == 0) sm.row_scale[1][par][v] = down_v;
            tc_wait_st();
            tc_before();
            __syncwarp();
            if (lane == 0) bar_arrive(bar(kVReady));
            // S = S diag(G_63) + V'^T (k G_63 / G)
            bad = !bar_wait(bar(kDDone), par, abort);
            tc_after();
#pragma unroll
            for (int i = 0; i < H; i += 16) {
                uint32_t r[16];
                tc_ld16(r, mine + Col::d + half * H + i);
                float4 gs[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) gs[j] = *reinterpret_cast<const float4 *>(meta + half * H + i + 4 * j);
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    S[i + 4 * j] = fmaf(S[i + 4 * j], gs[j].x, __uint_as_float(r[4 * j]) * down_k * down_v);
                    S[i + 4 * j + 1] = fmaf(S[i + 4 * j + 1], gs[j].y, __uint_as_float(r[4 * j + 1]) * down_k * down_v);
                    S[i + 4 * j + 2] = fmaf(S[i + 4 * j + 2], gs[j].z, __uint_as_float(r[4 * j + 2]) * down_k * down_v);
                    S[i + 4 * j + 3] = fmaf(S[i + 4 * j + 3], gs[j].w, __uint_as_float(r[4 * j + 3]) * down_k * down_v);
                }
            }
            __syncwarp();
            if (lane == 0) bar_arrive(bar(kUEmpty + par));  // U and the chunk's scales are read
        }
        bad = meet_any(bad);
        if (!bad && row_in) {
            float *to = nullptr;
            if (!kOut) to = w.summary + (((seg_slot * p.heads + h) * 2 + which) * D + v) * D;
            else if (last_seg && seq.line >= 0) to = p.states + seq.line * p.ss[0] + h * p.ss[1] + v * D;
            if (to != nullptr)
#pragma unroll
                for (int i = 0; i < H; i += 4)
                    *reinterpret_cast<float4 *>(to + half * H + i) = make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
        }
    } else if (warp < 12) {
        // ---- output warps: row v, all tokens of the chunk
        if constexpr (kOut) {
            const int v = warp % 4 * 32 + lane;
            const uint32_t mine = tmem + ((uint32_t)(warp % 4 * 32) << 16);
            T *out = static_cast<T *>(p.out) + h * p.os[1] + v;
            for (int c = 0; c < chunks; ++c) {
                const uint32_t par = c & 1, ring = c >> 1 & 1;
                // The copy of the chunk's scales is visible only to who has waited for it.
                if (!bar_wait(bar(kUFull + par), ring, abort) || !bar_wait(bar(kODone), par, abort)) break;
                tc_after();
                const float *meta = sm.meta[par];
                const float f1 = meta[D + 2], f2 = meta[D + 3], f3 = meta[D + 4];
                const float ds = sm.row_scale[0][par][v], dv = sm.row_scale[1][par][v];
                float o[64];
#pragma unroll
                for (int i = 0; i < 64; i += 16) {
                    uint32_t r[16], x[16];
                    tc_ld16(r, mine + Col::o1 + i);
                    tc_ld16(x, mine + Col::o2 + i);
                    tc_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        o[i + j] = p.scale * (__uint_as_float(r[j]) * f1 * ds + __uint_as_float(x[j]) * f2 * f3 * dv);
                }
                tc_before();
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(bar(kOFree));
                    bar_arrive(bar(kUEmpty + par));
                }
                const int64_t t0 = begin + (int64_t)c * kChunk;
                const int n = (int)min((int64_t)kChunk, stop - t0);
                if (v < D) {
#pragma unroll
                    for (int j = 0; j < 64; ++j)
                        if (j < n) out[(t0 + j) * p.os[0]] = from_f<T>(o[j]);
                }
            }
        }
    } else if (warp == 12) {
        // ---- tensor-core warp
        if (lane == 0) {
            constexpr uint32_t id_n64 = instr_desc(64), id_d = instr_desc(D);
            for (int c = 0; c < chunks; ++c) {
                const uint32_t par = c & 1, ring = c >> 1 & 1;
                const uint32_t kst = Sm::kKStages == 2 ? par : 0, kring = Sm::kKStages == 2 ? ring : par;
                if (!bar_wait(bar(kWFull + par), ring, abort) || !bar_wait(bar(kSReady), par, abort)) break;
                tc_after();
                {
                    const uint32_t hi = smem_u32(sm.w[par]), lo = hi + Slot<D>::kW;
#pragma unroll
                    for (int i = 0; i < 3 * (D / 16); ++i) {
                        const int k = i % (D / 16), term = i / (D / 16);  // hi hi, hi lo, lo hi
                        const uint32_t b = (term == 1 ? lo : hi) + k / 4 * 8192 + k % 4 * 32;
                        tc_mma(tmem + Col::p, tmem + (term == 2 ? Col::s_lo : Col::s_hi) + k * 8, operand_desc(b),
                               id_n64, i != 0);
                    }
                }
                tc_commit(bar(kPDone));
                tc_commit(bar(kWEmpty + par));
                if (kOut) {
                    if (!bar_wait(bar(kQFull + par), ring, abort)) break;
                    if (c > 0 && !bar_wait(bar(kOFree), (c - 1) & 1, abort)) break;
                    tc_after();
                    const uint32_t q = smem_u32(sm.q[par]);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        tc_mma(tmem + Col::o1, tmem + Col::s_hi + k * 8, operand_desc(q + k / 4 * 8192 + k % 4 * 32),
                               id_n64, k != 0);
                    tc_commit(bar(kQEmpty + par));
                }
                if (!bar_wait(bar(kKFull + kst), kring, abort) || !bar_wait(bar(kVReady), par, abort)) break;
                tc_after();
                {
                    const uint32_t hi = smem_u32(sm.kk[kst]), lo = hi + Slot<D>::kW;
#pragma unroll
                    for (int i = 0; i < 12; ++i) {
                        const int k = i % 4, term = i / 4;
                        tc_mma(tmem + Col::d, tmem + (term == 2 ? Col::v_lo : Col::v_hi) + k * 8,
                               operand_desc((term == 1 ? lo : hi) + k * 32), id_d, i != 0);
                    }
                }
                tc_commit(bar(kDDone));
                tc_commit(bar(kKEmpty + kst));
                if (kOut) {
                    if (!bar_wait(bar(kAFull), par, abort)) break;
                    const uint32_t a = smem_u32(sm.a);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc_mma(tmem + Col::o2, tmem + Col::v_hi + k * 8, operand_desc(a + k * 32), id_n64, k != 0);
                    tc_commit(bar(kODone));
                    tc_commit(bar(kAEmpty));
                }
            }
        }
    } else if (lane == 0) {
        // ---- copy warp
        for (int c = 0; c < chunks; ++c) {
            const uint32_t par = c & 1, ring = c >> 1 & 1;
            const uint32_t kst = Sm::kKStages == 2 ? par : 0, kring = Sm::kKStages == 2 ? ring : par;
            const bool k_reused = Sm::kKStages == 2 ? c >= 2 : c >= 1;
            const char *from = slots + c * slot_step;
            if (c >= 2 && !bar_wait(bar(kWEmpty + par), ring ^ 1, abort)) break;
            bar_expect(bar(kWFull + par), 2 * Slot<D>::kW);
            bulk_load(smem_u32(sm.w[par]), from + Slot<D>::w_hi, 2 * Slot<D>::kW, bar(kWFull + par));
            if (c >= 2 && !bar_wait(bar(kUEmpty + par), ring ^ 1, abort)) break;
            bar_expect(bar(kUFull + par), kChunk * D * 4 + D * 4 + 64);
            bulk_load(smem_u32(sm.u[par]), from + Slot<D>::u, kChunk * D * 4, bar(kUFull + par));
            bulk_load(smem_u32(sm.meta[par]), from + Slot<D>::decay, D * 4 + 64, bar(kUFull + par));
            if (kOut) {
                if (c >= 2 && !bar_wait(bar(kQEmpty + par), ring ^ 1, abort)) break;
                bar_expect(bar(kQFull + par), Slot<D>::kW);
                bulk_load(smem_u32(sm.q[par]), from + Slot<D>::q, Slot<D>::kW, bar(kQFull + par));
            }
            if (k_reused && !bar_wait(bar(kKEmpty + kst), kring ^ 1, abort)) break;
            bar_expect(bar(kKFull + kst), 2 * Slot<D>::kW);
            bulk_load(smem_u32(sm.kk[kst]), from + Slot<D>::k_hi, 2 * Slot<D>::kW, bar(kKFull + kst));
            if (kOut) {
                if (c >= 1 && !bar_wait(bar(kAEmpty), par ^ 1, abort)) break;
                bar_expect(bar(kAFull), kChunk * kChunk * 2);
                bulk_load(smem_u32(sm.a), from + Slot<D>::a, kChunk * kChunk * 2, bar(kAFull));
            }
        }
    }
    tc_before();
    __syncthreads();
    tc_after();
    if (sm.abort != 0) {
        // A wait ran out (never in a correct run): say so, and give the copies in
        // flight time to land before the block's shared memory is given back.
        if (threadIdx.x == 0) *reinterpret_cast<volatile int *>(w.ws) = 1;
        const long long t = clock64();
        while (clock64() - t < 20000000) {
        }
        __syncthreads();
    }
    __syncwarp();
    if (warp == 12)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// ------------------------------------------------------------------ join

// first[0] = the cached state (the walk of the last segment overwrites it),
// first[seg + 1] = (seg ? first[seg] M[seg] : 0) + B[seg], segment by segment:
// one block per (sequence, head, kJoinRows rows of the state), a column per thread.
constexpr int kJoinRows = 8;

template <int D>
__global__ void __launch_bounds__(D) delta_join_kernel(const __grid_constant__ DeltaParams p, const __grid_constant__ WalkArgs w) {
    __shared__ float row[kJoinRows][D];
    dependency_wait();
    const int s = blockIdx.x / p.heads, h = blockIdx.x % p.heads;
    const int r0 = blockIdx.y * kJoinRows, k = threadIdx.x;
    const Seq seq = load_seq(p, s);
    const int64_t len = seq.end - seq.start;
    if (len <= w.short_len || len <= w.seg_tokens) return;
    const int segs = (int)((len + w.seg_tokens - 1) / w.seg_tokens);
    const int64_t base = seq.start / w.seg_tokens + s;
    float S[kJoinRows];
    {
        const float *from = p.states + (seq.reads ? seq.line : 0) * p.ss[0] + h * p.ss[1];
        float *to = w.first + (base * p.heads + h) * D * D;
#pragma unroll
        for (int r = 0; r < kJoinRows; ++r) to[(r0 + r) * D + k] = seq.reads ? from[(r0 + r) * D + k] : 0.0f;
    }
    for (int seg = 0; seg + 1 < segs; ++seg) {
        const int64_t at = (base + seg) * p.heads + h;
        const float *B = w.summary + at * 2 * D * D;
        float next[kJoinRows];
#pragma unroll
        for (int r = 0; r < kJoinRows; ++r) next[r] = B[(r0 + r) * D + k];
        if (seg > 0) {
            const float *M = B + D * D;
            __syncthreads();
#pragma unroll
            for (int r = 0; r < kJoinRows; ++r) row[r][k] = S[r];
            __syncthreads();
#pragma unroll 16
            for (int i = 0; i < D; ++i) {
                const float m = M[i * D + k];
#pragma unroll
                for (int r = 0; r < kJoinRows; ++r) next[r] = fmaf(row[r][i], m, next[r]);
            }
        }
        float *to = w.first + ((base + seg + 1) * p.heads + h) * D * D;
#pragma unroll
        for (int r = 0; r < kJoinRows; ++r) {
            S[r] = next[r];
            to[(r0 + r) * D + k] = next[r];
        }
    }
}

// ------------------------------------------------------------------ host

template <typename T, int D, bool kChannelGate, typename G>
cudaError_t launch_prepare(const DeltaParams &p, const ChunkPlan &plan, int short_len, char *ws, kda_stream_t stream) {
    auto *kernel = delta_prepare_kernel<T, D, kChannelGate, G>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(PrepSmem<D>));
    if (e != cudaSuccess) return e;
    return launch(kernel, dim3((unsigned)(plan.slots * p.heads)), 256, sizeof(PrepSmem<D>), stream, p, ws, short_len);
}

template <typename T, int D, int kMode>
cudaError_t launch_walk(const DeltaParams &p, const ChunkPlan &plan, const WalkArgs &w, kda_stream_t stream) {
    auto *kernel = delta_walk_kernel<T, D, kMode>;
    const size_t smem = sizeof(WalkSmem<D, kMode>) + 1024;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int64_t items = (plan.split ? plan.segments : p.num_seqs) * p.heads * (kMode == kWalkOut ? 1 : 2);
    return launch(kernel, dim3((unsigned)items), kWalkThreads, smem, stream, p, w);
}

template <typename T, int D>
cudaError_t run(const DeltaParams &p, const kda_delta_t *d, const ChunkPlan &plan, int short_len, char *ws,
                kda_stream_t stream) {
    cudaError_t e;
    if (!d->gate_per_channel) e = launch_prepare<T, D, false, float>(p, plan, short_len, ws, stream);
    else if (d->gate_dtype == KDA_DTYPE_F32) e = launch_prepare<T, D, true, float>(p, plan, short_len, ws, stream);
    else if (d->gate_dtype == KDA_DTYPE_BF16)
        e = launch_prepare<T, D, true, __nv_bfloat16>(p, plan, short_len, ws, stream);
    else e = launch_prepare<T, D, true, __half>(p, plan, short_len, ws, stream);
    if (e != cudaSuccess) return e;
    WalkArgs w = {};
    w.ws = ws;
    w.seg_tokens = (int64_t)plan.seg_chunks * kChunk;
    w.short_len = short_len;
    w.split = plan.split;
    if (plan.split) {
        w.summary = reinterpret_cast<float *>(ws + kHeader + plan.slots * p.heads * slot_bytes(D));
        w.first = w.summary + plan.segments * p.heads * 2 * D * D;
        e = launch_walk<T, D, kWalkSummary>(p, plan, w, stream);
        if (e != cudaSuccess) return e;
        e = launch(delta_join_kernel<D>, dim3((unsigned)(p.num_seqs * p.heads), D / kJoinRows), D, 0, stream, p, w);
        if (e != cudaSuccess) return e;
    }
    return launch_walk<T, D, kWalkOut>(p, plan, w, stream);
}

}  // namespace

ChunkPlan chunk_plan(int64_t tokens, int64_t num_seqs, int64_t heads, int head_dim, int sms) {
    ChunkPlan c = {};
    c.slots = tokens / kChunk + num_seqs;
    const int64_t chunks = (tokens + kChunk - 1) / kChunk;  // of one sequence, at most
    // One wave of segments if one sequence had all tokens, of at least 4 chunks.
    const int64_t parts = sms / heads > 1 ? sms / heads : 1;
    int64_t seg = (chunks + parts - 1) / parts;
    if (seg < 4) seg = 4;
    c.seg_chunks = (int)seg;
    c.split = chunks > seg;
    c.segments = c.split ? tokens / (seg * kChunk) + num_seqs : num_seqs;
    c.bytes = kHeader + c.slots * heads * slot_bytes(head_dim);
    if (c.split) c.bytes += c.segments * heads * 3 * head_dim * head_dim * 4;
    return c;
}

cudaError_t run_chunked(const DeltaParams &p, const kda_delta_t *d, const ChunkPlan &plan, int short_len,
                        void *ws, kda_stream_t stream) {
    char *base = static_cast<char *>(ws);
    if (d->x_dtype == KDA_DTYPE_BF16)
        return d->head_dim == 64 ? run<__nv_bfloat16, 64>(p, d, plan, short_len, base, stream)
                                 : run<__nv_bfloat16, 128>(p, d, plan, short_len, base, stream);
    return d->head_dim == 64 ? run<__half, 64>(p, d, plan, short_len, base, stream)
                             : run<__half, 128>(p, d, plan, short_len, base, stream);
}

}  // namespace kda_layer

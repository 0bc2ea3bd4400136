// The norms around a KDA block (include/kda_layer.h): the gated per-head RMS
// norm and the residual join.  Both read every element once and write every
// result once, so HBM bandwidth bounds them; nothing is contracted.
#include "kda_layer.cuh"

namespace kda_layer {

thread_local char g_error[256] = "";

char *error_buffer() { return g_error; }

kda_status_t cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return KDA_OK;
    snprintf(g_error, sizeof(g_error), "%s", cudaGetErrorString(e));
    (void)cudaGetLastError();
    return KDA_ERR_CUDA;
}

// SM count of the current device, kept per device (threads may race to fill an
// entry; they store the same value).
int current_sms() {
    static std::atomic<int> cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
    int n = cache[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
            n = 152;
        cache[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

namespace {

// The gate's factor. For a 16-bit gate the exponential and the reciprocal are the
// special-function unit's (relative error 2^-23 times the argument, below 2^-16
// where the factor is above e^-80): the accurate forms cost more issue slots than
// the loads and stores leave.
template <typename T, int kAct>
__device__ __forceinline__ float act_f(float z) {
    if constexpr (kAct == KDA_NORM_GATE_NONE) return 1.0f;
    float s;
    if constexpr (sizeof(T) == 2) {
        float e;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
    } else {
        s = sigmoid_f(z);
    }
    return kAct == KDA_NORM_GATE_SILU ? z * s : s;
}

struct GatedParams {
    const void *x, *gate;
    const float *weight;
    void *out;
    int64_t xs[2], gs[2], os[2];
    int64_t groups;  // rows * heads
    int heads;
    FastDiv heads_div;
    int vecs;  // 16-byte vectors per head
    float eps, inv_dim;
};

// kLanes neighbouring lanes own one (row, head); each holds kVpl vectors of it
// in registers, so x is read once and the sum of squares is a butterfly. A block
// takes kBatch times as many heads as it has groups of lanes, a block's width
// apart, with all their loads issued first: one head's two loads per thread leave
// too few bytes in flight (16384 x 12 x 128 bf16: 27.5 us, 5.50 TB/s; 34.8 with one).
template <typename T, int kLanes, int kVpl, int kBatch, int kAct>
__global__ void __launch_bounds__(256) gated_rmsnorm_kernel(const __grid_constant__ GatedParams p) {
    constexpr int N = 16 / sizeof(T), kPerBlock = 256 / kLanes;
    dependency_wait();
    const int lane = threadIdx.x % kLanes;
    const int64_t first = (int64_t)blockIdx.x * (kPerBlock * kBatch) + threadIdx.x / kLanes;
    Vec<T, N> xv[kBatch][kVpl], gv[kBatch][kVpl];
    auto at_of = [&](int b, const int64_t *s) {
        const int64_t group = min(first + b * kPerBlock, p.groups - 1);
        const int64_t row = fast_div((uint32_t)group, p.heads_div), head = group - row * p.heads;
        return row * s[0] + head * s[1];
    };
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
        const T *x = static_cast<const T *>(p.x) + at_of(b, p.xs);
        const T *gate = static_cast<const T *>(p.gate) + at_of(b, p.gs);
#pragma unroll
        for (int i = 0; i < kVpl; ++i) {
            const int at = min(lane + i * kLanes, p.vecs - 1);
            xv[b][i] = ld_stream<T, N>(x + at * N);
            if constexpr (kAct != KDA_NORM_GATE_NONE) gv[b][i] = ld_stream<T, N>(gate + at * N);
        }
    }
    float w[kVpl][N];
#pragma unroll
    for (int i = 0; i < kVpl; ++i)
#pragma unroll
        for (int j = 0; j < N; j += 4) {
            float4 f = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
            if (p.weight != nullptr)
                f = __ldg(reinterpret_cast<const float4 *>(p.weight + min(lane + i * kLanes, p.vecs - 1) * N + j));
            w[i][j] = f.x, w[i][j + 1] = f.y, w[i][j + 2] = f.z, w[i][j + 3] = f.w;
        }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kVpl; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float f = to_f<T>(xv[b][i].v[j]);
                if (lane + i * kLanes < p.vecs) sum = fmaf(f, f, sum);
            }
#pragma unroll
        for (int m = kLanes / 2; m > 0; m /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        const float inv = rsqrtf(fmaf(sum, p.inv_dim, p.eps));
        if (first + b * kPerBlock >= p.groups) continue;
        T *out = static_cast<T *>(p.out) + at_of(b, p.os);
#pragma unroll
        for (int i = 0; i < kVpl; ++i) {
            const int at = lane + i * kLanes;
            if (at >= p.vecs) continue;
            Vec<T, N> y;
#pragma unroll
            for (int j = 0; j < N; ++j)
                y.v[j] = from_f<T>(to_f<T>(xv[b][i].v[j]) * inv * w[i][j] * act_f<T, kAct>(to_f<T>(gv[b][i].v[j])));
            st_vec<T, N>(out + at * N, y);
        }
    }
}

template <typename T, int kLanes, int kVpl, int kBatch>
cudaError_t launch_gated_batch(const GatedParams &p, int act, kda_stream_t stream) {
    constexpr int kHeads = 256 / kLanes * kBatch;
    const dim3 grid((unsigned)((p.groups + kHeads - 1) / kHeads));
    if (act == KDA_NORM_GATE_NONE)
        return launch(gated_rmsnorm_kernel<T, kLanes, kVpl, kBatch, KDA_NORM_GATE_NONE>, grid, 256, 0, stream, p);
    if (act == KDA_NORM_GATE_SIGMOID)
        return launch(gated_rmsnorm_kernel<T, kLanes, kVpl, kBatch, KDA_NORM_GATE_SIGMOID>, grid, 256, 0, stream, p);
    return launch(gated_rmsnorm_kernel<T, kLanes, kVpl, kBatch, KDA_NORM_GATE_SILU>, grid, 256, 0, stream, p);
}

template <typename T, int kLanes, int kVpl>
cudaError_t launch_gated(const GatedParams &p, int act, kda_stream_t stream) {
    // Batches only where they still leave every SM several blocks.
    if constexpr (kVpl == 1)
        if (p.groups * kLanes >= (int64_t)256 * 4 * 8 * current_sms())
            return launch_gated_batch<T, kLanes, kVpl, 4>(p, act, stream);
    return launch_gated_batch<T, kLanes, kVpl, 1>(p, act, stream);
}

template <typename T>
cudaError_t dispatch_gated(const GatedParams &p, int act, kda_stream_t stream) {
    if (p.vecs <= 4) return launch_gated<T, 4, 1>(p, act, stream);
    if (p.vecs <= 8) return launch_gated<T, 8, 1>(p, act, stream);
    if (p.vecs <= 16) return launch_gated<T, 16, 1>(p, act, stream);
    if (p.vecs <= 32) return launch_gated<T, 32, 1>(p, act, stream);
    if (p.vecs <= 64) return launch_gated<T, 32, 2>(p, act, stream);
    return launch_gated<T, 32, 4>(p, act, stream);
}

struct ResidualParams {
    const void *y, *gate, *residual;
    const float *weight, *post;
    void *out, *residual_out;
    int64_t ys, gs, rs, os, ros;
    int64_t rows;
    int vecs;  // 16-byte vectors of T per row
    float scale, eps, inv_width;
};

// The sum over the block of every thread's value; `slot` alternates so that
// one barrier per sum is enough.
__device__ __forceinline__ float block_sum(float v, float *slot, int warps) {
#pragma unroll
    for (int m = 16; m > 0; m /= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
    if (threadIdx.x % 32 == 0) slot[threadIdx.x / 32] = v;
    __syncthreads();
    float s = threadIdx.x % 32 < warps ? slot[threadIdx.x % 32] : 0.0f;
#pragma unroll
    for (int m = 16; m > 0; m /= 2) s += __shfl_xor_sync(0xffffffffu, s, m);
    return s;
}

__device__ __forceinline__ void copy16(void *to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}
template <int kLeft>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory"); }

// 16-byte pieces a thread holds of one row.
template <typename T, typename R, int kVpt, bool kGate>
constexpr int kPieces = kVpt * (1 + (kGate ? 1 : 0) + (int)(sizeof(R) / sizeof(T)));
template <int kVpt>
constexpr int kRowsAhead = kVpt < 4 ? 2 : 1;  // the widest rows' pieces fill 128 KB

// A block takes rows blockIdx.x, + gridDim.x, ...; a thread owns kVpt vectors of a
// row, keeps y and then r in registers between the reductions, and has its pieces
// of the next kRowsAhead rows on their way into its own part of shared memory (it
// alone reads them, so no barrier guards them): held in registers they would leave
// too few threads on the SM to keep HBM busy (16384 x 4608 bf16: 118.6 us, 6.37 TB/s,
// 95% of a copy's rate; 160 one row at a time, 277 with the next row in registers).
template <typename T, typename R, int kVpt, int kAct, bool kPost>
__global__ void __launch_bounds__(512) residual_rmsnorm_kernel(const __grid_constant__ ResidualParams p) {
    constexpr bool kGate = kAct != KDA_NORM_GATE_NONE;
    constexpr int N = 16 / sizeof(T), NR = sizeof(R) / sizeof(T), RE = 16 / sizeof(R);
    constexpr int kAll = kPieces<T, R, kVpt, kGate>;
    __shared__ float slots[2][32];
    extern __shared__ uint4 ring[];  // [row ahead][piece][thread]
    dependency_wait();
    const int warps = blockDim.x / 32;
    auto fetch = [&](int64_t row, int slot) {
        if (row < p.rows) {
            uint4 *to = ring + slot * kAll * blockDim.x + threadIdx.x;
#pragma unroll
            for (int i = 0; i < kVpt; ++i) {
                const int at = threadIdx.x + i * blockDim.x;
                if (at >= p.vecs) continue;
                copy16(to + i * blockDim.x, static_cast<const T *>(p.y) + row * p.ys + at * N);
                if constexpr (kGate)
                    copy16(to + (kVpt + i) * blockDim.x, static_cast<const T *>(p.gate) + row * p.gs + at * N);
#pragma unroll
                for (int c = 0; c < NR; ++c)
                    copy16(to + ((kGate ? 2 : 1) * kVpt + i * NR + c) * blockDim.x,
                           static_cast<const R *>(p.residual) + row * p.rs + at * N + c * RE);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kRowsAhead<kVpt>; ++i) fetch(blockIdx.x + (int64_t)i * gridDim.x, i);
    int slot = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, slot = slot + 1 == kRowsAhead<kVpt> ? 0 : slot + 1) {
        copies_wait<kRowsAhead<kVpt> - 1>();
        const uint4 *from = ring + slot * kAll * blockDim.x + threadIdx.x;
        Vec<T, N> yv[kVpt], gv[kVpt];
        Vec<R, RE> rv[kVpt][NR];
#pragma unroll
        for (int i = 0; i < kVpt; ++i) {
            *reinterpret_cast<uint4 *>(&yv[i]) = from[i * blockDim.x];
            if constexpr (kGate) *reinterpret_cast<uint4 *>(&gv[i]) = from[(kVpt + i) * blockDim.x];
#pragma unroll
            for (int c = 0; c < NR; ++c)
                *reinterpret_cast<uint4 *>(&rv[i][c]) = from[((kGate ? 2 : 1) * kVpt + i * NR + c) * blockDim.x];
        }
        fetch(row + (int64_t)kRowsAhead<kVpt> * gridDim.x, slot);
        float inv_y = 1.0f;
        if constexpr (kPost) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kVpt; ++i)
                if ((int)(threadIdx.x + i * blockDim.x) < p.vecs)
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        const float f = to_f<T>(yv[i].v[j]);
                        sum = fmaf(f, f, sum);
                    }
            inv_y = rsqrtf(fmaf(block_sum(sum, slots[0], warps), p.inv_width, p.eps));
        }
        float r[kVpt][N];
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kVpt; ++i) {
            const int at = threadIdx.x + i * blockDim.x;
            const bool in = at < p.vecs;
#pragma unroll
            for (int j = 0; j < N; j += 4) {
                float4 w = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
                if constexpr (kPost)
                    if (in) w = __ldg(reinterpret_cast<const float4 *>(p.post + at * N + j));
                const float ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float b = to_f<T>(yv[i].v[j + c]);
                    if constexpr (kPost) b = b * inv_y * ws[c];
                    if constexpr (kGate) b *= act_f<T, kAct>(to_f<T>(gv[i].v[j + c]));
                    const float f = fmaf(p.scale, b, to_f<R>(rv[i][(j + c) / RE].v[(j + c) % RE]));
                    r[i][j + c] = in ? f : 0.0f;
                    sum = fmaf(r[i][j + c], r[i][j + c], sum);
                }
            }
        }
        R *ro = static_cast<R *>(p.residual_out) + row * p.ros;
#pragma unroll
        for (int i = 0; i < kVpt; ++i) {
            const int at = threadIdx.x + i * blockDim.x;
            if (at >= p.vecs) continue;
#pragma unroll
            for (int c = 0; c < NR; ++c) {
                Vec<R, RE> o;
#pragma unroll
                for (int j = 0; j < RE; ++j) o.v[j] = from_f<R>(r[i][c * RE + j]);
                st_vec<R, RE>(ro + at * N + c * RE, o);
            }
        }
        const float inv = rsqrtf(fmaf(block_sum(sum, slots[1], warps), p.inv_width, p.eps));
        T *out = static_cast<T *>(p.out) + row * p.os;
#pragma unroll
        for (int i = 0; i < kVpt; ++i) {
            const int at = threadIdx.x + i * blockDim.x;
            if (at >= p.vecs) continue;
            Vec<T, N> o;
#pragma unroll
            for (int j = 0; j < N; j += 4) {
                float4 w = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
                if (p.weight != nullptr)
                    w = __ldg(reinterpret_cast<const float4 *>(p.weight + at * N + j));
                o.v[j] = from_f<T>(r[i][j] * inv * w.x);
                o.v[j + 1] = from_f<T>(r[i][j + 1] * inv * w.y);
                o.v[j + 2] = from_f<T>(r[i][j + 2] * inv * w.z);
                o.v[j + 3] = from_f<T>(r[i][j + 3] * inv * w.w);
            }
            st_vec<T, N>(out + at * N, o);
        }
        // Without the norm of y one barrier separates two rows' use of slots[1]:
        // a thread may still read it when another starts the next row.
        if constexpr (!kPost) __syncthreads();
    }
}

template <typename T, typename R, int kVpt, int kAct, bool kPost>
cudaError_t launch_residual_post(const ResidualParams &p, kda_stream_t stream) {
    const unsigned threads = (unsigned)(((p.vecs + kVpt - 1) / kVpt + 31) / 32 * 32);
    auto *kernel = residual_rmsnorm_kernel<T, R, kVpt, kAct, kPost>;
    const size_t smem = (size_t)threads * 16 * kRowsAhead<kVpt> * kPieces<T, R, kVpt, kAct != KDA_NORM_GATE_NONE>;
    static std::atomic<uint64_t> done;
    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(kernel), 512 * 16 * kRowsAhead<kVpt> *
                                     kPieces<T, R, kVpt, kAct != KDA_NORM_GATE_NONE>, done);
    if (e != cudaSuccess) return e;
    // About as many blocks as are resident; they loop over the rows.
    const int64_t fit = 1536 / threads, room = (int64_t)(220 * 1024 / smem);
    const int64_t most = current_sms() * (fit < 1 || room < 1 ? 1 : fit < room ? fit : room);
    const int64_t blocks = p.rows < most ? p.rows : most;
    return launch(kernel, dim3((unsigned)blocks), threads, smem, stream, p);
}

template <typename T, typename R, int kVpt, int kAct>
cudaError_t launch_residual(const ResidualParams &p, kda_stream_t stream) {
    return p.post != nullptr ? launch_residual_post<T, R, kVpt, kAct, true>(p, stream)
                             : launch_residual_post<T, R, kVpt, kAct, false>(p, stream);
}

template <typename T, typename R, int kVpt>
cudaError_t act_residual(const ResidualParams &p, int act, kda_stream_t stream) {
    if (act == KDA_NORM_GATE_NONE) return launch_residual<T, R, kVpt, KDA_NORM_GATE_NONE>(p, stream);
    if (act == KDA_NORM_GATE_SIGMOID)
        return launch_residual<T, R, kVpt, KDA_NORM_GATE_SIGMOID>(p, stream);
    return launch_residual<T, R, kVpt, KDA_NORM_GATE_SILU>(p, stream);
}

template <typename T, typename R>
cudaError_t dispatch_residual(const ResidualParams &p, int act, kda_stream_t stream) {
    // One vector per thread up to 512 threads, then two, then four (at most 512
    // threads of four: 2048 vectors, the documented width limit).
    if (p.vecs <= 512) return act_residual<T, R, 1>(p, act, stream);
    if (p.vecs <= 1024) return act_residual<T, R, 2>(p, act, stream);
    return act_residual<T, R, 4>(p, act, stream);
}

bool strides_ok(const int64_t *s, int n, int64_t quantum) {
    for (int i = 0; i < n; ++i)
        if (s[i] < 0 || s[i] % quantum != 0) return false;
    return true;
}

bool norm_scalars_ok(float eps, int act, const void *gate) {
    if (!(eps >= 0.0f) || isinf(eps)) return false;
    if (act < KDA_NORM_GATE_NONE || act > KDA_NORM_GATE_SILU) return false;
    return act == KDA_NORM_GATE_NONE || gate != nullptr;
}

}  // namespace
}  // namespace kda_layer

using namespace kda_layer;

extern "C" {

const char *kda_layer_error_string(void) { return error_buffer(); }

kda_status_t kda_gated_rmsnorm(const void *x, const int64_t x_stride[2], const void *gate,
                               const int64_t gate_stride[2], const float *weight, float eps,
                               int activation, int64_t rows, int64_t heads, int64_t head_dim,
                               int dtype, void *out, const int64_t out_stride[2],
                               kda_stream_t stream) {
    if (rows < 0 || heads <= 0 || head_dim <= 0 || !dtype_ok(dtype) ||
        !norm_scalars_ok(eps, activation, rows > 0 ? gate : &eps))
        return KDA_ERR_INVALID_ARG;
    const int64_t quantum = 16 / dtype_bytes(dtype);
    if (head_dim % quantum != 0 || head_dim > 128 * quantum || heads > (1 << 30))
        return KDA_ERR_UNSUPPORTED;
    if (rows == 0) return KDA_OK;
    const bool gated = activation != KDA_NORM_GATE_NONE;
    if (x == nullptr || out == nullptr || x_stride == nullptr || out_stride == nullptr ||
        (gated && gate_stride == nullptr) || rows > (int64_t(1) << 40) / heads)
        return KDA_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(out, 16) || !aligned(weight, 16) || !strides_ok(x_stride, 2, quantum) ||
        !strides_ok(out_stride, 2, quantum) ||
        (gated && (!aligned(gate, 16) || !strides_ok(gate_stride, 2, quantum))))
        return KDA_ERR_MISALIGNED;
    GatedParams p = {};
    p.x = x, p.gate = gated ? gate : x, p.weight = weight, p.out = out;
    for (int i = 0; i < 2; ++i) {
        p.xs[i] = x_stride[i], p.os[i] = out_stride[i];
        p.gs[i] = gated ? gate_stride[i] : x_stride[i];
    }
    p.groups = rows * heads;
    p.heads = (int)heads;
    p.heads_div = make_fast_div((uint32_t)heads);
    p.vecs = (int)(head_dim / quantum);
    p.eps = eps;
    p.inv_dim = 1.0f / (float)head_dim;
    if (p.groups > (int64_t(1) << 31)) return KDA_ERR_INVALID_ARG;  // grid of up to 2^28 blocks
    if (dtype == KDA_DTYPE_BF16) return cuda_status(dispatch_gated<__nv_bfloat16>(p, activation, stream));
    if (dtype == KDA_DTYPE_F16) return cuda_status(dispatch_gated<__half>(p, activation, stream));
    return cuda_status(dispatch_gated<float>(p, activation, stream));
}

kda_status_t kda_residual_rmsnorm(const void *y, int64_t y_stride, const void *residual,
                                  int64_t residual_stride, const void *gate, int64_t gate_stride,
                                  const float *weight, const float *post_weight, float scale,
                                  float eps, int activation, int64_t rows, int64_t width,
                                  int dtype, int residual_f32, void *out, int64_t out_stride,
                                  void *residual_out, int64_t residual_out_stride,
                                  kda_stream_t stream) {
    if (rows < 0 || width <= 0 || !dtype_ok(dtype) || (residual_f32 != 0 && residual_f32 != 1) ||
        !norm_scalars_ok(eps, activation, rows > 0 ? gate : &eps))
        return KDA_ERR_INVALID_ARG;
    const int64_t quantum = 16 / dtype_bytes(dtype);
    if (width % quantum != 0 || width > 2048 * quantum) return KDA_ERR_UNSUPPORTED;
    if (rows == 0) return KDA_OK;
    if (y == nullptr || residual == nullptr || out == nullptr || residual_out == nullptr)
        return KDA_ERR_INVALID_ARG;
    const bool gated = activation != KDA_NORM_GATE_NONE;
    const bool f32 = residual_f32 != 0 || dtype == KDA_DTYPE_F32;
    const int64_t rq = f32 ? 4 : 8;
    if (!aligned(y, 16) || !aligned(residual, 16) || !aligned(out, 16) || !aligned(residual_out, 16) ||
        !aligned(weight, 16) || !aligned(post_weight, 16) || !strides_ok(&y_stride, 1, quantum) ||
        !strides_ok(&out_stride, 1, quantum) || !strides_ok(&residual_stride, 1, rq) ||
        !strides_ok(&residual_out_stride, 1, rq) ||
        (gated && (!aligned(gate, 16) || !strides_ok(&gate_stride, 1, quantum))))
        return KDA_ERR_MISALIGNED;
    ResidualParams p = {};
    p.y = y, p.gate = gated ? gate : y, p.residual = residual;
    p.weight = weight, p.post = post_weight;
    p.out = out, p.residual_out = residual_out;
    p.ys = y_stride, p.gs = gated ? gate_stride : y_stride, p.rs = residual_stride;
    p.os = out_stride, p.ros = residual_out_stride;
    p.rows = rows;
    p.vecs = (int)(width / quantum);
    p.scale = scale, p.eps = eps, p.inv_width = 1.0f / (float)width;
    if (dtype == KDA_DTYPE_F32) return cuda_status(dispatch_residual<float, float>(p, activation, stream));
    if (dtype == KDA_DTYPE_BF16)
        return cuda_status(f32 ? dispatch_residual<__nv_bfloat16, float>(p, activation, stream)
                               : dispatch_residual<__nv_bfloat16, __nv_bfloat16>(p, activation, stream));
    return cuda_status(f32 ? dispatch_residual<__half, float>(p, activation, stream)
                           : dispatch_residual<__half, __half>(p, activation, stream));
}

}  // extern "C"

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

template <int kAct>
__device__ __forceinline__ float act_f(float z) {
    if constexpr (kAct == KDA_NORM_GATE_NONE) return 1.0f;
    const float s = sigmoid_f(z);
    return kAct == KDA_NORM_GATE_SILU ? z * s : s;
}

struct GatedParams {
    const void *x, *gate;
    const float *weight;
    void *out;
    int64_t xs[2], gs[2], os[2];
    int64_t groups;  // rows * heads
    int heads;
    int vecs;  // 16-byte vectors per head
    float eps, inv_dim;
};

// kLanes neighbouring lanes own one (row, head); each holds kVpl vectors of it
// in registers, so x is read once and the sum of squares is a butterfly.
template <typename T, int kLanes, int kVpl, int kAct>
__global__ void __launch_bounds__(256) gated_rmsnorm_kernel(GatedParams p) {
    constexpr int N = 16 / sizeof(T);
    dependency_wait();
    const int64_t group = (int64_t(blockIdx.x) * 256 + threadIdx.x) / kLanes;
    const int lane = threadIdx.x % kLanes;
    const bool live = group < p.groups;
    const int64_t row = live ? group / p.heads : 0, head = live ? group % p.heads : 0;
    const T *x = static_cast<const T *>(p.x) + row * p.xs[0] + head * p.xs[1];
    const T *gate = static_cast<const T *>(p.gate) + row * p.gs[0] + head * p.gs[1];
    T *out = static_cast<T *>(p.out) + row * p.os[0] + head * p.os[1];
    Vec<T, N> xv[kVpl], gv[kVpl];
#pragma unroll
    for (int i = 0; i < kVpl; ++i) {
        const int at = lane + i * kLanes;
        if (live && at < p.vecs) {
            xv[i] = ld_vec<T, N>(x + at * N);
            if constexpr (kAct != KDA_NORM_GATE_NONE) gv[i] = ld_vec<T, N>(gate + at * N);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) xv[i].v[j] = gv[i].v[j] = from_f<T>(0.0f);
        }
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kVpl; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float f = to_f<T>(xv[i].v[j]);
            sum = fmaf(f, f, sum);
        }
#pragma unroll
    for (int m = kLanes / 2; m > 0; m /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    const float inv = rsqrtf(fmaf(sum, p.inv_dim, p.eps));
#pragma unroll
    for (int i = 0; i < kVpl; ++i) {
        const int at = lane + i * kLanes;
        if (!live || at >= p.vecs) continue;
        float w[N];
#pragma unroll
        for (int j = 0; j < N; j += 4) {
            float4 f = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
            if (p.weight != nullptr)
                f = __ldg(reinterpret_cast<const float4 *>(p.weight + at * N + j));
            w[j] = f.x, w[j + 1] = f.y, w[j + 2] = f.z, w[j + 3] = f.w;
        }
        Vec<T, N> y;
#pragma unroll
        for (int j = 0; j < N; ++j)
            y.v[j] = from_f<T>(to_f<T>(xv[i].v[j]) * inv * w[j] * act_f<kAct>(to_f<T>(gv[i].v[j])));
        st_vec<T, N>(out + at * N, y);
    }
}

template <typename T, int kLanes, int kVpl>
cudaError_t launch_gated(const GatedParams &p, int act, kda_stream_t stream) {
    const int64_t blocks = (p.groups * kLanes + 255) / 256;
    const dim3 grid((unsigned)blocks);
    if (act == KDA_NORM_GATE_NONE)
        return launch(gated_rmsnorm_kernel<T, kLanes, kVpl, KDA_NORM_GATE_NONE>, grid, 256, 0, stream, p);
    if (act == KDA_NORM_GATE_SIGMOID)
        return launch(gated_rmsnorm_kernel<T, kLanes, kVpl, KDA_NORM_GATE_SIGMOID>, grid, 256, 0, stream, p);
    return launch(gated_rmsnorm_kernel<T, kLanes, kVpl, KDA_NORM_GATE_SILU>, grid, 256, 0, stream, p);
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

// One block per row at a time; a thread owns kVpt vectors of the row, keeps y
// and then r in registers between the reductions.
template <typename T, typename R, int kVpt, int kAct, bool kPost>
__global__ void __launch_bounds__(512) residual_rmsnorm_kernel(ResidualParams p) {
    constexpr int N = 16 / sizeof(T);
    constexpr int NR = N * sizeof(R) / 16;   // 16-byte loads of a residual vector
    constexpr int RE = 16 / sizeof(R);
    __shared__ float slots[2][32];
    dependency_wait();
    const int warps = blockDim.x / 32;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T *y = static_cast<const T *>(p.y) + row * p.ys;
        const T *gate = static_cast<const T *>(p.gate) + row * p.gs;
        const R *res = static_cast<const R *>(p.residual) + row * p.rs;
        Vec<T, N> yv[kVpt], gv[kVpt];
        Vec<R, RE> rv[kVpt][NR];
#pragma unroll
        for (int i = 0; i < kVpt; ++i) {
            const int at = threadIdx.x + i * blockDim.x;
            if (at < p.vecs) {
                yv[i] = ld_vec<T, N>(y + at * N);
                if constexpr (kAct != KDA_NORM_GATE_NONE) gv[i] = ld_vec<T, N>(gate + at * N);
#pragma unroll
                for (int c = 0; c < NR; ++c) rv[i][c] = ld_vec<R, RE>(res + at * N + c * RE);
            } else {
#pragma unroll
                for (int j = 0; j < N; ++j) yv[i].v[j] = gv[i].v[j] = from_f<T>(0.0f);
#pragma unroll
                for (int c = 0; c < NR; ++c)
#pragma unroll
                    for (int j = 0; j < RE; ++j) rv[i][c].v[j] = from_f<R>(0.0f);
            }
        }
        float inv_y = 1.0f;
        if constexpr (kPost) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kVpt; ++i)
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
                    if constexpr (kAct != KDA_NORM_GATE_NONE) b *= act_f<kAct>(to_f<T>(gv[i].v[j + c]));
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

template <typename T, typename R, int kVpt, int kAct>
cudaError_t launch_residual(const ResidualParams &p, kda_stream_t stream) {
    const unsigned threads = (unsigned)(((p.vecs + kVpt - 1) / kVpt + 31) / 32 * 32);
    const dim3 grid((unsigned)(p.rows < (int64_t(1) << 30) ? p.rows : (int64_t(1) << 30)));
    if (p.post != nullptr)
        return launch(residual_rmsnorm_kernel<T, R, kVpt, kAct, true>, grid, threads, 0, stream, p);
    return launch(residual_rmsnorm_kernel<T, R, kVpt, kAct, false>, grid, threads, 0, stream, p);
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
    if (head_dim % quantum != 0 || head_dim > 128 * quantum || heads > INT32_MAX)
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

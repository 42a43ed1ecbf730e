// gdn_linear.cu -- matrix product with bias, activation and residual, and its gradients.
//
//     pre = x W^T + bias,  y = act(pre) + res
//     dpre = dy act'(pre),  dx = dpre W,  dW = dpre^T x,  dbias = sum_m dpre
#include "gdn_layer.cuh"

namespace gdn {

namespace {

constexpr int kTile = 64, kDepth = 16;
constexpr int kBiasSlices = 64;

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

__device__ __forceinline__ float act_rt(int act, float x) {
    return act == kActSilu ? silu_hw(x) : act == kActGelu ? gelu_f(x) : x;
}
__device__ __forceinline__ float dact_rt(int act, float x) {
    return act == kActSilu ? dsilu_hw(x) : act == kActGelu ? dgelu_f(x) : 1.f;
}

// One operand: element (r, k) at p[r * rs + k * cs].
template <typename T>
struct Operand {
    const T *p;
    long long rs, cs;
};

}  // namespace

// out[m][n] = act(sum_k A[m][k] B[n][k] + bias[n]) + res[m][n]
template <typename T>
__global__ void __launch_bounds__(256) linear_simple_kernel(Operand<T> A, Operand<T> B, int M, int N, int K, const T *bias,
                                                            int act, const T *res, long long ldres, T *out, T *pre) {
    __shared__ float sa[kDepth][kTile + 1], sb[kDepth][kTile + 1];
    const int m0 = blockIdx.y * kTile, n0 = blockIdx.x * kTile, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < K; k0 += kDepth) {
        for (int e = threadIdx.x; e < kTile * kDepth; e += 256) {
            const int r = e / kDepth, k = e % kDepth;
            sa[k][r] = m0 + r < M && k0 + k < K ? to_f32(A.p[(m0 + r) * A.rs + (k0 + k) * A.cs]) : 0.f;
            sb[k][r] = n0 + r < N && k0 + k < K ? to_f32(B.p[(n0 + r) * B.rs + (k0 + k) * B.cs]) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kDepth; ++k) {
            float a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = sa[k][ty + 16 * i];
                b[i] = sb[k][tx + 16 * i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
        }
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m >= M || n >= N) continue;
            const float v = acc[i][j] + (bias != nullptr ? to_f32(bias[n]) : 0.f);
            if (pre != nullptr) pre[(size_t)m * N + n] = from_f32<T>(v);
            out[(size_t)m * N + n] = from_f32<T>(__fadd_rn(act_rt(act, v), res != nullptr ? to_f32(res[m * ldres + n]) : 0.f));
        }
}

// dpre = dy act'(pre) (dpre null: dy itself is it), and each slice of rows' column sums of it.
template <typename T>
__global__ void __launch_bounds__(256) linear_dpre_kernel(const T *dy, const T *pre, T *dpre, float *part, int M, int N, int act) {
    const int n = blockIdx.x * 256 + threadIdx.x;
    if (n >= N) return;
    float s = 0.f;
    for (size_t m = blockIdx.y; m < (size_t)M; m += gridDim.y) {
        float d = to_f32(dy[m * N + n]);
        if (act != kActNone) d *= dact_rt(act, to_f32(pre[m * N + n]));
        if (dpre != nullptr) dpre[m * N + n] = from_f32<T>(d);
        s += d;
    }
    part[(size_t)blockIdx.y * N + n] = s;
}

template <typename T>
__global__ void __launch_bounds__(256) linear_dbias_kernel(const float *part, T *dbias, int slices, int N) {
    const int n = blockIdx.x * 256 + threadIdx.x;
    if (n >= N) return;
    float s = 0.f;
    for (int k = 0; k < slices; ++k) s += part[(size_t)k * N + n];
    dbias[n] = from_f32<T>(s);
}

size_t linear_fwd_workspace(const LinearParams &, int) { return 0; }

size_t linear_bwd_workspace(const LinearParams &p, int dtype) {
    return up256((size_t)p.M * p.N * (dtype == 0 ? 4 : 2)) + up256((size_t)kBiasSlices * p.N * 4);
}

namespace {

template <typename T>
cudaError_t product(const char *name, Operand<T> A, Operand<T> B, int M, int N, int K, const void *bias, int act, const void *res,
                    long long ldres, void *out, void *pre, cudaStream_t s) {
    timing_mark(name, 0, s);
    linear_simple_kernel<T><<<dim3((N + kTile - 1) / kTile, (M + kTile - 1) / kTile), 256, 0, s>>>(
        A, B, M, N, K, static_cast<const T *>(bias), act, static_cast<const T *>(res), ldres, static_cast<T *>(out),
        static_cast<T *>(pre));
    timing_mark(name, 1, s);
    return cudaGetLastError();
}

template <typename T>
cudaError_t bwd_any(const LinearParams &p, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    const T *dpre = static_cast<const T *>(p.dy);
    float *part = reinterpret_cast<float *>(p.ws + up256((size_t)p.M * p.N * sizeof(T)));
    if (p.act != kActNone || p.dbias != nullptr) {
        T *to = p.act != kActNone ? reinterpret_cast<T *>(p.ws) : nullptr;
        const int slices = p.M < kBiasSlices ? p.M : kBiasSlices;
        timing_mark("linear_dpre", 0, s);
        linear_dpre_kernel<T><<<dim3((p.N + 255) / 256, slices), 256, 0, s>>>(
            static_cast<const T *>(p.dy), static_cast<const T *>(p.pre_in), to, part, p.M, p.N, p.act);
        timing_mark("linear_dpre", 1, s);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        if (to != nullptr) dpre = to;
        if (p.dbias != nullptr) {
            timing_mark("linear_dbias", 0, s);
            linear_dbias_kernel<T><<<(p.N + 255) / 256, 256, 0, s>>>(part, static_cast<T *>(p.dbias), slices, p.N);
            timing_mark("linear_dbias", 1, s);
            if ((e = cudaGetLastError()) != cudaSuccess) return e;
        }
    }
    const Operand<T> x_t = {static_cast<const T *>(p.x), 1, p.ldx}, w_t = {static_cast<const T *>(p.W), 1, p.ldw};
    if (p.dx != nullptr)
        e = product<T>("linear_dx", Operand<T>{dpre, p.N, 1}, w_t, p.M, p.K, p.N, nullptr, kActNone, nullptr, 0, p.dx, nullptr, s);
    if (e == cudaSuccess && p.dW != nullptr)
        e = product<T>("linear_dw", Operand<T>{dpre, 1, p.N}, x_t, p.N, p.K, p.M, nullptr, kActNone, nullptr, 0, p.dW, nullptr, s);
    return e;
}

}  // namespace

int launch_linear_fwd(const LinearParams &p, int dtype, cudaStream_t s) {
    if (dtype == 0)
        return api_cuda_status(product<float>("linear_fwd", {static_cast<const float *>(p.x), p.ldx, 1},
                                              {static_cast<const float *>(p.W), p.ldw, 1}, p.M, p.N, p.K, p.bias, p.act, p.res,
                                              p.ldres, p.y, p.pre, s));
    return api_cuda_status(product<__nv_bfloat16>("linear_fwd", {static_cast<const __nv_bfloat16 *>(p.x), p.ldx, 1},
                                                  {static_cast<const __nv_bfloat16 *>(p.W), p.ldw, 1}, p.M, p.N, p.K, p.bias,
                                                  p.act, p.res, p.ldres, p.y, p.pre, s));
}

int launch_linear_bwd(const LinearParams &p, int dtype, cudaStream_t s) {
    return api_cuda_status(dtype == 0 ? bwd_any<float>(p, s) : bwd_any<__nv_bfloat16>(p, s));
}

}  // namespace gdn

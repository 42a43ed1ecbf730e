// gdn_conv.cu -- the short causal convolution in front of the recurrence, its carried state, and
// its VJP.
//
//     pre[t,c] = bias[c] + sum_{j < W} w[c,j] x~[t-W+1+j,c],   y = act(pre)
// with x~ the carried state (W-1 inputs) followed by x. For cotangents dy of y and ds_T of the
// state behind the last valid step:
//     dpre = dy act'(pre),   dx~[s] = sum_j w[j] dpre[s+W-1-j] (+ ds_T where s is one of the last
//     W-1 inputs),   dw[j] = sum_t dpre[t] x~[t-W+1+j],   dbias = sum_t dpre[t]
//
// A thread takes V neighbouring channels (16 bytes) and walks a run of steps with the last W-1
// inputs in registers, so that x is read once and the taps once per run. Each channel's W products
// are far below the memory time: the kernels are bound by the bytes of x and y (and dy, dx).
#include "gdn_layer.cuh"

namespace gdn {

namespace {

constexpr int kConvThreads = 256;
constexpr int kConvBwdWarps = 8;

template <typename T, int V>
__device__ __forceinline__ void load_or_zero(const T *p, bool ok, float (&o)[V]) {
    if (ok) load_vec<T, V>(p, o);
    else {
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = 0.f;
    }
}

// x~ at step t (negative: the carried state) for the V channels from c
template <typename T, int V>
__device__ __forceinline__ void load_input(const ConvParams &p, int W, int b, int t, int c, float (&o)[V]) {
    if (t >= 0) load_vec<T, V>(static_cast<const T *>(p.x) + ((size_t)b * p.T + t) * p.ldx + c, o);
    else
        load_or_zero<T, V>(static_cast<const T *>(p.s0) + ((size_t)b * (W - 1) + (W - 1 + t)) * p.C + c,
                           p.s0 != nullptr && t >= 1 - W, o);
}

template <int W, int V>
__device__ __forceinline__ void load_taps(const ConvParams &p, int c, float (&w)[V][W], float (&bias)[V]) {
    if constexpr (V % 4 == 0) {
        float flat[V * W];
#pragma unroll
        for (int i = 0; i < V * W / 4; ++i) {
            const float4 q = *reinterpret_cast<const float4 *>(p.w + (size_t)c * W + 4 * i);
            flat[4 * i] = q.x; flat[4 * i + 1] = q.y; flat[4 * i + 2] = q.z; flat[4 * i + 3] = q.w;
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int j = 0; j < W; ++j) w[v][j] = flat[v * W + j];
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int j = 0; j < W; ++j) w[v][j] = p.w[(size_t)(c + v) * W + j];
    }
#pragma unroll
    for (int v = 0; v < V; ++v) bias[v] = p.bias ? p.bias[c + v] : 0.f;
}

}  // namespace

// Threads over (batch row, run of `run` steps, V channels). The thread of a row's first run also
// writes the state behind the row's last valid step.
template <typename T, int W, int V>
__global__ void __launch_bounds__(kConvThreads) conv_fwd_kernel(ConvParams p, int run, int runs) {
    constexpr int U = 4;                                   // steps loaded ahead
    const int CV = p.C / V;
    const size_t id = (size_t)blockIdx.x * kConvThreads + threadIdx.x;
    if (id >= (size_t)p.B * runs * CV) return;
    const int c = (int)(id % CV) * V;
    const size_t rb = id / CV;
    const int r = (int)(rb % runs), b = (int)(rb / runs);
    const int L = row_length(p.lens, b, p.T);
    const int t0 = r * run, t1 = min(t0 + run, p.T);
    float w[V][W], bias[V], win[W][V];
    load_taps<W, V>(p, c, w, bias);
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
#pragma unroll
        for (int v = 0; v < V; ++v) win[i][v] = 0.f;
        if (t0 + i - (W - 1) < L) load_input<T, V>(p, W, b, t0 + i - (W - 1), c, win[i]);
    }
    if (r == 0 && p.s_T != nullptr) {
        float keep[W][V];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) load_input<T, V>(p, W, b, L - (W - 1) + j, c, keep[j]);
        T *out = static_cast<T *>(p.s_T) + (size_t)b * (W - 1) * p.C + c;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) store_vec<T, V>(out + (size_t)j * p.C, keep[j]);
    }
    const T *x = static_cast<const T *>(p.x) + (size_t)b * p.T * p.ldx + c;
    T *y = static_cast<T *>(p.y) + (size_t)b * p.T * p.C + c;
    for (int t = t0; t < t1; t += U) {
        float in[U][V];
#pragma unroll
        for (int i = 0; i < U; ++i) load_or_zero<T, V>(x + (size_t)(t + i) * p.ldx, t + i < min(t1, L), in[i]);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (t + i >= t1) break;
            float o[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                win[W - 1][v] = in[i][v];
                float pre = bias[v];
#pragma unroll
                for (int j = 0; j < W; ++j) pre = fmaf(w[v][j], win[j][v], pre);
                o[v] = t + i < L ? (p.act == kActSilu ? silu_hw(pre) : pre) : 0.f;
#pragma unroll
                for (int j = 0; j < W - 1; ++j) win[j][v] = win[j + 1][v];
            }
            store_vec<T, V>(y + (size_t)(t + i) * p.C, o);
        }
    }
}

// A CTA takes 32 V channels and 8 runs of steps (one per warp) of one batch row. The parameter sums
// go over a thread's steps, then over the CTA's warps in ascending order, into the CTA's slice of
// the partial sums: a fixed order.
template <typename T, int W, int V>
__global__ void __launch_bounds__(32 * kConvBwdWarps) conv_bwd_kernel(ConvParams p, int run, int slices_row) {
    __shared__ float sums[kConvBwdWarps][W + 1][32 * V];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = (blockIdx.y * 32 + lane) * V;
    const int b = blockIdx.x / slices_row, sl = blockIdx.x % slices_row;
    const int L = row_length(p.lens, b, p.T);
    const int t0 = (sl * kConvBwdWarps + warp) * run, t1 = min(t0 + run, p.T);
    float dw[W][V], db[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        db[v] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][v] = 0.f;
    }
    if (c < p.C && t0 < t1) {
        float w[V][W], bias[V], win[W][V], dwin[W][V];
        load_taps<W, V>(p, c, w, bias);
#pragma unroll
        for (int i = 0; i < W; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) win[i][v] = dwin[i][v] = 0.f;
#pragma unroll
        for (int i = 0; i < W - 1; ++i)
            if (t0 + i - (W - 1) < L) load_input<T, V>(p, W, b, t0 + i - (W - 1), c, win[i]);
        const T *x = static_cast<const T *>(p.x) + (size_t)b * p.T * p.ldx + c;
        const T *dy = static_cast<const T *>(p.dy) + (size_t)b * p.T * p.C + c;
        const T *ds_T = static_cast<const T *>(p.ds_T) + (size_t)b * (W - 1) * p.C + c;
        T *dx = static_cast<T *>(p.dx) + (size_t)b * p.T * p.C + c;
        T *ds0 = static_cast<T *>(p.ds0) + (size_t)b * (W - 1) * p.C + c;
        constexpr int U = 4;
        for (int tb = t0; tb < t1 + W - 1; tb += U) {
            float xin[U][V], din[U][V];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const bool ok = tb + i < min(t1 + W - 1, L);
                load_or_zero<T, V>(x + (size_t)(tb + i) * p.ldx, ok, xin[i]);
                load_or_zero<T, V>(dy + (size_t)(tb + i) * p.C, ok, din[i]);
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int t = tb + i;
                if (t >= t1 + W - 1) break;
                float o[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    win[W - 1][v] = xin[i][v];
                    float pre = bias[v];
#pragma unroll
                    for (int j = 0; j < W; ++j) pre = fmaf(w[v][j], win[j][v], pre);
                    const float dpre = t < L ? (p.act == kActSilu ? din[i][v] * dsilu_hw(pre) : din[i][v]) : 0.f;
                    dwin[W - 1][v] = dpre;
                    if (t < t1) {
                        db[v] += dpre;
#pragma unroll
                        for (int j = 0; j < W; ++j) dw[j][v] = fmaf(dpre, win[j][v], dw[j][v]);
                    }
                    o[v] = 0.f;
#pragma unroll
                    for (int j = 0; j < W; ++j) o[v] = fmaf(w[v][j], dwin[W - 1 - j][v], o[v]);
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) {
                        win[j][v] = win[j + 1][v];
                        dwin[j][v] = dwin[j + 1][v];
                    }
                }
                const int s = t - (W - 1);            // the input whose gradient is complete now
                if (s >= t0) {
                    const int j = s - (L - (W - 1));  // its place in the state behind the row, if any
                    if (p.ds_T != nullptr && j >= 0 && j < W - 1) {
                        float e[V];
                        load_vec<T, V>(ds_T + (size_t)j * p.C, e);
#pragma unroll
                        for (int v = 0; v < V; ++v) o[v] += e[v];
                    }
                    if (s >= L) {
#pragma unroll
                        for (int v = 0; v < V; ++v) o[v] = 0.f;
                    }
                    store_vec<T, V>(dx + (size_t)s * p.C, o);
                } else if (t0 == 0 && p.ds0 != nullptr) {
                    const int j = t - L;              // row t of s0 is row t - L of the state behind the row
                    if (p.ds_T != nullptr && j >= 0) {
                        float e[V];
                        load_vec<T, V>(ds_T + (size_t)j * p.C, e);
#pragma unroll
                        for (int v = 0; v < V; ++v) o[v] += e[v];
                    }
                    store_vec<T, V>(ds0 + (size_t)t * p.C, o);
                }
            }
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        sums[warp][W][lane * V + v] = db[v];
#pragma unroll
        for (int j = 0; j < W; ++j) sums[warp][j][lane * V + v] = dw[j][v];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (W + 1) * 32 * V; i += 32 * kConvBwdWarps) {
        const int j = i / (32 * V), cc = i % (32 * V);
        if (blockIdx.y * 32 * V + cc >= p.C) continue;
        float a = 0.f;
#pragma unroll
        for (int k = 0; k < kConvBwdWarps; ++k) a += sums[k][j][cc];
        p.part[((size_t)blockIdx.x * (W + 1) + j) * p.C + blockIdx.y * 32 * V + cc] = a;
    }
}

// dw[c][j] and dbias[c] from the slices' partial sums, in ascending order.
__global__ void __launch_bounds__(256) conv_reduce_kernel(ConvParams p, int slices) {
    const int W = p.W;
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (size_t)(W + 1) * p.C) return;
    const int j = (int)(i / p.C), c = (int)(i % p.C);
    double a = 0.0;
    for (int s = 0; s < slices; ++s) a += (double)p.part[((size_t)s * (W + 1) + j) * p.C + c];
    if (j < W) p.dw[(size_t)c * W + j] = (float)a;
    else if (p.dbias != nullptr) p.dbias[c] = (float)a;
}

namespace {

bool conv_aligned(const ConvParams &p, int V, size_t e) {
    return p.C % V == 0 && p.ldx % V == 0 && (uintptr_t)p.x % (V * e) == 0;
}

// Steps per warp of the backward: up to 32, fewer while that leaves under 512 CTAs (3 per SM).
int conv_bwd_run(const ConvParams &p) {
    int run = (p.T + kConvBwdWarps - 1) / kConvBwdWarps;
    run = run > 32 ? 32 : run;
    const long long cols = (p.C + 127) / 128;
    while (run > 8 && cols * p.B * ((p.T + kConvBwdWarps * run - 1) / (kConvBwdWarps * run)) < 512) run /= 2;
    return run;
}

template <typename T, int W, int V>
cudaError_t conv_fwd_launch(const ConvParams &p, cudaStream_t s) {
    // Steps per thread: each run reads W-1 inputs again, so up to 32, fewer while the threads would
    // not fill the SMs.
    const size_t cv = p.C / V;
    int run = 32;
    while (run > 1 && (size_t)p.B * ((p.T + run - 1) / run) * cv < (size_t)152 * 1024) run /= 2;
    const int runs = (p.T + run - 1) / run;
    const size_t n = (size_t)p.B * runs * cv;
    timing_mark("conv_fwd", 0, s);
    conv_fwd_kernel<T, W, V><<<(unsigned)((n + kConvThreads - 1) / kConvThreads), kConvThreads, 0, s>>>(p, run, runs);
    timing_mark("conv_fwd", 1, s);
    return cudaGetLastError();
}

template <typename T, int W, int V>
cudaError_t conv_bwd_launch(const ConvParams &p, cudaStream_t s) {
    const int run = conv_bwd_run(p), slices_row = (p.T + kConvBwdWarps * run - 1) / (kConvBwdWarps * run);
    const int slices = p.B * slices_row;
    timing_mark("conv_bwd", 0, s);
    conv_bwd_kernel<T, W, V><<<dim3(slices, (p.C + 32 * V - 1) / (32 * V)), 32 * kConvBwdWarps, 0, s>>>(p, run, slices_row);
    timing_mark("conv_bwd", 1, s);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    timing_mark("conv_reduce", 0, s);
    conv_reduce_kernel<<<(unsigned)(((size_t)(W + 1) * p.C + 255) / 256), 256, 0, s>>>(p, slices);
    timing_mark("conv_reduce", 1, s);
    return cudaGetLastError();
}

template <typename T, int V>
cudaError_t conv_fwd_taps(const ConvParams &p, cudaStream_t s) {
    switch (p.W) {
        case 1: return conv_fwd_launch<T, 1, V>(p, s);
        case 2: return conv_fwd_launch<T, 2, V>(p, s);
        case 3: return conv_fwd_launch<T, 3, V>(p, s);
        default: return conv_fwd_launch<T, 4, V>(p, s);
    }
}
template <typename T, int V>
cudaError_t conv_bwd_taps(const ConvParams &p, cudaStream_t s) {
    switch (p.W) {
        case 1: return conv_bwd_launch<T, 1, V>(p, s);
        case 2: return conv_bwd_launch<T, 2, V>(p, s);
        case 3: return conv_bwd_launch<T, 3, V>(p, s);
        default: return conv_bwd_launch<T, 4, V>(p, s);
    }
}

}  // namespace

int conv_bwd_slices(const ConvParams &p) {
    const int run = conv_bwd_run(p);
    return p.B * ((p.T + kConvBwdWarps * run - 1) / (kConvBwdWarps * run));
}

cudaError_t launch_conv_fwd(const ConvParams &p, int dtype, cudaStream_t s) {
    if (dtype == 0) return conv_aligned(p, 4, 4) ? conv_fwd_taps<float, 4>(p, s) : conv_fwd_taps<float, 1>(p, s);
    return conv_aligned(p, 8, 2) ? conv_fwd_taps<__nv_bfloat16, 8>(p, s) : conv_fwd_taps<__nv_bfloat16, 1>(p, s);
}

cudaError_t launch_conv_bwd(const ConvParams &p, int dtype, cudaStream_t s) {
    if (dtype == 0) return conv_aligned(p, 4, 4) ? conv_bwd_taps<float, 4>(p, s) : conv_bwd_taps<float, 1>(p, s);
    return conv_aligned(p, 4, 2) ? conv_bwd_taps<__nv_bfloat16, 4>(p, s) : conv_bwd_taps<__nv_bfloat16, 1>(p, s);
}

}  // namespace gdn

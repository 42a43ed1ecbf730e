// gdn_conv.cu -- the short causal convolution in front of the recurrence, its carried state, and
// its VJP.
//
//     pre[t,c] = bias[c] + sum_{j < W} w[c,j] x~[t-W+1+j,c],   y = act(pre)
// with x~ the carried state (W-1 inputs) followed by x. For cotangents dy of y and ds_T of the
// state behind the last valid step:
//     dpre = dy act'(pre),   dx~[s] = sum_j w[j] dpre[s+W-1-j] (+ ds_T where s is one of the last
//     W-1 inputs),   dw[j] = sum_t dpre[t] x~[t-W+1+j],   dbias = sum_t dpre[t]
//
// A thread takes V neighbouring channels (four, fewer where they are not aligned) and walks a run of
// steps with the last W-1 inputs in registers, so that x is read once and the taps once per run. Each channel's W products
// are far below the memory time: the kernels are bound by the bytes of x and y (and dy, dx).
// Measured on 8 x 4096 steps of 8192 channels, 4 taps, SiLU, bf16: forward 161 us, 6.7 TB/s, a plain
// copy's rate; backward 290 us, 5.6 TB/s of x, dy and dx, instructions issuing in 53 % of the cycles:
// it forms pre and its sigmoid again, and adds up W + 1 sums per channel. float32: 322 and 497 us.
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

// Channels in pairs, for the packed float32 instructions (V = 1: the second of the pair is unused).
template <int V>
constexpr int kPairs = V / 2 > 0 ? V / 2 : 1;

template <int V>
__device__ __forceinline__ void to_pairs(const float (&x)[V], float2 (&o)[kPairs<V>]) {
#pragma unroll
    for (int i = 0; i < kPairs<V>; ++i) o[i] = make_float2(x[V > 1 ? 2 * i : 0], V > 1 ? x[2 * i + 1] : 0.f);
}
template <int V>
__device__ __forceinline__ void from_pairs(const float2 (&x)[kPairs<V>], float (&o)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = v % 2 ? x[v / 2].y : x[v / 2].x;
}

// The taps and the bias of V channels.
template <int W, int V>
__device__ __forceinline__ void load_taps(const ConvParams &p, int c, float2 (&w)[W][kPairs<V>], float2 (&bias)[kPairs<V>]) {
    float flat[V * W], bs[V];
    if constexpr (V * W % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V * W / 4; ++i) {
            const float4 q = *reinterpret_cast<const float4 *>(p.w + (size_t)c * W + 4 * i);
            flat[4 * i] = q.x; flat[4 * i + 1] = q.y; flat[4 * i + 2] = q.z; flat[4 * i + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V * W; ++i) flat[i] = p.w[(size_t)c * W + i];
    }
#pragma unroll
    for (int v = 0; v < V; ++v) bs[v] = p.bias ? p.bias[c + v] : 0.f;
    to_pairs<V>(bs, bias);
#pragma unroll
    for (int j = 0; j < W; ++j) {
        float col[V];
#pragma unroll
        for (int v = 0; v < V; ++v) col[v] = flat[v * W + j];
        to_pairs<V>(col, w[j]);
    }
}

// A thread's own inputs of the next steps, kBlocks blocks of kStep steps: asynchronous copies into its
// own places in shared memory (no other thread reads them, so no barrier is needed), which keep some
// 50 KB per SM in flight without registers. Elements of 2 bytes alone (V = 1, bf16) are below the
// smallest copy: they are loaded a block ahead into registers.
constexpr int kStep = 8, kBlocks = 2;

template <typename T, int V, int THREADS>
struct Ring {
    static constexpr bool kAsync = V * sizeof(T) >= 4;
    static constexpr int kBytes = kAsync ? kBlocks * kStep * THREADS * V * (int)sizeof(T) : 0;
    Raw<T, V> *mine;
    const T *src;
    long long ld;
    int end;              // steps from `end` on read as zeros
    T now[kAsync ? 1 : kStep], next[kAsync ? 1 : kStep];
    static_assert(kBlocks == 2, "the register form holds two blocks");

    __device__ __forceinline__ Ring(void *smem, const T *src, long long ld, int end)
        : mine(static_cast<Raw<T, V> *>(smem) + threadIdx.x), src(src), ld(ld), end(end) {}
    // starts the copies of steps t .. t + kStep - 1, block number blk
    __device__ __forceinline__ void start(int blk, int t) {
        if constexpr (kAsync) {
#pragma unroll
            for (int i = 0; i < kStep; ++i) {
                const bool ok = t + i < end;
                const T *from = ok ? src + (size_t)(t + i) * ld : src;
                const uint32_t to = smem_addr(mine + ((blk & (kBlocks - 1)) * kStep + i) * THREADS);
                if constexpr (V * sizeof(T) == 16)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(ok ? 16 : 0) : "memory");
                else
                    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(to), "l"(from),
                                 "r"(ok ? (int)(V * sizeof(T)) : 0), "n"(V * (int)sizeof(T))
                                 : "memory");
            }
        } else {
#pragma unroll
            for (int i = 0; i < kStep; ++i) {
                now[i] = next[i];
                next[i] = from_f32<T>(0.f);
                if (t + i < end) next[i] = src[(size_t)(t + i) * ld];
            }
        }
    }
    // step i of block blk
    __device__ __forceinline__ void get(int blk, int i, float (&o)[V]) const {
        if constexpr (kAsync) unpack<T, V>(mine[((blk & (kBlocks - 1)) * kStep + i) * THREADS], o);
        else o[0] = to_f32(now[i]);
    }
};

}  // namespace

// Threads over (batch row, run of `run` steps, V channels). The thread of a row's first run also
// writes the state behind the row's last valid step. The next U steps' inputs are loaded before the
// present ones are used; groups of U steps inside the row and the run take a path without tests.
template <typename T, int W, int V, bool SILU>
__global__ void __launch_bounds__(kConvThreads, 4) conv_fwd_kernel(ConvParams p, int run, int runs) {
    constexpr int U = kStep, P = kPairs<V>;
    extern __shared__ __align__(16) unsigned char smem[];
    const int CV = p.C / V;
    const size_t id = (size_t)blockIdx.x * kConvThreads + threadIdx.x;
    if (id >= (size_t)p.B * runs * CV) return;
    const int c = (int)(id % CV) * V;
    const size_t rb = id / CV;
    const int r = (int)(rb % runs), b = (int)(rb / runs);
    const int L = row_length(p.lens, b, p.T);
    const int t0 = r * run, t1 = min(t0 + run, p.T), t_in = min(t1, L);
    const T *x = static_cast<const T *>(p.x) + (size_t)b * p.T * p.ldx + c;
    T *y = static_cast<T *>(p.y) + (size_t)b * p.T * p.C + c;
    Ring<T, V, kConvThreads> in(smem, x, p.ldx, t_in);
#pragma unroll
    for (int k = 0; k < kBlocks - 1; ++k) {
        in.start(k, t0 + k * U);
        cp_async_commit();
    }
    float2 w[W][P], bias[P], win[W][P];
    load_taps<W, V>(p, c, w, bias);
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
        float e[V] = {};
        if (t0 + i - (W - 1) < L) load_input<T, V>(p, W, b, t0 + i - (W - 1), c, e);
        to_pairs<V>(e, win[i]);
    }
    if (r == 0 && p.s_T != nullptr) {
        float keep[W][V];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) load_input<T, V>(p, W, b, L - (W - 1) + j, c, keep[j]);
        T *out = static_cast<T *>(p.s_T) + (size_t)b * (W - 1) * p.C + c;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) store_vec<T, V>(out + (size_t)j * p.C, keep[j]);
    }
    auto step = [&](int blk, int i, int tb, bool valid) {
        float o[V], e[V];
        in.get(blk, i, e);
        to_pairs<V>(e, win[W - 1]);
        float2 pre[P];
#pragma unroll
        for (int q = 0; q < P; ++q) {
            pre[q] = bias[q];
#pragma unroll
            for (int j = 0; j < W; ++j) pre[q] = __ffma2_rn(w[j][q], win[j][q], pre[q]);
#pragma unroll
            for (int j = 0; j < W - 1; ++j) win[j][q] = win[j + 1][q];
            if (SILU) pre[q] = __fmul2_rn(pre[q], sigmoid2_hw(pre[q]));
        }
        from_pairs<V>(pre, o);
        if (!valid)
#pragma unroll
            for (int v = 0; v < V; ++v) o[v] = 0.f;
        store_vec<T, V>(y + (size_t)(tb + i) * p.C, o);
    };
    for (int tb = t0, blk = 0; tb < t1; tb += U, ++blk) {
        in.start(blk + kBlocks - 1, tb + (kBlocks - 1) * U);
        cp_async_commit();
        cp_async_wait<kBlocks - 1>();
        if (tb + U <= t_in) {
#pragma unroll
            for (int i = 0; i < U; ++i) step(blk, i, tb, true);
        } else {
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (tb + i < t1) step(blk, i, tb, tb + i < L);
        }
    }
}

// A CTA takes 32 V channels and 8 runs of steps (one per warp) of one batch row. A thread forms dpre
// for its run and the W-1 steps before it; dx[s] is complete, and stored, at step s + W-1, so a run
// stores the inputs from W-1 steps before it on, and the row's last run goes on for W-1 steps behind
// the row (where dpre is 0). The parameter sums go over a thread's steps, then over the CTA's warps in
// ascending order, into the CTA's slice of the partial sums: a fixed order.
template <typename T, int W, int V, bool SILU>
__global__ void __launch_bounds__(32 * kConvBwdWarps, 2) conv_bwd_kernel(ConvParams p, int run, int slices_row) {
    constexpr int U = kStep, P = kPairs<V>;
    using In = Ring<T, V, 32 * kConvBwdWarps>;
    extern __shared__ __align__(16) unsigned char smem[];
    auto &sums = *reinterpret_cast<float(*)[kConvBwdWarps][W + 1][32 * V]>(smem);   // over the rings, behind the steps
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c0 = (int)(blockIdx.y + blockIdx.z * gridDim.y) * 32 * V, c = c0 + lane * V;   // may lie past the channels
    const int b = blockIdx.x / slices_row, sl = blockIdx.x % slices_row;
    const int L = row_length(p.lens, b, p.T);
    const int t0 = (sl * kConvBwdWarps + warp) * run, t1 = min(t0 + run, p.T);
    float2 dw[W][P], db[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        db[i] = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][i] = make_float2(0.f, 0.f);
    }
    if (c < p.C && t0 < t1) {
        const int t_in = min(t1, L), t_end = t1 == p.T ? t1 + W - 1 : t1;
        const T *x = static_cast<const T *>(p.x) + (size_t)b * p.T * p.ldx + c;
        const T *dy = static_cast<const T *>(p.dy) + (size_t)b * p.T * p.C + c;
        const T *ds_T = static_cast<const T *>(p.ds_T) + (size_t)b * (W - 1) * p.C + c;
        T *dx = static_cast<T *>(p.dx) + (size_t)b * p.T * p.C + c;
        T *ds0 = static_cast<T *>(p.ds0) + (size_t)b * (W - 1) * p.C + c;
        In in_x(smem, x, p.ldx, t_in), in_d(smem + In::kBytes, dy, p.C, t_in);
        auto start = [&](int blk, int t) {
            in_x.start(blk, t);
            in_d.start(blk, t);
            cp_async_commit();
        };
#pragma unroll
        for (int k = 0; k < kBlocks - 1; ++k) start(k, t0 + k * U);
        float2 w[W][P], bias[P], win[W][P], dwin[W][P];
        load_taps<W, V>(p, c, w, bias);
        // dpre of one step from the window whose newest input is in place, into dwin[W - 1]
        auto grad = [&](const float (&d)[V], bool valid) {
            float2 dd[P];
            to_pairs<V>(d, dd);
#pragma unroll
            for (int q = 0; q < P; ++q) {
                float2 pre = bias[q];
#pragma unroll
                for (int j = 0; j < W; ++j) pre = __ffma2_rn(w[j][q], win[j][q], pre);
                if (SILU) {              // silu' = s (1 + pre (1 - s))
                    const float2 one = make_float2(1.f, 1.f), sg = sigmoid2_hw(pre);
                    const float2 up = __ffma2_rn(pre, __ffma2_rn(sg, make_float2(-1.f, -1.f), one), one);
                    dd[q] = __fmul2_rn(dd[q], __fmul2_rn(sg, up));
                }
                dwin[W - 1][q] = valid ? dd[q] : make_float2(0.f, 0.f);
            }
        };
        auto shift = [&](float2(&a)[W][P]) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int i = 0; i < P; ++i) a[j][i] = a[j + 1][i];
        };
        // the windows in front of the run: inputs from t0 - 2 (W-1) on, dpre from t0 - (W-1) on
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int i = 0; i < P; ++i) win[j][i] = dwin[j][i] = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 2 * (W - 1); ++i) {
            const int t = t0 - 2 * (W - 1) + i;
            float e[V] = {}, d[V] = {};
            if (t < L) load_input<T, V>(p, W, b, t, c, e);
            to_pairs<V>(e, win[W - 1]);
            if (i >= W - 1) {
                const bool valid = t >= 0 && t < L;
                if (valid) load_vec<T, V>(dy + (size_t)t * p.C, d);
                grad(d, valid);
                shift(dwin);
            }
            shift(win);
        }
        // one step: the sums, and dx of the input W-1 steps back
        auto step = [&](int blk, int i, int tb, bool valid, float (&o)[V]) {
            float e[V], d[V];
            in_x.get(blk, i, e);
            in_d.get(blk, i, d);
            to_pairs<V>(e, win[W - 1]);
            grad(d, valid);
            float2 s[P];
#pragma unroll
            for (int q = 0; q < P; ++q) {
                db[q] = __fadd2_rn(db[q], dwin[W - 1][q]);
#pragma unroll
                for (int j = 0; j < W; ++j) {    // 0 x a carried state that is not finite would be NaN
                    const float2 in = valid ? win[j][q] : make_float2(0.f, 0.f);
                    dw[j][q] = __ffma2_rn(dwin[W - 1][q], in, dw[j][q]);
                }
                s[q] = __fmul2_rn(w[0][q], dwin[W - 1][q]);
#pragma unroll
                for (int j = 1; j < W; ++j) s[q] = __ffma2_rn(w[j][q], dwin[W - 1 - j][q], s[q]);
            }
            from_pairs<V>(s, o);
            shift(win);
            shift(dwin);
        };
        for (int tb = t0, blk = 0; tb < t_end; tb += U, ++blk) {
            start(blk + kBlocks - 1, tb + (kBlocks - 1) * U);
            cp_async_wait<kBlocks - 1>();
            float o[V];
            if (tb >= W - 1 && tb + U <= t_in) {      // inside the row: the state takes no part
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    step(blk, i, tb, true, o);
                    store_vec<T, V>(dx + (size_t)(tb + i - (W - 1)) * p.C, o);
                }
                continue;
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int t = tb + i, s = t - (W - 1);
                if (t >= t_end) break;
                step(blk, i, tb, t < L, o);
                // s is input s of the row, or row t of the state in front of it; either may be one of
                // the W-1 inputs behind the last valid step
                const int j = s - (L - (W - 1));
                if (p.ds_T != nullptr && j >= 0 && j < W - 1) {
                    float e[V];
                    load_vec<T, V>(ds_T + (size_t)j * p.C, e);
#pragma unroll
                    for (int v = 0; v < V; ++v) o[v] += e[v];
                }
                if (s >= 0) store_vec<T, V>(dx + (size_t)s * p.C, o);
                else if (p.ds0 != nullptr) store_vec<T, V>(ds0 + (size_t)t * p.C, o);
            }
        }
    }
    cp_async_wait<0>();
    __syncthreads();
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        float e[V];
        from_pairs<V>(j < W ? dw[j < W ? j : 0] : db, e);
#pragma unroll
        for (int v = 0; v < V; ++v) sums[warp][j][lane * V + v] = e[v];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (W + 1) * 32 * V; i += 32 * kConvBwdWarps) {
        const int j = i / (32 * V), cc = i % (32 * V);
        if (c0 + cc >= p.C) continue;
        float a = 0.f;
#pragma unroll
        for (int k = 0; k < kConvBwdWarps; ++k) a += sums[k][j][cc];
        p.part[((size_t)blockIdx.x * (W + 1) + j) * p.C + c0 + cc] = a;
    }
}

// dw[c][j] and dbias[c] from the slices' partial sums.
__global__ void __launch_bounds__(256) conv_reduce_kernel(ConvParams p, int slices) {
    const size_t n = (size_t)(p.W + 1) * p.C, i = (size_t)blockIdx.x * 32 + threadIdx.x;
    const float a = slice_sum(p.part, slices, n, blockIdx.x);
    if (threadIdx.x >= 32 || i >= n) return;
    const int j = (int)(i / p.C), c = (int)(i % p.C);
    if (j < p.W) p.dw[(size_t)c * p.W + j] = a;
    else if (p.dbias != nullptr) p.dbias[c] = a;
}

namespace {

bool conv_aligned(const ConvParams &p, int V, size_t e) {
    return p.C % V == 0 && p.ldx % V == 0 && (uintptr_t)p.x % (V * e) == 0;
}

// Steps per warp of the backward: up to 256, fewer while that leaves under 512 CTAs (3 per SM). 8 x
// 4096 steps of 8192 channels: 290 us, 318 with runs of 64, whose first steps are read twice; 4 x 128
// steps of 1024 channels, where runs are cut to 8: 7 us, 9 uncut.
int conv_bwd_run(const ConvParams &p) {
    int run = (p.T + kConvBwdWarps - 1) / kConvBwdWarps;
    run = run > 256 ? 256 : run;
    const long long cols = (p.C + 127) / 128;
    while (run > 8 && cols * p.B * ((p.T + kConvBwdWarps * run - 1) / (kConvBwdWarps * run)) < 512) run /= 2;
    return run;
}

template <typename T, int W, int V, bool SILU>
cudaError_t conv_fwd_launch(const ConvParams &p, cudaStream_t s) {
    // Steps per thread: each run reads W-1 inputs again, so up to 64, fewer while the threads would
    // not fill the SMs. 8 x 4096 steps of 8192 channels: 161 us, 208 with runs of 16; 4 x 128 steps of
    // 1024 channels, where runs are cut to 1: 6 us, 10 uncut.
    const size_t cv = p.C / V;
    int run = 64;
    while (run > 1 && (size_t)p.B * ((p.T + run - 1) / run) * cv < (size_t)152 * 1024) run /= 2;
    const int runs = (p.T + run - 1) / run;
    const size_t n = (size_t)p.B * runs * cv;
    timing_mark("conv_fwd", 0, s);
    constexpr int smem = Ring<T, V, kConvThreads>::kBytes;
    if (smem > 48 * 1024) {
        const cudaError_t e = allow_smem<conv_fwd_kernel<T, W, V, SILU>>(smem);
        if (e != cudaSuccess) return e;
    }
    conv_fwd_kernel<T, W, V, SILU><<<(unsigned)((n + kConvThreads - 1) / kConvThreads), kConvThreads, smem, s>>>(p, run, runs);
    timing_mark("conv_fwd", 1, s);
    return cudaGetLastError();
}

template <typename T, int W, int V, bool SILU>
cudaError_t conv_bwd_launch(const ConvParams &p, cudaStream_t s) {
    const int run = conv_bwd_run(p), slices_row = (p.T + kConvBwdWarps * run - 1) / (kConvBwdWarps * run);
    const int slices = p.B * slices_row;
    timing_mark("conv_bwd", 0, s);
    constexpr int ring = 2 * Ring<T, V, 32 * kConvBwdWarps>::kBytes, sums = kConvBwdWarps * (W + 1) * 32 * V * 4;
    constexpr int smem = ring > sums ? ring : sums;
    cudaError_t e = allow_smem<conv_bwd_kernel<T, W, V, SILU>>(smem);
    if (e != cudaSuccess) return e;
    // blocks of channels over y and, where one axis of the grid (65535) does not hold them, z
    const int blocks = (p.C + 32 * V - 1) / (32 * V), z = (blocks + 65534) / 65535, y = (blocks + z - 1) / z;
    conv_bwd_kernel<T, W, V, SILU><<<dim3(slices, y, z), 32 * kConvBwdWarps, smem, s>>>(p, run, slices_row);
    timing_mark("conv_bwd", 1, s);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    timing_mark("conv_reduce", 0, s);
    conv_reduce_kernel<<<(unsigned)(((size_t)(W + 1) * p.C + 31) / 32), 256, 0, s>>>(p, slices);
    timing_mark("conv_reduce", 1, s);
    return cudaGetLastError();
}

template <typename T, int W, int V>
cudaError_t conv_act(const ConvParams &p, bool bwd, cudaStream_t s) {
    if (bwd) return p.act == kActSilu ? conv_bwd_launch<T, W, V, true>(p, s) : conv_bwd_launch<T, W, V, false>(p, s);
    return p.act == kActSilu ? conv_fwd_launch<T, W, V, true>(p, s) : conv_fwd_launch<T, W, V, false>(p, s);
}
template <typename T, int V>
cudaError_t conv_taps(const ConvParams &p, bool bwd, cudaStream_t s) {
    switch (p.W) {
        case 1: return conv_act<T, 1, V>(p, bwd, s);
        case 2: return conv_act<T, 2, V>(p, bwd, s);
        case 3: return conv_act<T, 3, V>(p, bwd, s);
        default: return conv_act<T, 4, V>(p, bwd, s);
    }
}

// Four channels per thread, or two or one where four are not aligned (forward and backward of 8 x 4096
// steps of 8192 channels: 462 us by fours, 596 by pairs, 1034 one by one).
cudaError_t conv_any(const ConvParams &p, int dtype, bool bwd, cudaStream_t s) {
    if (dtype == 0) return conv_aligned(p, 4, 4) ? conv_taps<float, 4>(p, bwd, s) : conv_taps<float, 1>(p, bwd, s);
    if (conv_aligned(p, 4, 2)) return conv_taps<__nv_bfloat16, 4>(p, bwd, s);
    return conv_aligned(p, 2, 2) ? conv_taps<__nv_bfloat16, 2>(p, bwd, s) : conv_taps<__nv_bfloat16, 1>(p, bwd, s);
}

}  // namespace

int conv_bwd_slices(const ConvParams &p) {
    const int run = conv_bwd_run(p);
    return p.B * ((p.T + kConvBwdWarps * run - 1) / (kConvBwdWarps * run));
}

cudaError_t launch_conv_fwd(const ConvParams &p, int dtype, cudaStream_t s) { return conv_any(p, dtype, false, s); }
cudaError_t launch_conv_bwd(const ConvParams &p, int dtype, cudaStream_t s) { return conv_any(p, dtype, true, s); }

}  // namespace gdn

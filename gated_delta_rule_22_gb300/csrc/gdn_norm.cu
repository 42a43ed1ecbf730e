// gdn_norm.cu -- group norm over the channels of each row, with an activation or a gate, and its VJP.
//
// Row m, group g of D channels: xh = (x - mean) rstd, rstd = 1 / sqrt(var + eps) (center = 0: mean
// taken as 0 and var as mean(x^2)), aff = xh w + b, y = act(aff) or y = aff act(z). Backward:
//     daff = dy act'(aff)   or   daff = dy act(z), dz = dy aff act'(z)
//     dxh = daff w,  dx = rstd (dxh - mean(dxh) - xh mean(dxh xh))   (center = 0: no mean(dxh) term)
//     dw = sum_m daff xh,  db = sum_m daff
// Bound by memory: x (and z, dy) are read once and stay in registers between the statistics and
// the output. The mean is subtracted before the squares are summed. Measured on 32768 rows of 32
// groups of 128 channels with a gate, bf16: forward 132 us, 6.1 TB/s; backward 243 us, 5.5 TB/s of x, z,
// dy, dx and dz (float32: 253 and 486 us). 8192 rows of one group of 4096: 41 and 92 us, 4.9 and 3.6 TB/s, a barrier per sum.
#include "gdn_layer.cuh"

#include <type_traits>

namespace gdn {

namespace {

constexpr int kNormThreads = 256;
constexpr int kNormWarps = kNormThreads / 32;

__device__ __forceinline__ float act_rt(int act, float x) {
    return act == kActSilu ? silu_hw(x) : act == kActGelu ? gelu_f(x) : x;
}
__device__ __forceinline__ float dact_rt(int act, float x) {
    return act == kActSilu ? dsilu_hw(x) : act == kActGelu ? dgelu_f(x) : 1.f;
}

// Sums over the LPG lanes of a group (a part of a warp; kNormThreads: the CTA, through shared memory,
// two buffers in turn so that one barrier per sum is enough).
template <int LPG>
struct GroupSum {
    int turn = 0;
    __device__ __forceinline__ float2 operator()(float2 x) {
        constexpr int W = LPG < 32 ? LPG : 32;
#pragma unroll
        for (int m = W / 2; m >= 1; m >>= 1)
            x = __fadd2_rn(x, make_float2(__shfl_xor_sync(kFullMask, x.x, m), __shfl_xor_sync(kFullMask, x.y, m)));
        if constexpr (LPG > 32) {
            __shared__ float2 buf[2][kNormWarps];
            if ((threadIdx.x & 31) == 0) buf[turn][threadIdx.x >> 5] = x;
            __syncthreads();
            x = buf[turn][0];
#pragma unroll
            for (int w = 1; w < kNormWarps; ++w) x = __fadd2_rn(x, buf[turn][w]);
            turn ^= 1;
        }
        return x;
    }
    __device__ __forceinline__ float operator()(float x) {
        if constexpr (LPG > 32) {
            return (*this)(make_float2(x, 0.f)).x;
        } else {
#pragma unroll
            for (int m = LPG / 2; m >= 1; m >>= 1) x += __shfl_xor_sync(kFullMask, x, m);
            return x;
        }
    }
};

// sum / D with one correction of the quotient by its remainder: the product with 1 / D alone is often an
// ulp off, and a group of equal values then has a variance, which counts where ulp^2 nears eps.
__device__ __forceinline__ float mean_of(float sum, int D, float inv_D) {
    const float q = sum * inv_D;
    return fmaf(fmaf(-q, (float)D, sum), inv_D, q);
}

__device__ __forceinline__ float block_sum(float x, float *buf) {
    x = warp_sum(x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kNormWarps; ++w) s += buf[w];
    return s;
}

}  // namespace

// A lane's E elements as pairs, for the packed float32 instructions (E = 1: the second is unused).
template <int E>
struct Pairs {
    static constexpr int N = (E + 1) / 2;
    float2 p[N];
    __device__ __forceinline__ void fill(float x) {
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = make_float2(x, x);
    }
    __device__ __forceinline__ void set(int e, float x) {
        if (e % 2) p[e / 2].y = x;
        else p[e / 2].x = x;
    }
    __device__ __forceinline__ float get(int e) const { return e % 2 ? p[e / 2].y : p[e / 2].x; }
    __device__ __forceinline__ float total() const {
        float2 s = p[0];
#pragma unroll
        for (int i = 1; i < N; ++i) s = __fadd2_rn(s, p[i]);
        return E == 1 ? s.x : s.x + s.y;
    }
};

// act(x) and, where asked, act'(x) of a pair
template <int ACT>
__device__ __forceinline__ float2 act2(float2 x) {
    if (ACT == kActSilu) return __fmul2_rn(x, sigmoid2_hw(x));
    if (ACT == kActGelu) return make_float2(gelu_f(x.x), gelu_f(x.y));
    return x;
}
template <int ACT>
__device__ __forceinline__ float2 act2(float2 x, float2 &slope) {
    if (ACT == kActSilu) {
        const float2 one = make_float2(1.f, 1.f), s = sigmoid2_hw(x);
        slope = __fmul2_rn(s, __ffma2_rn(x, __ffma2_rn(s, make_float2(-1.f, -1.f), one), one));
        return __fmul2_rn(x, s);
    }
    if (ACT == kActGelu) {
        slope = make_float2(dgelu_f(x.x), dgelu_f(x.y));
        return make_float2(gelu_f(x.x), gelu_f(x.y));
    }
    slope = make_float2(1.f, 1.f);
    return x;
}

// f<ACT>() for the activation of the call: the test is made once per row, not per element.
template <typename F>
__device__ __forceinline__ void with_act(int act, F f) {
    if (act == kActSilu) f(std::integral_constant<int, kActSilu>());
    else if (act == kActGelu) f(std::integral_constant<int, kActGelu>());
    else f(std::integral_constant<int, kActNone>());
}

// Where a lane's elements lie: LPG lanes per group, V neighbouring channels per lane, IT pieces
// (D <= LPG V IT). A warp takes 32 / LPG groups of a row; with LPG = kNormThreads a CTA takes one group.
template <typename T, int V, int LPG, int IT>
struct NormLane {
    static constexpr int E = V * IT, kGroups = LPG < 32 ? 32 / LPG : 1;    // groups of a warp (or CTA)
    static constexpr int kRows = LPG <= 32 ? kNormWarps : 1;               // rows that a CTA takes at once
    int g, j;
    size_t col;
    bool ok[IT], full;
    __device__ __forceinline__ explicit NormLane(const NormParams &p) {
        const int lane = LPG <= 32 ? threadIdx.x & 31 : threadIdx.x;
        g = blockIdx.y * kGroups + lane / LPG;
        j = lane % LPG;
        col = (size_t)g * p.D + j * V;
#pragma unroll
        for (int i = 0; i < IT; ++i) ok[i] = g < p.G && (i * LPG + j) * V < p.D;
        full = p.D == LPG * V * IT && p.G % kGroups == 0;
    }
    // parameters of the lane's channels (w, b), or `other`
    __device__ __forceinline__ void params(const float *w, float other, Pairs<E> &o) const {
        o.fill(other);
        if (w == nullptr) return;
#pragma unroll
        for (int i = 0; i < IT; ++i)
            if (ok[i])
#pragma unroll
                for (int v = 0; v < V; ++v) o.set(i * V + v, w[col + i * LPG * V + v]);
    }
    __device__ __forceinline__ void load(const void *t, size_t at, Raw<T, V> (&o)[IT]) const {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            o[i] = Raw<T, V>();
            if (ok[i]) o[i] = load_raw<T, V>(static_cast<const T *>(t) + at + col + i * LPG * V);
        }
    }
    __device__ __forceinline__ void floats(const Raw<T, V> (&r)[IT], Pairs<E> &o) const {
        if (E == 1) o.p[0].y = 0.f;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            float e[V];
            unpack<T, V>(r[i], e);
#pragma unroll
            for (int v = 0; v < V; ++v) o.set(i * V + v, e[v]);
        }
    }
    __device__ __forceinline__ void store(void *t, size_t at, const Pairs<E> &x) const {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            float e[V];
#pragma unroll
            for (int v = 0; v < V; ++v) e[v] = x.get(i * V + v);
            if (ok[i]) store_vec<T, V>(static_cast<T *>(t) + at + col + i * LPG * V, e);
        }
    }
    // zeros in the places beyond the group
    __device__ __forceinline__ void mask(Pairs<E> &x) const {
        if (full) return;
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (!ok[e / V]) x.set(e, 0.f);
    }
};

// A warp keeps its groups' w and b in registers over the rows that it walks, and loads the next row
// while it works on one.
template <typename T, int V, int LPG, int IT>
__global__ void __launch_bounds__(kNormThreads) norm_fwd_kernel(NormParams p) {
    constexpr int E = V * IT, P = Pairs<E>::N;
    const NormLane<T, V, LPG, IT> at(p);
    GroupSum<LPG> group_sum;
    const int rows = gridDim.x * at.kRows;
    int m = blockIdx.x * at.kRows + (threadIdx.x >> 5) % at.kRows;
    Raw<T, V> rx[IT], rz[IT];
    auto fetch = [&](int row) {
        at.load(p.x, (size_t)row * p.ldx, rx);
        if (p.z != nullptr) at.load(p.z, (size_t)row * p.ldz, rz);
    };
    if (m < p.M) fetch(m);
    Pairs<E> w, b;
    at.params(p.w, 1.f, w);
    at.params(p.b, 0.f, b);
    const float inv_D = 1.f / p.D;
    for (; m < p.M; m += rows) {
        Pairs<E> x, z;
        at.floats(rx, x);
        if (p.z != nullptr) at.floats(rz, z);
        if (m + rows < p.M) fetch(m + rows);
        float mean = 0.f;
        if (p.center) {
            mean = mean_of(group_sum(x.total()), p.D, inv_D);
#pragma unroll
            for (int i = 0; i < P; ++i) x.p[i] = __fadd2_rn(x.p[i], make_float2(-mean, -mean));
            at.mask(x);
        }
        Pairs<E> sq;
#pragma unroll
        for (int i = 0; i < P; ++i) sq.p[i] = __fmul2_rn(x.p[i], x.p[i]);
        const float rstd = 1.f / sqrtf(fmaf(group_sum(sq.total()), inv_D, p.eps));
        if (p.stats != nullptr && at.j == 0 && at.g < p.G)
            *reinterpret_cast<float2 *>(p.stats + 2 * ((size_t)m * p.G + at.g)) = make_float2(mean, rstd);
        with_act(p.act, [&](auto act) {
            constexpr int ACT = decltype(act)::value;
#pragma unroll
            for (int i = 0; i < P; ++i) x.p[i] = __ffma2_rn(__fmul2_rn(x.p[i], make_float2(rstd, rstd)), w.p[i], b.p[i]);
            if (p.z != nullptr) {
#pragma unroll
                for (int i = 0; i < P; ++i) x.p[i] = __fmul2_rn(x.p[i], act2<ACT>(z.p[i]));
            } else {
#pragma unroll
                for (int i = 0; i < P; ++i) x.p[i] = act2<ACT>(x.p[i]);
            }
        });
        at.store(p.y, (size_t)m * p.G * p.D, x);
    }
}

// The same layout. The parameter gradients are summed over a warp's rows, then over the CTA's warps
// in ascending order, into the CTA's slice of the partial sums.
template <typename T, int V, int LPG, int IT>
__global__ void __launch_bounds__(kNormThreads) norm_bwd_kernel(NormParams p) {
    constexpr int E = V * IT, P = Pairs<E>::N;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const NormLane<T, V, LPG, IT> at(p);
    GroupSum<LPG> group_sum;
    const int rows = gridDim.x * at.kRows;
    int m = blockIdx.x * at.kRows + warp % at.kRows;
    const size_t C = (size_t)p.G * p.D;
    Raw<T, V> rx[IT], rz[IT], ry[IT];
    float2 rs = make_float2(0.f, 0.f);
    auto fetch = [&](int row) {
        at.load(p.x, (size_t)row * p.ldx, rx);
        at.load(p.dy, (size_t)row * C, ry);
        if (p.z != nullptr) at.load(p.z, (size_t)row * p.ldz, rz);
        if (at.g < p.G) rs = *reinterpret_cast<const float2 *>(p.stats_in + 2 * ((size_t)row * p.G + at.g));
    };
    if (m < p.M) fetch(m);
    Pairs<E> w, b, dw, db;
    at.params(p.w, 1.f, w);
    at.params(p.b, 0.f, b);
    dw.fill(0.f);
    db.fill(0.f);
    const float inv_D = 1.f / p.D;
    for (; m < p.M; m += rows) {
        Pairs<E> x, z, g;
        const float2 st = rs;
        at.floats(rx, x);
        at.floats(ry, g);
        if (p.z != nullptr) at.floats(rz, z);
        if (m + rows < p.M) fetch(m + rows);
#pragma unroll
        for (int i = 0; i < P; ++i) x.p[i] = __fmul2_rn(__fadd2_rn(x.p[i], make_float2(-st.x, -st.x)), make_float2(st.y, st.y));
        at.mask(x);
        with_act(p.act, [&](auto act) {
            constexpr int ACT = decltype(act)::value;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float2 aff = __ffma2_rn(x.p[i], w.p[i], b.p[i]);
                float2 slope;
                if (p.z != nullptr) {
                    const float2 gate = act2<ACT>(z.p[i], slope);
                    z.p[i] = __fmul2_rn(__fmul2_rn(g.p[i], aff), slope);      // dz
                    g.p[i] = __fmul2_rn(g.p[i], gate);
                } else {
                    act2<ACT>(aff, slope);
                    g.p[i] = __fmul2_rn(g.p[i], slope);
                }
            }
        });
        Pairs<E> gx;
#pragma unroll
        for (int i = 0; i < P; ++i) {                     // g: daff, then dxh
            db.p[i] = __fadd2_rn(db.p[i], g.p[i]);
            dw.p[i] = __ffma2_rn(g.p[i], x.p[i], dw.p[i]);
            g.p[i] = __fmul2_rn(g.p[i], w.p[i]);
            gx.p[i] = __fmul2_rn(g.p[i], x.p[i]);
        }
        if (p.dz != nullptr) at.store(p.dz, (size_t)m * C, z);
        const float2 sums = group_sum(make_float2(g.total(), gx.total()));
        const float s1 = p.center ? sums.x * inv_D : 0.f, s2 = sums.y * inv_D;
#pragma unroll
        for (int i = 0; i < P; ++i)
            x.p[i] = __fmul2_rn(__fadd2_rn(__ffma2_rn(x.p[i], make_float2(-s2, -s2), g.p[i]), make_float2(-s1, -s1)), make_float2(st.y, st.y));
        at.store(p.dx, (size_t)m * C, x);
    }
    float *part = p.part + (size_t)blockIdx.x * 2 * C;
    if constexpr (LPG > 32) {                             // every thread has channels of its own
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = (e / V * LPG + at.j) * V + e % V;
            if (!at.ok[e / V]) continue;
            part[(size_t)at.g * p.D + c] = dw.get(e);
            part[C + (size_t)at.g * p.D + c] = db.get(e);
        }
    } else {
        __shared__ float sums[2][kNormWarps][32 * E];
#pragma unroll
        for (int i = 0; i < IT; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                sums[0][warp][(i * 32 + lane) * V + v] = dw.get(i * V + v);
                sums[1][warp][(i * 32 + lane) * V + v] = db.get(i * V + v);
            }
        __syncthreads();
        for (int k = threadIdx.x; k < 2 * 32 * E; k += kNormThreads) {
            const int which = k / (32 * E), n = k % (32 * E), i = n / (32 * V), ln = n / V % 32, v = n % V;
            const int gg = blockIdx.y * at.kGroups + ln / LPG, e = (i * LPG + ln % LPG) * V + v;
            if (gg >= p.G || e >= p.D) continue;
            float a = 0.f;
#pragma unroll
            for (int u = 0; u < kNormWarps; ++u) a += sums[which][u][n];
            part[which * C + (size_t)gg * p.D + e] = a;
        }
    }
}

// Groups wider than a CTA's registers take: a CTA per row and group, passes over the channels
// through the caches.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_fwd_wide_kernel(NormParams p) {
    __shared__ float buf[kNormWarps];
    const int m = blockIdx.x, g = blockIdx.y;
    const T *x = static_cast<const T *>(p.x) + (size_t)m * p.ldx + (size_t)g * p.D;
    const T *z = static_cast<const T *>(p.z) + (size_t)m * p.ldz + (size_t)g * p.D;
    T *y = static_cast<T *>(p.y) + ((size_t)m * p.G + g) * p.D;
    const float inv_D = 1.f / p.D;
    float mean = 0.f;
    if (p.center) {
        float s = 0.f;
        for (int e = threadIdx.x; e < p.D; e += kNormThreads) s += to_f32(x[e]);
        mean = mean_of(block_sum(s, buf), p.D, inv_D);
    }
    float ss = 0.f;
    for (int e = threadIdx.x; e < p.D; e += kNormThreads) {
        const float d = to_f32(x[e]) - mean;
        ss = fmaf(d, d, ss);
    }
    const float rstd = 1.f / sqrtf(fmaf(block_sum(ss, buf), inv_D, p.eps));
    if (p.stats != nullptr && threadIdx.x == 0)
        *reinterpret_cast<float2 *>(p.stats + 2 * ((size_t)m * p.G + g)) = make_float2(mean, rstd);
    for (int e = threadIdx.x; e < p.D; e += kNormThreads) {
        const float w = p.w != nullptr ? p.w[(size_t)g * p.D + e] : 1.f, b = p.b != nullptr ? p.b[(size_t)g * p.D + e] : 0.f;
        const float aff = fmaf((to_f32(x[e]) - mean) * rstd, w, b);
        y[e] = from_f32<T>(p.z != nullptr ? aff * act_rt(p.act, to_f32(z[e])) : act_rt(p.act, aff));
    }
}

// xh and daff of one channel
template <typename T>
__device__ __forceinline__ void norm_grad_at(const NormParams &p, size_t m, int g, int e, float2 st, float &xh,
                                             float &daff, float &dz) {
    const size_t ch = (size_t)g * p.D + e;
    const float w = p.w != nullptr ? p.w[ch] : 1.f, b = p.b != nullptr ? p.b[ch] : 0.f;
    const float dy = to_f32(static_cast<const T *>(p.dy)[m * p.G * p.D + ch]);
    xh = (to_f32(static_cast<const T *>(p.x)[m * p.ldx + ch]) - st.x) * st.y;
    const float aff = fmaf(xh, w, b);
    if (p.z != nullptr) {
        const float z = to_f32(static_cast<const T *>(p.z)[m * p.ldz + ch]);
        daff = dy * act_rt(p.act, z);
        dz = dy * aff * dact_rt(p.act, z);
    } else {
        daff = dy * dact_rt(p.act, aff);
        dz = 0.f;
    }
}

template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_bwd_wide_kernel(NormParams p) {
    __shared__ float buf[kNormWarps];
    const int g = blockIdx.y;
    const size_t m = blockIdx.x, out = (m * p.G + g) * p.D;
    const float2 st = *reinterpret_cast<const float2 *>(p.stats_in + 2 * (m * p.G + g));
    const float inv_D = 1.f / p.D;
    float s1 = 0.f, s2 = 0.f;
    for (int e = threadIdx.x; e < p.D; e += kNormThreads) {
        float xh, daff, dz;
        norm_grad_at<T>(p, m, g, e, st, xh, daff, dz);
        const float dxh = daff * (p.w != nullptr ? p.w[(size_t)g * p.D + e] : 1.f);
        s1 += dxh;
        s2 = fmaf(dxh, xh, s2);
        if (p.dz != nullptr) static_cast<T *>(p.dz)[out + e] = from_f32<T>(dz);
    }
    s1 = block_sum(s1, buf) * inv_D;
    s2 = block_sum(s2, buf) * inv_D;
    if (!p.center) s1 = 0.f;
    for (int e = threadIdx.x; e < p.D; e += kNormThreads) {
        float xh, daff, dz;
        norm_grad_at<T>(p, m, g, e, st, xh, daff, dz);
        const float dxh = daff * (p.w != nullptr ? p.w[(size_t)g * p.D + e] : 1.f);
        static_cast<T *>(p.dx)[out + e] = from_f32<T>(st.y * (dxh - s1 - xh * s2));
    }
}

// Partial dw, db of wide groups: a thread per channel and slice of the rows.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_bwd_wide_sums_kernel(NormParams p) {
    const size_t C = (size_t)p.G * p.D, ch = (size_t)blockIdx.x * kNormThreads + threadIdx.x;
    if (ch >= C) return;
    const int g = (int)(ch / p.D), e = (int)(ch % p.D);
    float dw = 0.f, db = 0.f;
    for (size_t m = blockIdx.y; m < (size_t)p.M; m += gridDim.y) {
        const float2 st = *reinterpret_cast<const float2 *>(p.stats_in + 2 * (m * p.G + g));
        float xh, daff, dz;
        norm_grad_at<T>(p, m, g, e, st, xh, daff, dz);
        dw = fmaf(daff, xh, dw);
        db += daff;
    }
    p.part[(size_t)blockIdx.y * 2 * C + ch] = dw;
    p.part[((size_t)blockIdx.y * 2 + 1) * C + ch] = db;
}

// dw, db from the slices' partial sums.
__global__ void __launch_bounds__(256) norm_reduce_kernel(NormParams p) {
    const size_t C = (size_t)p.G * p.D, i = (size_t)blockIdx.x * 32 + threadIdx.x;
    const float a = slice_sum(p.part, p.slices, 2 * C, blockIdx.x);
    if (threadIdx.x >= 32 || i >= 2 * C) return;
    float *out = i < C ? p.dw : p.db;
    if (out != nullptr) out[i % C] = a;
}

namespace {

// How a group lies on the lanes: V channels per lane, lanes per group (up to a warp, then a whole CTA),
// pieces of at most 16 channels in all (0: the wide kernels, which read a row again for each sum: 8192
// rows of 4096 channels, forward and backward, 345 us against 154 with a row in a CTA's registers).
struct NormGeo {
    int V, lanes, pieces;
};
NormGeo norm_geo(int D, int V) {
    NormGeo q = {V, 8, 1};
    while (q.lanes < 32 && q.lanes * V < D) q.lanes *= 2;
    if (q.lanes * V < D && D > 512) q.lanes = kNormThreads;
    while (q.lanes * V * q.pieces < D) q.pieces *= 2;
    if (V * q.pieces > 16) q.pieces = 0;
    return q;
}

// Groups and row slices of the grid: about 4 CTAs per SM, at most one warp (or CTA) per row (32768 rows
// of 32 x 128 channels, forward and backward: 385 us; 428 with 2 per SM, 393 with 8).
int norm_slices(int M, int G, const NormGeo &q) {
    const int sets = q.lanes < 32 ? (G + 32 / q.lanes - 1) / (32 / q.lanes) : G, rows = q.lanes <= 32 ? kNormWarps : 1;
    const int most = (M + rows - 1) / rows, want = (152 * 4 + sets - 1) / sets;
    return want < most ? want : most;
}

bool norm_aligned(const NormParams &p, int V, size_t e) {
    return p.D % V == 0 && p.ldx % V == 0 && p.ldz % V == 0 && (uintptr_t)p.x % (V * e) == 0 && (uintptr_t)p.z % (V * e) == 0;
}

template <typename T, int V, int LPG, int IT>
cudaError_t norm_launch(NormParams p, bool bwd, cudaStream_t s) {
    const int groups = NormLane<T, V, LPG, IT>::kGroups;
    const dim3 grid(bwd ? p.slices : norm_slices(p.M, p.G, {V, LPG, IT}), (p.G + groups - 1) / groups);
    const char *name = bwd ? "norm_bwd" : "norm_fwd";
    timing_mark(name, 0, s);
    if (bwd) norm_bwd_kernel<T, V, LPG, IT><<<grid, kNormThreads, 0, s>>>(p);
    else norm_fwd_kernel<T, V, LPG, IT><<<grid, kNormThreads, 0, s>>>(p);
    timing_mark(name, 1, s);
    return cudaGetLastError();
}

template <typename T, int V, int LPG>
cudaError_t norm_pieces(const NormParams &p, const NormGeo &q, bool bwd, cudaStream_t s) {
    if (q.pieces == 1) return norm_launch<T, V, LPG, 1>(p, bwd, s);
    if (q.pieces == 2) return norm_launch<T, V, LPG, 2>(p, bwd, s);
    if constexpr (V <= 4) {
        if (q.pieces == 4) return norm_launch<T, V, LPG, 4>(p, bwd, s);
    }
    if constexpr (V <= 2) {
        if (q.pieces == 8) return norm_launch<T, V, LPG, 8>(p, bwd, s);
    }
    if constexpr (V == 1) {
        if (q.pieces == 16) return norm_launch<T, V, LPG, 16>(p, bwd, s);
    }
    return cudaErrorInvalidValue;
}
template <typename T, int V>
cudaError_t norm_pick(const NormParams &p, const NormGeo &q, bool bwd, cudaStream_t s) {
    if (q.lanes == 8) return norm_launch<T, V, 8, 1>(p, bwd, s);
    if (q.lanes == 16) return norm_launch<T, V, 16, 1>(p, bwd, s);
    return q.lanes == 32 ? norm_pieces<T, V, 32>(p, q, bwd, s) : norm_pieces<T, V, kNormThreads>(p, q, bwd, s);
}

template <typename T>
cudaError_t norm_wide(const NormParams &p, bool bwd, cudaStream_t s) {
    const char *name = bwd ? "norm_bwd" : "norm_fwd";
    timing_mark(name, 0, s);
    if (bwd) norm_bwd_wide_kernel<T><<<dim3(p.M, p.G), kNormThreads, 0, s>>>(p);
    else norm_fwd_wide_kernel<T><<<dim3(p.M, p.G), kNormThreads, 0, s>>>(p);
    timing_mark(name, 1, s);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !bwd || (p.dw == nullptr && p.db == nullptr)) return e;
    const size_t C = (size_t)p.G * p.D;
    timing_mark("norm_sums", 0, s);
    norm_bwd_wide_sums_kernel<T><<<dim3((unsigned)((C + kNormThreads - 1) / kNormThreads), p.slices), kNormThreads, 0, s>>>(p);
    timing_mark("norm_sums", 1, s);
    return cudaGetLastError();
}

template <typename T>
cudaError_t norm_any(const NormParams &p, bool bwd, cudaStream_t s) {
    // 16 bytes; else pairs (the same case: 431 us against 385), or single channels
    constexpr int W = sizeof(T) == 2 ? 8 : 4;
    const int V = norm_aligned(p, W, sizeof(T)) ? W : norm_aligned(p, 2, sizeof(T)) ? 2 : 1;
    const NormGeo q = norm_geo(p.D, V);
    if (q.pieces == 0) return norm_wide<T>(p, bwd, s);
    if constexpr (W == 8) {
        // 8 channels per lane would leave half of the CTA idle
        if (V == W && q.lanes == kNormThreads && p.D <= 4 * kNormThreads) return norm_launch<T, 4, kNormThreads, 1>(p, bwd, s);
    }
    return V == W ? norm_pick<T, W>(p, q, bwd, s) : V == 2 ? norm_pick<T, 2>(p, q, bwd, s) : norm_pick<T, 1>(p, q, bwd, s);
}

}  // namespace

// Slices of the rows whose partial dw, db the backward sums. The size query knows no addresses, so
// the count goes by the widest layout that D allows, whatever the alignment.
int norm_bwd_slices(int M, int G, int D, int dtype) {
    const int W = dtype == 0 ? 4 : 8;
    const NormGeo q = norm_geo(D, D % W == 0 ? W : D % 2 == 0 ? 2 : 1);
    if (q.pieces == 0) return M < 64 ? M : 64;
    return norm_slices(M, G, q);
}

cudaError_t launch_norm_fwd(const NormParams &p, int dtype, cudaStream_t s) {
    return dtype == 0 ? norm_any<float>(p, false, s) : norm_any<__nv_bfloat16>(p, false, s);
}

cudaError_t launch_norm_bwd(const NormParams &p, int dtype, cudaStream_t s) {
    cudaError_t e = dtype == 0 ? norm_any<float>(p, true, s) : norm_any<__nv_bfloat16>(p, true, s);
    if (e != cudaSuccess || (p.dw == nullptr && p.db == nullptr)) return e;
    timing_mark("norm_reduce", 0, s);
    norm_reduce_kernel<<<(unsigned)(((size_t)2 * p.G * p.D + 31) / 32), 256, 0, s>>>(p);
    timing_mark("norm_reduce", 1, s);
    return cudaGetLastError();
}

}  // namespace gdn

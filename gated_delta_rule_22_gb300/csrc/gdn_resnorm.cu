// gdn_resnorm.cu -- the residual stream between two blocks: the norm of a block's output, its gate and
// residual scale, the addition, and the norm in front of the next block, in one pass; and the VJP.
//
//     n = h rstd_h w_post,  r = x + scale act(z) n,  y = r rstd_r w_pre        (root mean square norms)
// Backward, with u = scale act(z), hh = h rstd_h, rh = r rstd_r:
//     e = dy w_pre,   gr = dr + rstd_r (e - rh mean(e rh))                     (the gradient of r: dx)
//     f = gr u w_post,  dh = rstd_h (f - hh mean(f hh))
//     dz = gr scale n act'(z),  dscale = sum gr act(z) n,  dw_post = sum gr u hh,  dw_pre = sum dy rh
#include "gdn_layer.cuh"

#include <type_traits>

namespace gdn {

namespace {

__device__ __forceinline__ float act_rt(int act, float x) {
    return act == kActSilu ? silu_hw(x) : act == kActGelu ? gelu_f(x) : x;
}
__device__ __forceinline__ float dact_rt(int act, float x) {
    return act == kActSilu ? dsilu_hw(x) : act == kActGelu ? dgelu_f(x) : 1.f;
}

// Sum over the LPR lanes of a row: a part of a warp, or a CTA of LPR threads (through shared memory, two
// buffers in turn so that one barrier per sum is enough).
template <int LPR>
struct RowSum {
    int turn = 0;
    __device__ __forceinline__ float operator()(float x) {
#pragma unroll
        for (int m = (LPR < 32 ? LPR : 32) / 2; m >= 1; m >>= 1) x += __shfl_xor_sync(kFullMask, x, m);
        if constexpr (LPR > 32) {
            __shared__ float buf[2][LPR / 32];
            if ((threadIdx.x & 31) == 0) buf[turn][threadIdx.x >> 5] = x;
            __syncthreads();
            x = buf[turn][0];
#pragma unroll
            for (int w = 1; w < LPR / 32; ++w) x += buf[turn][w];
            turn ^= 1;
        }
        return x;
    }
};

// A row by LPR lanes, lane j holding channels (i LPR + j) V .. + V - 1 for i < IT (D <= LPR V IT); CTAs of
// at least 128 threads.
template <typename T, int V, int LPR, int IT>
struct RowLane {
    static constexpr int kThreads = LPR < 128 ? 128 : LPR, kRows = kThreads / LPR, E = V * IT;
    int j, slot, D;
    __device__ __forceinline__ explicit RowLane(int D_) : j(threadIdx.x % LPR), slot(threadIdx.x / LPR), D(D_) {}
    __device__ __forceinline__ int col(int i) const { return (i * LPR + j) * V; }
    __device__ __forceinline__ bool ok(int i) const { return col(i) < D; }
    __device__ __forceinline__ void load(const void *t, size_t at, Raw<T, V> (&o)[IT]) const {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            o[i] = Raw<T, V>();
            if (ok(i)) o[i] = load_raw<T, V>(static_cast<const T *>(t) + at + col(i));
        }
    }
    __device__ __forceinline__ void floats(const Raw<T, V> (&r)[IT], float (&o)[E]) const {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            float e[V];
            unpack<T, V>(r[i], e);
#pragma unroll
            for (int v = 0; v < V; ++v) o[i * V + v] = e[v];
        }
    }
    __device__ __forceinline__ void store(void *t, size_t at, const float (&x)[E]) const {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            float e[V];
#pragma unroll
            for (int v = 0; v < V; ++v) e[v] = x[i * V + v];
            if (ok(i)) store_vec<T, V>(static_cast<T *>(t) + at + col(i), e);
        }
    }
    // parameters of the lane's channels, 1 where there are none
    __device__ __forceinline__ void params(const float *w, float (&o)[E]) const {
#pragma unroll
        for (int i = 0; i < IT; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) o[i * V + v] = w != nullptr && ok(i) ? w[col(i) + v] : 1.f;
    }
    __device__ __forceinline__ void put(float *t, const float (&x)[E]) const {
#pragma unroll
        for (int i = 0; i < IT; ++i)
            if (ok(i))
#pragma unroll
                for (int v = 0; v < V; ++v) t[col(i) + v] = x[i * V + v];
    }
};

constexpr int kUnitTarget = 1216;   // CTAs of a backward: 152 SMs, up to 8 each

}  // namespace

template <typename T, int V, int LPR, int IT>
__global__ void __launch_bounds__(LPR < 128 ? 128 : LPR) resnorm_fwd_kernel(const ResnormParams p) {
    using Lane = RowLane<T, V, LPR, IT>;
    constexpr int E = Lane::E;
    const Lane at(p.D);
    RowSum<LPR> row_sum;
    const int rows = gridDim.x * Lane::kRows;
    int m = blockIdx.x * Lane::kRows + at.slot;
    const float inv_D = 1.f / p.D;
    Raw<T, V> rx[IT], rh[IT], rz[IT];
    auto fetch = [&](int row) {
        at.load(p.x, (size_t)row * p.ldx, rx);
        at.load(p.h, (size_t)row * p.ldh, rh);
        if (p.z != nullptr) at.load(p.z, (size_t)(row / p.gate_rows) * p.ldz, rz);
    };
    // (all lanes of a warp walk together: a row behind the last is computed from zeros and not stored)
    if (m < p.M) fetch(m);
    else
#pragma unroll
        for (int i = 0; i < IT; ++i) rx[i] = rh[i] = rz[i] = Raw<T, V>();
    float sc[E], wo[E], wr[E];
    at.params(p.scale, sc);
    at.params(p.w_post, wo);
    at.params(p.w_pre, wr);
    for (; m - at.slot < p.M; m += rows) {
        const bool live = m < p.M;
        float x[E], h[E];
        at.floats(rx, x);
        at.floats(rh, h);
        float z[E];
        if (p.z != nullptr) at.floats(rz, z);
        if (m + rows < p.M) fetch(m + rows);
        float rs = 1.f;
        if (p.post) {
            float q = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) q = fmaf(h[e], h[e], q);
            rs = 1.f / sqrtf(fmaf(row_sum(q), inv_D, p.eps));
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float u = p.z != nullptr ? sc[e] * act_rt(p.act, z[e]) : sc[e];
            x[e] = fmaf(u, p.post ? h[e] * rs * wo[e] : h[e], x[e]);
        }
        if (live) at.store(p.r, (size_t)m * p.D, x);
        float rr = 1.f;
        if (p.pre) {
            float q = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) q = fmaf(x[e], x[e], q);
            rr = 1.f / sqrtf(fmaf(row_sum(q), inv_D, p.eps));
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = x[e] * rr * wr[e];
            if (live) at.store(p.y, (size_t)m * p.D, x);
        }
        if (live && p.stats != nullptr && at.j == 0) *reinterpret_cast<float2 *>(p.stats + 2 * (size_t)m) = make_float2(rs, rr);
    }
}

// A CTA takes units of p.unit consecutive rows that share a row of z (gate_rows = 1: any rows), sums the
// parameter gradients over all its units into its slice of the partial sums, and the gate's over each.
template <typename T, int V, int LPR, int IT>
__global__ void __launch_bounds__(LPR < 128 ? 128 : LPR) resnorm_bwd_kernel(const ResnormParams p) {
    using Lane = RowLane<T, V, LPR, IT>;
    constexpr int E = Lane::E, ROWS = Lane::kRows;
    const Lane at(p.D);
    RowSum<LPR> row_sum;
    const float inv_D = 1.f / p.D;
    const bool shared_z = p.z != nullptr && p.gate_rows > 1;
    float sc[E], wo[E], wr[E], dsc[E], dwo[E], dwr[E], dzs[E];
    at.params(p.scale, sc);
    at.params(p.w_post, wo);
    at.params(p.w_pre, wr);
#pragma unroll
    for (int e = 0; e < E; ++e) dsc[e] = dwo[e] = dwr[e] = 0.f;
    // the slots' sums of a CTA, in ascending order
    auto over_slots = [&](float (&x)[E]) {
        if constexpr (ROWS > 1) {
            __shared__ float buf[ROWS][LPR * E];
            __syncthreads();
#pragma unroll
            for (int e = 0; e < E; ++e) buf[at.slot][e * LPR + at.j] = x[e];
            __syncthreads();
            if (at.slot == 0)
                for (int s = 1; s < ROWS; ++s)
#pragma unroll
                    for (int e = 0; e < E; ++e) x[e] += buf[s][e * LPR + at.j];
        }
    };
    for (int unit = blockIdx.x; unit < p.units; unit += p.ctas) {
        const int gate = unit / p.per_gate, span = shared_z ? p.gate_rows : p.M;
        const int first = gate * span + unit % p.per_gate * p.unit;
        const int last = min(first + p.unit, min((gate + 1) * span, p.M));
#pragma unroll
        for (int e = 0; e < E; ++e) dzs[e] = 0.f;
        for (int m0 = first; m0 < last; m0 += ROWS) {
            const int m = m0 + at.slot;
            const bool live = m < last;
            const int row = live ? m : first;
            Raw<T, V> rx[IT], rh[IT], rz[IT], ry[IT], rr[IT];
            at.load(p.x, (size_t)row * p.ldx, rx);
            at.load(p.h, (size_t)row * p.ldh, rh);
            if (p.z != nullptr) at.load(p.z, (size_t)(row / p.gate_rows) * p.ldz, rz);
            if (p.pre) at.load(p.dy, (size_t)row * p.D, ry);
            if (p.dr != nullptr) at.load(p.dr, (size_t)row * p.D, rr);
            const float2 st = *reinterpret_cast<const float2 *>(p.stats_in + 2 * (size_t)row);
            float x[E], h[E], z[E], u[E], g[E];
            at.floats(rx, x);
            at.floats(rh, h);
            if (p.z != nullptr) at.floats(rz, z);
            if (p.dr != nullptr) at.floats(rr, g);
            else
#pragma unroll
                for (int e = 0; e < E; ++e) g[e] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                h[e] *= st.x;                                              // hh
                u[e] = p.z != nullptr ? act_rt(p.act, z[e]) : 1.f;
                x[e] = fmaf(sc[e] * u[e], h[e] * wo[e], x[e]) * st.y;       // rh
            }
            if (p.pre) {
                float dy[E], q = 0.f;
                at.floats(ry, dy);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    if (live) dwr[e] = fmaf(dy[e], x[e], dwr[e]);
                    dy[e] *= wr[e];
                    q = fmaf(dy[e], x[e], q);
                }
                q = row_sum(q) * inv_D;
#pragma unroll
                for (int e = 0; e < E; ++e) g[e] = fmaf(st.y, fmaf(-x[e], q, dy[e]), g[e]);
            }
            if (live) at.store(p.dx, (size_t)m * p.D, g);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float n = h[e] * wo[e], gn = g[e] * n;
                if (p.z != nullptr) {
                    if (shared_z) dzs[e] = live ? fmaf(gn, sc[e], dzs[e]) : dzs[e];
                    else x[e] = gn * sc[e] * dact_rt(p.act, z[e]);
                }
                if (live) {
                    dsc[e] = fmaf(gn, u[e], dsc[e]);
                    dwo[e] = fmaf(g[e] * sc[e] * u[e], h[e], dwo[e]);
                }
                g[e] *= sc[e] * u[e] * wo[e];                               // f
            }
            if (live && p.dz != nullptr && !shared_z) at.store(p.dz, (size_t)m * p.D, x);
            if (p.post) {
                float q = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) q = fmaf(g[e], h[e], q);
                q = row_sum(q) * inv_D;
#pragma unroll
                for (int e = 0; e < E; ++e) g[e] = st.x * fmaf(-h[e], q, g[e]);
            }
            if (live) at.store(p.dh, (size_t)m * p.D, g);
        }
        if (shared_z && p.dz != nullptr) {
            over_slots(dzs);
            if (at.slot == 0) at.put(p.part_z + (size_t)unit * p.D, dzs);
        }
    }
    over_slots(dsc);
    over_slots(dwo);
    over_slots(dwr);
    if (at.slot == 0) {
        float *part = p.part + (size_t)blockIdx.x * 3 * p.D;
        at.put(part, dsc);
        at.put(part + p.D, dwo);
        at.put(part + 2 * (size_t)p.D, dwr);
    }
}

// The parameter gradients: sums over the CTAs' slices.
__global__ void __launch_bounds__(256) resnorm_sum_kernel(const ResnormParams p) {
    const size_t n = 3 * (size_t)p.D;
    const float s = slice_sum(p.part, p.ctas, n, blockIdx.x);
    const size_t i = (size_t)blockIdx.x * 32 + threadIdx.x;
    if (threadIdx.x >= 32 || i >= n) return;
    float *out = i < p.D ? p.dscale : i < 2 * (size_t)p.D ? p.dw_post : p.dw_pre;
    if (out != nullptr) out[i % p.D] = s;
}

// dz of a gate whose rows are shared: the units' sums, times act'(z).
template <typename T>
__global__ void __launch_bounds__(256) resnorm_gate_kernel(const ResnormParams p) {
    const int gate = blockIdx.y;
    const float s = slice_sum(p.part_z + (size_t)gate * p.per_gate * p.D, p.per_gate, p.D, blockIdx.x);
    const int d = blockIdx.x * 32 + threadIdx.x;
    if (threadIdx.x >= 32 || d >= p.D) return;
    const float z = to_f32(static_cast<const T *>(p.z)[(size_t)gate * p.ldz + d]);
    static_cast<T *>(p.dz)[(size_t)gate * p.D + d] = from_f32<T>(s * dact_rt(p.act, z));
}

void resnorm_units(ResnormParams *p, int) {
    const bool shared_z = p->gate_rows > 1;
    const int gates = shared_z ? p->M / p->gate_rows : 1, span = shared_z ? p->gate_rows : p->M;
    const int want = gates >= kUnitTarget ? 1 : (kUnitTarget + gates - 1) / gates;
    p->unit = (span + want - 1) / want;
    p->per_gate = (span + p->unit - 1) / p->unit;
    p->units = gates * p->per_gate;
    p->ctas = p->units < kUnitTarget ? p->units : kUnitTarget;
}

// f(kernel parameters as types): the form for D channels of a type at a vector width
template <typename T, typename F>
static cudaError_t with_row(int D, bool vec, F f) {
    constexpr int V = 16 / (int)sizeof(T);
#define GDN_ROW(V_, LPR_, IT_) return f(std::integral_constant<int, V_>(), std::integral_constant<int, LPR_>(), std::integral_constant<int, IT_>())
    if (vec) {
        if (D <= 8 * V) GDN_ROW(V, 8, 1);
        if (D <= 32 * V) GDN_ROW(V, 32, 1);
        if (D <= 128 * V) GDN_ROW(V, 128, 1);
        if (D <= 256 * V) GDN_ROW(V, 256, 1);
        if (D <= 512 * V) GDN_ROW(V, 512, 1);
        if (D <= 1024 * V) GDN_ROW(V, 1024, 1);
        GDN_ROW(V, 1024, 16384 / (1024 * V));
    }
    if (D <= 256) GDN_ROW(1, 32, 8);
    if (D <= 1024) GDN_ROW(1, 128, 8);
    if (D <= 4096) GDN_ROW(1, 512, 8);
    GDN_ROW(1, 1024, 16);
#undef GDN_ROW
}

static bool whole(const void *p, int bytes) { return p == nullptr || ((uintptr_t)p & (bytes - 1)) == 0; }

// 16-byte pieces of every row: D and the row strides multiples of a piece, the addresses aligned to it
template <typename T>
static bool rows_vec(const ResnormParams &p) {
    constexpr int V = 16 / (int)sizeof(T);
    return p.D % V == 0 && p.ldx % V == 0 && p.ldh % V == 0 && (p.z == nullptr || p.ldz % V == 0) && whole(p.x, 16) && whole(p.h, 16) &&
           whole(p.z, 16);
}

template <typename T>
static cudaError_t launch_fwd_t(const ResnormParams &p, cudaStream_t s) {
    return with_row<T>(p.D, rows_vec<T>(p), [&](auto v, auto lpr, auto it) {
        using Lane = RowLane<T, decltype(v)::value, decltype(lpr)::value, decltype(it)::value>;
        const int ctas = (p.M + Lane::kRows - 1) / Lane::kRows, most = 152 * (2048 / Lane::kThreads);
        resnorm_fwd_kernel<T, decltype(v)::value, decltype(lpr)::value, decltype(it)::value>
            <<<ctas < most ? ctas : most, Lane::kThreads, 0, s>>>(p);
        return cudaGetLastError();
    });
}

template <typename T>
static cudaError_t launch_bwd_t(const ResnormParams &p, cudaStream_t s) {
    timing_mark("resnorm_bwd", 0, s);
    cudaError_t e = with_row<T>(p.D, rows_vec<T>(p), [&](auto v, auto lpr, auto it) {
        using Lane = RowLane<T, decltype(v)::value, decltype(lpr)::value, decltype(it)::value>;
        resnorm_bwd_kernel<T, decltype(v)::value, decltype(lpr)::value, decltype(it)::value><<<p.ctas, Lane::kThreads, 0, s>>>(p);
        return cudaGetLastError();
    });
    timing_mark("resnorm_bwd", 1, s);
    if (e != cudaSuccess) return e;
    timing_mark("resnorm_sum", 0, s);
    if (p.dscale != nullptr || p.dw_post != nullptr || p.dw_pre != nullptr) resnorm_sum_kernel<<<(3 * p.D + 31) / 32, 256, 0, s>>>(p);
    if (p.dz != nullptr && p.gate_rows > 1) {
        // (the rows of z on the grid's second axis, at most 65535 of them at a time)
        const int gates = p.M / p.gate_rows;
        for (int g0 = 0; g0 < gates; g0 += 65535) {
            ResnormParams q = p;
            q.part_z += (size_t)g0 * p.per_gate * p.D;
            q.z = static_cast<const T *>(p.z) + (size_t)g0 * p.ldz;
            q.dz = static_cast<T *>(p.dz) + (size_t)g0 * p.D;
            resnorm_gate_kernel<T><<<dim3((p.D + 31) / 32, gates - g0 < 65535 ? gates - g0 : 65535), 256, 0, s>>>(q);
        }
    }
    timing_mark("resnorm_sum", 1, s);
    return cudaGetLastError();
}

cudaError_t launch_resnorm_fwd(const ResnormParams &p, int dtype, cudaStream_t s) {
    timing_mark("resnorm_fwd", 0, s);
    const cudaError_t e = dtype == 0 ? launch_fwd_t<float>(p, s) : launch_fwd_t<__nv_bfloat16>(p, s);
    timing_mark("resnorm_fwd", 1, s);
    return e;
}

cudaError_t launch_resnorm_bwd(const ResnormParams &p, int dtype, cudaStream_t s) {
    return dtype == 0 ? launch_bwd_t<float>(p, s) : launch_bwd_t<__nv_bfloat16>(p, s);
}

}  // namespace gdn

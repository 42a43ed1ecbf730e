// gdn_resnorm.cu -- the residual stream between two blocks: the norm of a block's output, its gate and
// residual scale, the addition, and the norm in front of the next block, in one pass; and the VJP.
//
//     n = h rstd_h w_post,  r = x + scale act(z) n,  y = r rstd_r w_pre        (root mean square norms)
// With hh = h rstd_h, rh = r rstd_r, k = scale w_post and u = act(z), so that r = x + k u hh:
//     e = dy w_pre,  q = mean(e rh),  gr = dr + rstd_r (e - rh q)              (the gradient of r: dx)
//     f = gr k u,    dh = rstd_h (f - hh mean(f hh)),  dz = gr k hh act'(z)
//     Q = sum_m gr u hh:  dscale = w_post Q,  dw_post = scale Q;   dw_pre = sum_m dy rh
// mean(f hh) = mean((dr + rstd_r e) k u hh) - rstd_r q mean(rh k u hh), so that a row's three sums are formed
// together and its threads meet once.
//
// Bound by memory: every tensor is read once and every output written once. What a thread reads of a row
// it copies into shared memory itself, asynchronously and some rows ahead (a ring of its own, so that
// nobody waits for anybody but for the row's sums).
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

// N sums over the LPR lanes of a row: a part of a warp, or a CTA of LPR threads (through shared memory, two
// buffers in turn so that one barrier is enough).
template <int LPR, int N>
struct RowSum {
    int turn = 0;
    __device__ __forceinline__ void operator()(float (&x)[N]) {
#pragma unroll
        for (int m = (LPR < 32 ? LPR : 32) / 2; m >= 1; m >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] += __shfl_xor_sync(kFullMask, x[i], m);
        if constexpr (LPR > 32) {
            __shared__ float buf[2][N][LPR / 32];
            if ((threadIdx.x & 31) == 0)
#pragma unroll
                for (int i = 0; i < N; ++i) buf[turn][i][threadIdx.x >> 5] = x[i];
            __syncthreads();
#pragma unroll
            for (int i = 0; i < N; ++i) {
                x[i] = buf[turn][i][0];
#pragma unroll
                for (int w = 1; w < LPR / 32; ++w) x[i] += buf[turn][i][w];
            }
            turn ^= 1;
        }
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
    __device__ __forceinline__ void read(const T *t, float (&o)[E]) const {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            float e[V];
            unpack<T, V>(ok(i) ? load_raw<T, V>(t + col(i)) : Raw<T, V>(), e);
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
    // the product of two parameters of the lane's channels, 1 where there are none
    __device__ __forceinline__ void params(const float *a, const float *b, float (&o)[E]) const {
#pragma unroll
        for (int i = 0; i < IT; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v)
                o[i * V + v] = (a != nullptr && ok(i) ? a[col(i) + v] : 1.f) * (b != nullptr && ok(i) ? b[col(i) + v] : 1.f);
    }
    __device__ __forceinline__ void put(float *t, const float (&x)[E]) const {
#pragma unroll
        for (int i = 0; i < IT; ++i)
            if (ok(i))
#pragma unroll
                for (int v = 0; v < V; ++v) t[col(i) + v] = x[i * V + v];
    }
};

// What a thread reads of the next rows, on its way through shared memory: kAhead rows of N tensors, 16 bytes for
// each piece. Rows that are not in pieces of 16 bytes are loaded when they are used.
template <typename Lane, typename T, int V, int IT, int N>
struct RowRing {
    static constexpr bool kRing = V * (int)sizeof(T) == 16 && (size_t)Lane::kThreads * N * IT * 16 * 2 <= 200 * 1024;
    static constexpr size_t kSlot = (size_t)Lane::kThreads * N * IT * 16;     // bytes of a row of the CTA
    static constexpr int kAhead = !kRing ? 1 : kSlot * 4 <= 88 * 1024 ? 4 : kSlot * 3 <= 100 * 1024 ? 3 : 2;
    static constexpr size_t kBytes = kRing ? kSlot * kAhead : 0;
    unsigned char *base;
    int put = 0, take = 0;
    __device__ __forceinline__ explicit RowRing(unsigned char *smem) : base(smem + threadIdx.x * 16) {}
    __device__ __forceinline__ unsigned char *at(int slot, int t, int i) const {
        return base + ((size_t)(slot * N + t) * IT + i) * Lane::kThreads * 16;
    }
    // starts the copies of a row: its N addresses, null where a tensor is not there (row behind the last: all null)
    __device__ __forceinline__ void fetch(const Lane &lane, const T *const (&src)[N]) {
        if constexpr (kRing) {
#pragma unroll
            for (int t = 0; t < N; ++t)
                if (src[t] != nullptr)
#pragma unroll
                    for (int i = 0; i < IT; ++i)
                        if (lane.ok(i)) cp_async16(at(put, t, i), src[t] + lane.col(i), 16);
            cp_async_commit();
            put = put + 1 == kAhead ? 0 : put + 1;
        }
    }
    __device__ __forceinline__ void arrive() const {
        if constexpr (kRing) cp_async_wait<kAhead - 1>();
    }
    // tensor t of the row that arrived, as floats (zeros behind the row's end)
    __device__ __forceinline__ void read(const Lane &lane, int t, const T *src, float (&o)[Lane::E]) const {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            float e[V];
            Raw<T, V> raw = Raw<T, V>();
            if (lane.ok(i)) {
                if constexpr (kRing) raw = *reinterpret_cast<const Raw<T, V> *>(at(take, t, i));
                else if (src != nullptr) raw = load_raw<T, V>(src + lane.col(i));
            }
            unpack<T, V>(raw, e);
#pragma unroll
            for (int v = 0; v < V; ++v) o[i * V + v] = e[v];
        }
    }
    // after a run of rows: nothing under way, the next row fetched is the next one read
    __device__ __forceinline__ void restart() {
        if constexpr (kRing) cp_async_wait<0>();
        take = put;
    }
    __device__ __forceinline__ void done() { take = take + 1 == kAhead ? 0 : take + 1; }
};

}  // namespace

template <typename T, int V, int LPR, int IT>
__global__ void __launch_bounds__(LPR < 128 ? 128 : LPR) resnorm_fwd_kernel(const ResnormParams p) {
    using Lane = RowLane<T, V, LPR, IT>;
    using Ring = RowRing<Lane, T, V, IT, 3>;
    extern __shared__ __align__(16) unsigned char smem[];
    constexpr int E = Lane::E;
    const Lane at(p.D);
    Ring ring(smem);
    RowSum<LPR, 1> row_sum;
    const int rows = gridDim.x * Lane::kRows;
    const float inv_D = 1.f / p.D;
    const T *src[3];
    auto locate = [&](int row) {
        const bool in = row < p.M;
        src[0] = in ? static_cast<const T *>(p.x) + (size_t)row * p.ldx : nullptr;
        src[1] = in ? static_cast<const T *>(p.h) + (size_t)row * p.ldh : nullptr;
        src[2] = in && p.z != nullptr ? static_cast<const T *>(p.z) + (size_t)(row / p.gate_rows) * p.ldz : nullptr;
    };
    int m = blockIdx.x * Lane::kRows + at.slot;
    for (int i = 0; i < Ring::kAhead - 1; ++i) {
        locate(m + i * rows);
        ring.fetch(at, src);
    }
    float k[E], wr[E];
    at.params(p.scale, p.w_post, k);
    at.params(p.w_pre, nullptr, wr);
    // (all lanes of a warp walk together: a row behind the last is computed from zeros and not stored)
    for (; m - at.slot < p.M; m += rows) {
        const bool live = m < p.M;
        locate(m + (Ring::kAhead - 1) * rows);
        ring.fetch(at, src);
        ring.arrive();
        locate(m);
        float x[E], h[E];
        ring.read(at, 0, src[0], x);
        ring.read(at, 1, src[1], h);
        float rs = 1.f;
        if (p.post) {
            float q[1] = {0.f};
#pragma unroll
            for (int e = 0; e < E; ++e) q[0] = fmaf(h[e], h[e], q[0]);
            row_sum(q);
            rs = 1.f / sqrtf(fmaf(q[0], inv_D, p.eps));
        }
        if (p.z != nullptr) {
            float z[E];
            ring.read(at, 2, src[2], z);
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = fmaf(k[e] * act_rt(p.act, z[e]), h[e] * rs, x[e]);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = fmaf(k[e], h[e] * rs, x[e]);
        }
        ring.done();
        if (live) at.store(p.r, (size_t)m * p.D, x);
        float rr = 1.f;
        if (p.pre) {
            float q[1] = {0.f};
#pragma unroll
            for (int e = 0; e < E; ++e) q[0] = fmaf(x[e], x[e], q[0]);
            row_sum(q);
            rr = 1.f / sqrtf(fmaf(q[0], inv_D, p.eps));
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = x[e] * rr * wr[e];
            if (live) at.store(p.y, (size_t)m * p.D, x);
        }
        if (live && p.stats != nullptr && at.j == 0) *reinterpret_cast<float2 *>(p.stats + 2 * (size_t)m) = make_float2(rs, rr);
    }
}

// A CTA takes units of p.unit consecutive rows that share a row of z (gate_rows = 1: any rows), sums Q and dw_pre
// over all its units into its slice of the partial sums, and the gate's gradient over each.
template <typename T, int V, int LPR, int IT>
__global__ void __launch_bounds__(LPR < 128 ? 128 : LPR) resnorm_bwd_kernel(const ResnormParams p) {
    using Lane = RowLane<T, V, LPR, IT>;
    using Ring = RowRing<Lane, T, V, IT, 5>;
    extern __shared__ __align__(16) unsigned char smem[];
    constexpr int E = Lane::E, ROWS = Lane::kRows;
    const Lane at(p.D);
    Ring ring(smem);
    RowSum<LPR, 3> row_sum;
    const float inv_D = 1.f / p.D;
    const bool shared_z = p.z != nullptr && p.gate_rows > 1;
    float k[E], wr[E], Q[E], dwr[E], dzs[E];
    at.params(p.scale, p.w_post, k);
    at.params(p.w_pre, nullptr, wr);
#pragma unroll
    for (int e = 0; e < E; ++e) Q[e] = dwr[e] = 0.f;
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
    const T *src[5];
    auto locate = [&](int row, bool in) {
        src[0] = in ? static_cast<const T *>(p.x) + (size_t)row * p.ldx : nullptr;
        src[1] = in ? static_cast<const T *>(p.h) + (size_t)row * p.ldh : nullptr;
        src[2] = in && p.pre ? static_cast<const T *>(p.dy) + (size_t)row * p.D : nullptr;
        src[3] = in && p.dr != nullptr ? static_cast<const T *>(p.dr) + (size_t)row * p.D : nullptr;
        src[4] = in && p.z != nullptr ? static_cast<const T *>(p.z) + (size_t)(row / p.gate_rows) * p.ldz : nullptr;
    };
    for (int unit = blockIdx.x; unit < p.units; unit += p.ctas) {
        const int gate = unit / p.per_gate, span = shared_z ? p.gate_rows : p.M;
        const int first = gate * span + unit % p.per_gate * p.unit;
        const int last = min(first + p.unit, min((gate + 1) * span, p.M));
#pragma unroll
        for (int e = 0; e < E; ++e) dzs[e] = 0.f;
        for (int i = 0; i < Ring::kAhead - 1; ++i) {
            const int m = first + i * ROWS + at.slot;
            locate(m, m < last);
            ring.fetch(at, src);
        }
        for (int m0 = first; m0 < last; m0 += ROWS) {
            const int m = m0 + at.slot, ahead = m + (Ring::kAhead - 1) * ROWS;
            const bool live = m < last;
            locate(ahead, ahead < last);
            ring.fetch(at, src);
            const float2 st = live ? *reinterpret_cast<const float2 *>(p.stats_in + 2 * (size_t)m) : make_float2(0.f, 0.f);
            ring.arrive();
            locate(m, live);
            // rh, hh, dr + rstd_r e, u; and the row's sums (a row behind the last adds nothing: its hh and rh are zeros)
            float rh[E], hh[E], g[E], u[E], q[3] = {0.f, 0.f, 0.f};
            ring.read(at, 0, src[0], rh);
            ring.read(at, 1, src[1], hh);
            if (p.z != nullptr) {
                ring.read(at, 4, src[4], u);
#pragma unroll
                for (int e = 0; e < E; ++e) u[e] = act_rt(p.act, u[e]);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) u[e] = 1.f;
            }
#pragma unroll
            for (int e = 0; e < E; ++e) {
                hh[e] *= st.x;
                rh[e] = fmaf(k[e] * u[e], hh[e], rh[e]) * st.y;
            }
            if (!live)
#pragma unroll
                for (int e = 0; e < E; ++e) hh[e] = rh[e] = u[e] = 0.f;
            if (p.dr != nullptr) ring.read(at, 3, src[3], g);
            else
#pragma unroll
                for (int e = 0; e < E; ++e) g[e] = 0.f;
            if (p.pre) {
                float dy[E];
                ring.read(at, 2, src[2], dy);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    if (live) dwr[e] = fmaf(dy[e], rh[e], dwr[e]);
                    dy[e] *= wr[e];
                    q[0] = fmaf(dy[e], rh[e], q[0]);
                    g[e] = fmaf(st.y, dy[e], g[e]);
                }
            }
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float t = k[e] * u[e] * hh[e];
                q[1] = fmaf(g[e], t, q[1]);
                q[2] = fmaf(rh[e], t, q[2]);
            }
            ring.done();
            row_sum(q);
            const float c = p.pre ? st.y * q[0] * inv_D : 0.f, mean = p.post ? fmaf(-c, q[2], q[1]) * inv_D : 0.f;
            float f[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                g[e] = fmaf(-c, rh[e], g[e]);                                    // gr
                const float gu = g[e] * u[e];
                if (live) Q[e] = fmaf(gu, hh[e], Q[e]);
                f[e] = st.x * fmaf(-hh[e], mean, gu * k[e]);
            }
            if (live) {
                at.store(p.dx, (size_t)m * p.D, g);
                at.store(p.dh, (size_t)m * p.D, f);
            }
            if (p.dz != nullptr) {
                if (shared_z) {
#pragma unroll
                    for (int e = 0; e < E; ++e) dzs[e] = live ? fmaf(g[e] * k[e], hh[e], dzs[e]) : dzs[e];
                } else if (live) {
                    float z[E];
                    at.read(static_cast<const T *>(p.z) + (size_t)m * p.ldz, z);   // (again, from the cache)
#pragma unroll
                    for (int e = 0; e < E; ++e) z[e] = g[e] * k[e] * hh[e] * dact_rt(p.act, z[e]);
                    at.store(p.dz, (size_t)m * p.D, z);
                }
            }
        }
        ring.restart();
        if (shared_z && p.dz != nullptr) {
            over_slots(dzs);
            if (at.slot == 0) at.put(p.part_z + (size_t)unit * p.D, dzs);
        }
    }
    over_slots(Q);
    over_slots(dwr);
    if (at.slot == 0) {
        float *part = p.part + (size_t)blockIdx.x * 2 * p.D;
        at.put(part, Q);
        at.put(part + p.D, dwr);
    }
}

// The parameter gradients: sums over the CTAs' slices.
__global__ void __launch_bounds__(256) resnorm_sum_kernel(const ResnormParams p) {
    const size_t n = 2 * (size_t)p.D;
    const float s = slice_sum(p.part, p.ctas, n, blockIdx.x);
    const size_t i = (size_t)blockIdx.x * 32 + threadIdx.x;
    if (threadIdx.x >= 32 || i >= n) return;
    if (i >= p.D) {
        if (p.dw_pre != nullptr) p.dw_pre[i - p.D] = s;
        return;
    }
    if (p.dscale != nullptr) p.dscale[i] = p.w_post != nullptr ? s * p.w_post[i] : s;
    if (p.dw_post != nullptr) p.dw_post[i] = p.scale != nullptr ? s * p.scale[i] : s;
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

// CTAs of a backward: as many as stay on the SMs, so that each has rows enough to fetch ahead (two of 256 threads
// and more, four smaller ones)
void resnorm_units(ResnormParams *p, int dtype) {
    const int target = 152 * ((size_t)p->D * (dtype == 0 ? 4 : 2) > 2048 ? 2 : 4);
    const bool shared_z = p->gate_rows > 1;
    const int gates = shared_z ? p->M / p->gate_rows : 1, span = shared_z ? p->gate_rows : p->M;
    const int want = gates >= target ? 1 : (target + gates - 1) / gates;
    p->unit = (span + want - 1) / want;
    p->per_gate = (span + p->unit - 1) / p->unit;
    p->units = gates * p->per_gate;
    p->ctas = p->units < target ? p->units : target;
}

// f(kernel parameters as types): the form for D channels of a type, in 16-byte pieces or one by one
template <typename T, typename F>
static cudaError_t with_row(int D, bool vec, F f) {
    constexpr int V = 16 / (int)sizeof(T), W = 8 / V;      // W: pieces of eight channels
#define GDN_ROW(V_, LPR_, IT_) return f(std::integral_constant<int, V_>(), std::integral_constant<int, LPR_>(), std::integral_constant<int, IT_>())
    if (vec) {
        if (D <= 64) GDN_ROW(V, 8, W);
        if (D <= 256) GDN_ROW(V, 32, W);
        if (D <= 512) GDN_ROW(V, 32, 2 * W);
        if (D <= 1024) GDN_ROW(V, 128, W);
        if (D <= 2048) GDN_ROW(V, 256, W);
        if (D <= 4096) GDN_ROW(V, 512, W);
        if (D <= 8192) GDN_ROW(V, 512, 2 * W);
        GDN_ROW(V, 1024, 2 * W);
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
        constexpr int V = decltype(v)::value, LPR = decltype(lpr)::value, IT = decltype(it)::value;
        using Lane = RowLane<T, V, LPR, IT>;
        using Ring = RowRing<Lane, T, V, IT, 3>;
        const cudaError_t e = allow_smem<resnorm_fwd_kernel<T, V, LPR, IT>>((int)Ring::kBytes);
        if (e != cudaSuccess) return e;
        const int ctas = (p.M + Lane::kRows - 1) / Lane::kRows, most = 152 * (1024 / Lane::kThreads);
        resnorm_fwd_kernel<T, V, LPR, IT><<<ctas < most ? ctas : most, Lane::kThreads, Ring::kBytes, s>>>(p);
        return cudaGetLastError();
    });
}

template <typename T>
static cudaError_t launch_bwd_t(const ResnormParams &p, cudaStream_t s) {
    timing_mark("resnorm_bwd", 0, s);
    cudaError_t e = with_row<T>(p.D, rows_vec<T>(p), [&](auto v, auto lpr, auto it) {
        constexpr int V = decltype(v)::value, LPR = decltype(lpr)::value, IT = decltype(it)::value;
        using Lane = RowLane<T, V, LPR, IT>;
        using Ring = RowRing<Lane, T, V, IT, 5>;
        const cudaError_t err = allow_smem<resnorm_bwd_kernel<T, V, LPR, IT>>((int)Ring::kBytes);
        if (err != cudaSuccess) return err;
        resnorm_bwd_kernel<T, V, LPR, IT><<<p.ctas, Lane::kThreads, Ring::kBytes, s>>>(p);
        return cudaGetLastError();
    });
    timing_mark("resnorm_bwd", 1, s);
    if (e != cudaSuccess) return e;
    timing_mark("resnorm_sum", 0, s);
    if (p.dscale != nullptr || p.dw_post != nullptr || p.dw_pre != nullptr) resnorm_sum_kernel<<<(2 * p.D + 31) / 32, 256, 0, s>>>(p);
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

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
// nobody waits for anybody but for the row's sums). 32768 x 2048 in bf16: forward 94 to 101 us, 5.3 to 5.7 TB/s; backward 153 us,
// 5.3 TB/s, and 10 for the parameters' sums. 8192 x 4096 with a gate for each sequence, forward: 56 us, 4.75 TB/s. 8192 x 8192:
// forward 97 us, 5.5 TB/s, backward 264 and 12; 4096 x 16384: 107, and 542 and 15: the backward of more than 4096 channels
// spills.
#include "gdn_layer.cuh"

#include <type_traits>

namespace gdn {

namespace {

__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

template <int ACT>
__device__ __forceinline__ float2 act2(float2 x) {
    return ACT == kActSilu ? mul2(x, sigmoid2_hw(x)) : ACT == kActGelu ? make_float2(gelu_f(x.x), gelu_f(x.y)) : x;
}
__device__ __forceinline__ float dact_rt(int act, float x) {
    return act == kActSilu ? dsilu_hw(x) : act == kActGelu ? dgelu_f(x) : 1.f;
}
template <int ACT>
__device__ __forceinline__ float2 dact2(float2 x) { return make_float2(dact_rt(ACT, x.x), dact_rt(ACT, x.y)); }
// f<ACT>() for the activation of the call: the test is made once per row, not per element.
template <typename F>
__device__ __forceinline__ void with_act(int act, F f) {
    if (act == kActSilu) f(std::integral_constant<int, kActSilu>());
    else if (act == kActGelu) f(std::integral_constant<int, kActGelu>());
    else f(std::integral_constant<int, kActNone>());
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

// A row by LPR lanes, lane j holding channels (i LPR + j) V .. + V - 1 for i < IT (D <= LPR V IT), as E / 2
// pairs for the packed instructions; CTAs of at least 128 threads.
template <typename T, int V, int LPR, int IT>
struct RowLane {
    static constexpr int kThreads = LPR < 128 ? 128 : LPR, kRows = kThreads / LPR, E = V * IT, P = E / 2;
    int j, slot, D;
    __device__ __forceinline__ explicit RowLane(int D_) : j(threadIdx.x % LPR), slot(threadIdx.x / LPR), D(D_) {}
    __device__ __forceinline__ int col(int i) const { return (i * LPR + j) * V; }
    __device__ __forceinline__ bool ok(int i) const { return col(i) < D; }
    __device__ __forceinline__ static void set(float2 (&o)[P], int e, float x) {
        if (e % 2) o[e / 2].y = x;
        else o[e / 2].x = x;
    }
    __device__ __forceinline__ static float get(const float2 (&x)[P], int e) { return e % 2 ? x[e / 2].y : x[e / 2].x; }
    __device__ __forceinline__ static void place(const Raw<T, V> &raw, int i, float2 (&o)[P]) {
        float e[V];
        unpack<T, V>(raw, e);
#pragma unroll
        for (int v = 0; v < V; ++v) set(o, i * V + v, e[v]);
    }
    __device__ __forceinline__ void read(const T *t, float2 (&o)[P]) const {
#pragma unroll
        for (int i = 0; i < IT; ++i) place(ok(i) ? load_raw<T, V>(t + col(i)) : Raw<T, V>(), i, o);
    }
    __device__ __forceinline__ void store(T *t, const float2 (&x)[P]) const {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            float e[V];
#pragma unroll
            for (int v = 0; v < V; ++v) e[v] = get(x, i * V + v);
            if (ok(i)) store_vec<T, V>(t + col(i), e);
        }
    }
    // the product of two parameters of the lane's channels, 1 where there are none
    __device__ __forceinline__ void params(const float *a, const float *b, float2 (&o)[P]) const {
#pragma unroll
        for (int i = 0; i < IT; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v)
                set(o, i * V + v, (a != nullptr && ok(i) ? a[col(i) + v] : 1.f) * (b != nullptr && ok(i) ? b[col(i) + v] : 1.f));
    }
    __device__ __forceinline__ void put(float *t, const float2 (&x)[P]) const {
#pragma unroll
        for (int i = 0; i < IT; ++i)
            if (ok(i))
#pragma unroll
                for (int v = 0; v < V; ++v) t[col(i) + v] = get(x, i * V + v);
    }
};

template <int BYTES>
__device__ __forceinline__ void copy_async(void *dst, const void *src) {
    if constexpr (BYTES == 16) cp_async16(dst, src, 16);
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_addr(dst)), "l"(src), "n"(BYTES) : "memory");
}

// What a thread reads of the next rows, on its way through shared memory: kAhead rows of N tensors, in pieces of
// 16, 8 or 4 bytes. Rows whose pieces are smaller are loaded when they are used.
template <typename Lane, typename T, int V, int IT, int N>
struct RowRing {
    static constexpr int kPiece = V * (int)sizeof(T);
    static constexpr bool kRing = kPiece >= 4 && (size_t)Lane::kThreads * N * IT * kPiece * 2 <= 200 * 1024;
    static constexpr size_t kSlot = (size_t)Lane::kThreads * N * IT * kPiece;     // bytes of a row of the CTA
    static constexpr int kAhead = !kRing ? 1 : kSlot * 4 <= 88 * 1024 ? 4 : kSlot * 3 <= 100 * 1024 ? 3 : 2;
    static constexpr size_t kBytes = kRing ? kSlot * kAhead : 0;
    unsigned char *base;
    int put = 0, take = 0;
    __device__ __forceinline__ explicit RowRing(unsigned char *smem) : base(smem + threadIdx.x * kPiece) {}
    __device__ __forceinline__ unsigned char *at(int slot, int t, int i) const {
        return base + ((size_t)(slot * N + t) * IT + i) * Lane::kThreads * kPiece;
    }
    // starts the copies of a row (in: there is one), tensor t's from src[t], null where it is not there
    __device__ __forceinline__ void fetch(const Lane &lane, const T *const (&src)[N], bool in) {
        if constexpr (kRing) {
#pragma unroll
            for (int t = 0; t < N; ++t)
                if (in && src[t] != nullptr)
#pragma unroll
                    for (int i = 0; i < IT; ++i)
                        if (lane.ok(i)) copy_async<kPiece>(at(put, t, i), src[t] + lane.col(i));
            cp_async_commit();
            put = put + 1 == kAhead ? 0 : put + 1;
        }
    }
    __device__ __forceinline__ void arrive() const {
        if constexpr (kRing) cp_async_wait<kAhead - 1>();
    }
    // tensor t of the row that arrived, as floats (zeros behind the row's end); without a ring, from src
    __device__ __forceinline__ void read(const Lane &lane, int t, const T *src, bool in, float2 (&o)[Lane::P]) const {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            Raw<T, V> raw = Raw<T, V>();
            if (lane.ok(i)) {
                if constexpr (kRing) raw = *reinterpret_cast<const Raw<T, V> *>(at(take, t, i));
                else if (in) raw = load_raw<T, V>(src + lane.col(i));
            }
            Lane::place(raw, i, o);
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
    constexpr int P = Lane::P;
    const Lane at(p.D);
    Ring ring(smem);
    RowSum<LPR, 1> row_sum;
    const unsigned rows = gridDim.x * Lane::kRows, M = p.M;    // (row numbers run past the last by some rounds)
    const float inv_D = 1.f / p.D;
    unsigned m = blockIdx.x * Lane::kRows + at.slot;
    const T *const x0 = static_cast<const T *>(p.x), *const h0 = static_cast<const T *>(p.h), *const z0 = static_cast<const T *>(p.z);
    const T *src[3];
    auto locate = [&](unsigned row) {
        src[0] = x0 + (size_t)row * p.ldx;
        src[1] = h0 + (size_t)row * p.ldh;
        src[2] = z0 == nullptr ? nullptr : z0 + (size_t)(p.gate_rows == 1 ? row : row / p.gate_rows) * p.ldz;
    };
    unsigned next = m;                                     // the next row to be fetched
    for (int i = 0; i < Ring::kAhead - 1; ++i, next += rows) {
        locate(next);
        ring.fetch(at, src, next < M);
    }
    float2 k[P], wr[P];
    at.params(p.scale, p.w_post, k);
    at.params(p.w_pre, nullptr, wr);
    // (all lanes of a warp walk together: a row behind the last is computed from anything and not stored)
    for (; m - at.slot < M; m += rows, next += rows) {
        const bool live = m < M;
        locate(next);
        ring.fetch(at, src, next < M);
        ring.arrive();
        if (!Ring::kRing) locate(m);
        float2 x[P], h[P];
        ring.read(at, 0, src[0], live, x);
        ring.read(at, 1, src[1], live, h);
        float rs = 1.f;
        if (p.post) {
            float2 s = both(0.f);
#pragma unroll
            for (int e = 0; e < P; ++e) s = fma2(h[e], h[e], s);
            float q[1] = {s.x + s.y};
            row_sum(q);
            rs = 1.f / sqrtf(fmaf(q[0], inv_D, p.eps));
        }
#pragma unroll
        for (int e = 0; e < P; ++e) h[e] = mul2(h[e], both(rs));
        if (z0 != nullptr) {
            float2 z[P];
            ring.read(at, 2, src[2], live, z);
            with_act(p.act, [&](auto act) {
#pragma unroll
                for (int e = 0; e < P; ++e) h[e] = mul2(h[e], act2<decltype(act)::value>(z[e]));
            });
        }
#pragma unroll
        for (int e = 0; e < P; ++e) x[e] = fma2(k[e], h[e], x[e]);
        ring.done();
        if (live) at.store(static_cast<T *>(p.r) + (size_t)m * p.D, x);
        float rr = 1.f;
        if (p.pre) {
            float2 s = both(0.f);
#pragma unroll
            for (int e = 0; e < P; ++e) s = fma2(x[e], x[e], s);
            float q[1] = {s.x + s.y};
            row_sum(q);
            rr = 1.f / sqrtf(fmaf(q[0], inv_D, p.eps));
#pragma unroll
            for (int e = 0; e < P; ++e) x[e] = mul2(mul2(x[e], both(rr)), wr[e]);
            if (live) at.store(static_cast<T *>(p.y) + (size_t)m * p.D, x);
        }
        if (live && p.stats != nullptr && at.j == 0) *reinterpret_cast<float2 *>(p.stats + 2 * (size_t)m) = make_float2(rs, rr);
    }
}

// A CTA takes units of p.unit consecutive rows that share a row of z (gate_rows = 1, as it is without z: any rows), sums Q and dw_pre
// over all its units into its slice of the partial sums, and the gate's gradient over each.
template <typename T, int V, int LPR, int IT>
__global__ void __launch_bounds__(LPR < 128 ? 128 : LPR, LPR <= 256 ? 2 : 1) resnorm_bwd_kernel(const ResnormParams p) {
    using Lane = RowLane<T, V, LPR, IT>;
    using Ring = RowRing<Lane, T, V, IT, 5>;
    extern __shared__ __align__(16) unsigned char smem[];
    constexpr int P = Lane::P, ROWS = Lane::kRows;
    const Lane at(p.D);
    Ring ring(smem);
    RowSum<LPR, 3> row_sum;
    const float inv_D = 1.f / p.D;
    const T *const z0 = static_cast<const T *>(p.z);
    const bool shared_z = p.gate_rows > 1;
    float2 k[P], wr[P], Q[P], dwr[P], dzs[P];
    at.params(p.scale, p.w_post, k);
    at.params(p.w_pre, nullptr, wr);
#pragma unroll
    for (int e = 0; e < P; ++e) Q[e] = dwr[e] = both(0.f);
    // the slots' sums of a CTA, in ascending order
    auto over_slots = [&](float2 (&x)[P]) {
        if constexpr (ROWS > 1) {
            __shared__ float2 buf[ROWS][LPR * P];
            __syncthreads();
#pragma unroll
            for (int e = 0; e < P; ++e) buf[at.slot][e * LPR + at.j] = x[e];
            __syncthreads();
            if (at.slot == 0)
                for (int s = 1; s < ROWS; ++s)
#pragma unroll
                    for (int e = 0; e < P; ++e) x[e] = __fadd2_rn(x[e], buf[s][e * LPR + at.j]);
        }
    };
    const T *src[5];
    auto locate = [&](int row) {
        src[0] = static_cast<const T *>(p.x) + (size_t)row * p.ldx;
        src[1] = static_cast<const T *>(p.h) + (size_t)row * p.ldh;
        src[2] = p.dy == nullptr ? nullptr : static_cast<const T *>(p.dy) + (size_t)row * p.D;
        src[3] = p.dr == nullptr ? nullptr : static_cast<const T *>(p.dr) + (size_t)row * p.D;
        src[4] = z0 == nullptr ? nullptr : z0 + (size_t)(p.gate_rows == 1 ? row : row / p.gate_rows) * p.ldz;
    };
    for (int unit = blockIdx.x; unit < p.units; unit += p.ctas) {
        const int gate = unit / p.per_gate, span = shared_z ? p.gate_rows : p.M;
        const int first = gate * span + unit % p.per_gate * p.unit;
        const int last = first + min(p.unit, min((gate + 1) * span, p.M) - first);
#pragma unroll
        for (int e = 0; e < P; ++e) dzs[e] = both(0.f);
        int next = first + at.slot;
        for (int i = 0; i < Ring::kAhead - 1; ++i, next += ROWS) {
            locate(next);
            ring.fetch(at, src, next < last);
        }
        for (int m = first + at.slot; m - at.slot < last; m += ROWS, next += ROWS) {
            const bool live = m < last;
            locate(next);
            ring.fetch(at, src, next < last);
            const float2 st = live ? *reinterpret_cast<const float2 *>(p.stats_in + 2 * (size_t)m) : both(0.f);
            ring.arrive();
            if (!Ring::kRing) locate(m);
            // rh, v = u hh, g = dr + rstd_r e, and the row's sums; a row behind the last is one of zeros
            float2 rh[P], hh[P], g[P], v[P], z[P];
            ring.read(at, 0, src[0], live, rh);
            ring.read(at, 1, src[1], live, hh);
            if (p.dr != nullptr) ring.read(at, 3, src[3], live, g);
            else
#pragma unroll
                for (int e = 0; e < P; ++e) g[e] = both(0.f);
            if (z0 != nullptr) ring.read(at, 4, src[4], live, z);
            if (!live)
#pragma unroll
                for (int e = 0; e < P; ++e) rh[e] = hh[e] = g[e] = z[e] = both(0.f);
#pragma unroll
            for (int e = 0; e < P; ++e) v[e] = hh[e] = mul2(hh[e], both(st.x));
            if (z0 != nullptr)
                with_act(p.act, [&](auto act) {
#pragma unroll
                    for (int e = 0; e < P; ++e) v[e] = mul2(act2<decltype(act)::value>(z[e]), hh[e]);
                });
#pragma unroll
            for (int e = 0; e < P; ++e) rh[e] = mul2(fma2(k[e], v[e], rh[e]), both(st.y));
            float2 q0 = both(0.f), q1 = both(0.f), q2 = both(0.f);
            if (p.pre) {
                float2 dy[P];
                ring.read(at, 2, src[2], live, dy);
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    if (ROWS > 1 && !live) dy[e] = both(0.f);
                    dwr[e] = fma2(dy[e], rh[e], dwr[e]);
                    dy[e] = mul2(dy[e], wr[e]);
                    q0 = fma2(dy[e], rh[e], q0);
                    g[e] = fma2(both(st.y), dy[e], g[e]);
                }
            }
#pragma unroll
            for (int e = 0; e < P; ++e) {
                const float2 t = mul2(k[e], v[e]);
                q1 = fma2(g[e], t, q1);
                q2 = fma2(rh[e], t, q2);
            }
            ring.done();
            float q[3] = {q0.x + q0.y, q1.x + q1.y, q2.x + q2.y};
            row_sum(q);
            const float c = p.pre ? st.y * q[0] * inv_D : 0.f, mean = p.post ? fmaf(-c, q[2], q[1]) * inv_D : 0.f;
#pragma unroll
            for (int e = 0; e < P; ++e) {
                g[e] = fma2(both(-c), rh[e], g[e]);                              // gr
                Q[e] = fma2(g[e], v[e], Q[e]);
            }
            if (live) at.store(static_cast<T *>(p.dx) + (size_t)m * p.D, g);
            float2 f[P];
#pragma unroll
            for (int e = 0; e < P; ++e) {
                const float2 gk = mul2(g[e], k[e]);
                f[e] = gk;
                g[e] = mul2(gk, hh[e]);                                          // dz before act'(z)
            }
            if (z0 != nullptr) {
                with_act(p.act, [&](auto act) {
                    constexpr int ACT = decltype(act)::value;
#pragma unroll
                    for (int e = 0; e < P; ++e) f[e] = mul2(f[e], act2<ACT>(z[e]));
                    if (!shared_z && ACT != kActNone)
#pragma unroll
                        for (int e = 0; e < P; ++e) g[e] = mul2(g[e], dact2<ACT>(z[e]));
                });
                if (shared_z)
#pragma unroll
                    for (int e = 0; e < P; ++e) dzs[e] = __fadd2_rn(dzs[e], g[e]);
                else if (live && p.dz != nullptr) at.store(static_cast<T *>(p.dz) + (size_t)m * p.D, g);
            }
#pragma unroll
            for (int e = 0; e < P; ++e) f[e] = mul2(fma2(both(-mean), hh[e], f[e]), both(st.x));
            if (live) at.store(static_cast<T *>(p.dh) + (size_t)m * p.D, f);
        }
        ring.restart();
        if (shared_z && p.dz != nullptr) {
            over_slots(dzs);
            if (at.slot == 0 && p.per_gate > 1) {
                at.put(p.part_z + (size_t)unit * p.D, dzs);
            } else if (at.slot == 0) {
                float2 z[P];
                at.read(z0 + (size_t)gate * p.ldz, z);
#pragma unroll
                for (int e = 0; e < P; ++e) dzs[e] = mul2(dzs[e], make_float2(dact_rt(p.act, z[e].x), dact_rt(p.act, z[e].y)));
                at.store(static_cast<T *>(p.dz) + (size_t)gate * p.D, dzs);
            }
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

// dz of a gate whose rows are shared by more than one unit: the units' sums, times act'(z).
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
// and more, four smaller ones; 32768 x 2048 in bf16 with two for each SM 172 us, with four 184)
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

// f(kernel parameters as types): the form for D channels of a type, in pieces of `width` of them (16 bytes, two or one).
// 999 x 1030 in float32 with a gate, in pairs and one by one: forward 11 and 15 us, backward 17 and 28.
// Eight channels of a thread on as few threads as hold the row, so that its sums meet in few places; sixteen where a
// warp can hold it so (to 512 channels) and where it would need more than 512 threads. The backward's five tensors, parameters and
// sums of eight channels are 126 registers; of sixteen it spills, 490 bytes of a thread with 512 threads, 1500 to 2200
// with 1024: 2^26 channels in bf16 in rows of 4096 take it 173 us, of 8192 264, of 16384 542.
template <typename T, typename F>
static cudaError_t with_row(int D, int width, F f) {
    constexpr int V = 16 / (int)sizeof(T), W = 8 / V;      // W: pieces of eight channels
#define GDN_ROW(V_, LPR_, IT_) return f(std::integral_constant<int, V_>(), std::integral_constant<int, LPR_>(), std::integral_constant<int, IT_>())
    if (width == V) {
        if (D <= 64) GDN_ROW(V, 8, W);
        if (D <= 256) GDN_ROW(V, 32, W);
        if (D <= 512) GDN_ROW(V, 32, 2 * W);
        if (D <= 1024) GDN_ROW(V, 128, W);
        if (D <= 2048) GDN_ROW(V, 256, W);
        if (D <= 4096) GDN_ROW(V, 512, W);
        if (D <= 8192) GDN_ROW(V, 512, 2 * W);
        GDN_ROW(V, 1024, 2 * W);
    }
    if (width == 2) {
        if (D <= 256) GDN_ROW(2, 32, 4);
        if (D <= 1024) GDN_ROW(2, 128, 4);
        if (D <= 2048) GDN_ROW(2, 256, 4);
        if (D <= 4096) GDN_ROW(2, 512, 4);
        GDN_ROW(2, 1024, 8);
    }
    if (D <= 256) GDN_ROW(1, 32, 8);
    if (D <= 1024) GDN_ROW(1, 128, 8);
    if (D <= 4096) GDN_ROW(1, 512, 8);
    GDN_ROW(1, 1024, 16);
#undef GDN_ROW
}

// Channels of a piece of every row: D and the row strides multiples of it, the addresses aligned to it
template <typename T>
static int rows_width(const ResnormParams &p) {
    for (int v : {16 / (int)sizeof(T), 2}) {
        const uintptr_t bytes = v * sizeof(T);
        if (p.D % v == 0 && p.ldx % v == 0 && p.ldh % v == 0 && (p.z == nullptr || p.ldz % v == 0) &&
            (((uintptr_t)p.x | (uintptr_t)p.h | (uintptr_t)p.z) & (bytes - 1)) == 0)
            return v;
    }
    return 1;
}

template <typename T>
static cudaError_t launch_fwd_t(const ResnormParams &p, cudaStream_t s) {
    return with_row<T>(p.D, rows_width<T>(p), [&](auto v, auto lpr, auto it) {
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
    cudaError_t e = with_row<T>(p.D, rows_width<T>(p), [&](auto v, auto lpr, auto it) {
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
    if (p.dz != nullptr && p.gate_rows > 1 && p.per_gate > 1)                   // (fewer gates than CTAs then)
        resnorm_gate_kernel<T><<<dim3((p.D + 31) / 32, p.M / p.gate_rows), 256, 0, s>>>(p);
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

// gdn_scan_bwd.cu -- selective state space scan, backward.
//
// With dcore = dy silu(z) and e_t the adjoint of h_t,
//     e_t = C_t dcore_t + a_{t+1} e_{t+1},  a = exp(d A)      (behind the last step: dh_T)
//     dC_t = sum_c dcore h_t,   dB_t = sum_c e d u,   dsu = sum_n e B,   kept = e a h_{t-1}
//     dd = sum_n kept A + dsu u,   ddt = dd sigmoid(dt + dt_bias),   du = dsu d + D dcore
//     dA_log = A sum kept d,   dD = sum dcore u,   dz = dy (C . h + D u) silu'(z),   dh0 = a_0 e_0
// The sums over c run over the channels that share B and C.
//
// A CTA of 4 warps walks its channels' tiles of 16 steps from the last to the first, and each half of
// a tile: from the tile's checkpoint it forms the half's states again, keeps them in registers, and
// sweeps back over them. What costs most is not that arithmetic but the sums: per step, dB and dC over
// the channels and three sums over a channel's states. So a group of LPC lanes takes two channels (8
// states a lane): the two are added in registers, and the rest by exchanging halves, where lanes hold
// their states, and their two channels, in different order, chosen so that every lane keeps its first
// registers and sends the others, without selects. Per state and step that takes half of the
// instructions and of the shared-memory passes that one channel per group takes.
//
// Measured on 2 x 2048 steps of 4096 channels x 16 states, bf16, in 7 segments: 67 us for the segments'
// start adjoints, 319 us for the sweep, 18 and 4 us for the sums and the combination. The sweep issues 217
// instructions per step of 256 states, in 53 % of the cycles, with two CTAs of 252 registers per SM: it is
// bound by instructions and their latency, not by its 140 MB. Decays formed twice instead of kept (three
// CTAs per SM) and segments of any count: 83 us more, forward and backward.
#include "gdn_scan.cuh"

namespace gdn {

namespace {

constexpr int kRevThreads = 128, kRevWarps = kRevThreads / 32, kHalf = kScanTile / 2, kRevCtas = 2;

// The order of a lane's states: register k holds state n0 + (k ^ order).
template <int LPC>
__device__ __forceinline__ int state_order(int lane) {
    if (LPC == 4) return (lane >> 3 & 1) * 2 + (lane >> 2 & 1);
    if (LPC == 8) return (lane >> 3 & 1) * 2 + (lane >> 4 & 1);
    return (lane >> 4 & 1) * 2;
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float4 lds4(const float *p) { return *reinterpret_cast<const float4 *>(p); }

template <int LPC, typename T>
struct BwdSmem {
    using G = ScanGeo<LPC>;
    static constexpr int CH = G::CH, NP = G::NP, TT = kScanTile;
    // staged inputs: d, d u, dcore, sigmoid(dt + dt_bias); results: dsu and sum kept A (their rows 16
    // banks apart, as one store writes both), C . h
    float d[TT][CH], xu[TT][CH], dc[TT][CH], sg[TT][CH];
    float dsu[TT][CH], gap[16], kd[TT][CH], core[TT][CH];
    float B[TT][4][NP], C[TT][4][NP];             // for each order of the states
    float bc[kRevWarps][TT][2 * NP];              // a warp's dB, dC
    float D[CH], bias[CH];
    T u[TT][CH], z[TT][CH], dy[TT][CH];
};

// V floats from shared memory (aligned to V floats)
template <int V>
__device__ __forceinline__ void lds(const float *p, float (&o)[V]) { load_vec<float, V>(p, o); }
// the pairs (x, x) of two neighbouring values
__device__ __forceinline__ void lds_pairs(const float *p, float2 (&o)[2]) {
    const float2 x = *reinterpret_cast<const float2 *>(p);
    o[0] = both(x.x);
    o[1] = both(x.y);
}
__device__ __forceinline__ float2 dsilu2_hw(float2 x) {
    const float2 one = make_float2(1.f, 1.f), s = sigmoid2_hw(x);
    return __fmul2_rn(s, __ffma2_rn(x, __ffma2_rn(s, make_float2(-1.f, -1.f), one), one));
}

}  // namespace

// LITE: the segment's start adjoint from a zero end and its sum of d, nothing else.
template <int LPC, typename T, bool VEC, bool LITE>
__global__ void __launch_bounds__(kRevThreads, LITE ? 4 : kRevCtas) scan_bwd_kernel(ScanParams p) {
    using G = ScanGeo<LPC>;
    constexpr int CH = G::CH, NP = G::NP, V = G::V, TT = kScanTile, KB = NP * TT / kRevThreads;
    constexpr int PASS = TT * CH / V / kRevThreads;               // staged groups of V per thread (2)
    extern __shared__ __align__(16) unsigned char smem_raw[];
    BwdSmem<LPC, T> &sm = *reinterpret_cast<BwdSmem<LPC, T> *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const ScanPlace q = scan_place<LPC>(p);
    if (q.first >= q.last) return;
    const int L = row_length(p.lens, q.b, p.T);
    // staged elements: steps ts and ts + 8 of a tile, V channels from cv
    const int ts = tid >> 4, cv = (tid & 15) * V, nv = q.nc - cv;
    // states: channels cb and cb + 1, states n0 + (k ^ order)
    const int n0 = 4 * (lane % LPC), order = state_order<LPC>(lane);
    const int cb = (warp * G::CPW + lane / LPC) * 2;
    const T *u = static_cast<const T *>(p.u) + (size_t)q.b * p.T * p.ldu + q.c0 + cv;
    const T *dt = static_cast<const T *>(p.dt) + (size_t)q.b * p.T * p.lddt + q.c0 + cv;
    const T *z = static_cast<const T *>(p.z) + (size_t)q.b * p.T * p.ldz + q.c0 + cv;
    const size_t row = (size_t)q.b * p.T * p.Cn + q.c0 + cv;      // packed [B, T, C] tensors
    const T *dy = static_cast<const T *>(p.dy) + row;
    const T *Bm = static_cast<const T *>(p.B) + (size_t)q.b * p.T * p.ldB + q.g * p.N;
    const T *Cm = static_cast<const T *>(p.C) + (size_t)q.b * p.T * p.ldC + q.g * p.N;
    const int tiles = (p.T + TT - 1) / TT;
    // this lane's states of rows [channel][N], in its order (zeros, or nothing, beyond channels and N)
    auto load_mine = [&](const float *rows, float2 (&o)[2][2]) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float e[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int n = n0 + (k ^ order);
                e[k] = 0.f;
                if (n < p.N && cb + r < q.nc) e[k] = rows[(size_t)(q.c0 + cb + r) * p.N + n];
            }
            o[r][0] = make_float2(e[0], e[1]);
            o[r][1] = make_float2(e[2], e[3]);
        }
    };
    auto store_mine = [&](float *rows, const float2 (&o)[2][2]) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float e[4] = {o[r][0].x, o[r][0].y, o[r][1].x, o[r][1].y};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int n = n0 + (k ^ order);
                if (n < p.N && cb + r < q.nc) rows[(size_t)(q.c0 + cb + r) * p.N + n] = e[k];
            }
        }
    };
    Staged<T, V, VEC> ru[PASS], rd[PASS], rz[PASS], ry[PASS];
    T rB[KB], rC[KB];
    float2 rh[2][2];
    auto fetch = [&](int tile) {
#pragma unroll
        for (int i = 0; i < PASS; ++i) {
            const int t = tile * TT + ts + 8 * i, n = t < L ? nv : 0;
            if (!LITE) ru[i].load(u + (size_t)t * p.ldu, n);
            rd[i].load(dt + (size_t)t * p.lddt, n);
            if (p.z != nullptr) rz[i].load(z + (size_t)t * p.ldz, n);
            ry[i].load(dy + (size_t)t * p.Cn, n);
        }
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            const int e = tid + kRevThreads * k, tb = tile * TT + e / NP, n1 = e % NP;
            const bool ok = tb < L && n1 < p.N;
            rB[k] = rC[k] = from_f32<T>(0.f);
            if (!LITE && ok) rB[k] = Bm[(size_t)tb * p.ldB + n1];
            if (ok) rC[k] = Cm[(size_t)tb * p.ldC + n1];
        }
        if (!LITE) load_mine(p.ckpt + ((size_t)q.b * tiles + tile) * p.Cn * p.N, rh);
    };
    // the segment's tiles with valid steps are [q.first, live). Those behind them pass the adjoint on and
    // have no gradients; a state that is not finite (a row without valid steps may carry one) would make
    // NaN of the zeros that they would add.
    const int live = min(q.last, max(q.first, (L + TT - 1) / TT));
    if (live > q.first) fetch(live - 1);
    for (int i = tid; i < CH; i += kRevThreads) {
        sm.D[i] = p.D != nullptr && i < q.nc ? p.D[q.c0 + i] : 0.f;
        sm.bias[i] = p.dt_bias != nullptr && i < q.nc ? p.dt_bias[q.c0 + i] : 0.f;
    }
    float2 A2[2][2], ge[2][2], dA[2][2];           // A log2 e
    load_mine(p.A_log, A2);
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const bool in0 = cb + r < q.nc && n0 + ((2 * k) ^ order) < p.N, in1 = cb + r < q.nc && n0 + ((2 * k + 1) ^ order) < p.N;
            A2[r][k] = make_float2(in0 ? -expf(A2[r][k].x) * kLog2e : 0.f, in1 ? -expf(A2[r][k].y) * kLog2e : 0.f);
            ge[r][k] = dA[r][k] = both(0.f);
        }
    const size_t states = (size_t)p.Cn * p.N;
    if (!LITE) {
        if (p.segs > 1) load_mine(p.seg_state + ((size_t)q.seg * p.Bn + q.b) * states, ge);
        else if (p.dh_T != nullptr) load_mine(p.dh_T + q.b * states, ge);
    }
    float sum_d[V], sum_D[V], sum_b[V];
#pragma unroll
    for (int v = 0; v < V; ++v) sum_d[v] = sum_D[v] = sum_b[v] = 0.f;
    __syncthreads();
    for (int tile = live - 1; tile >= q.first; --tile) {
#pragma unroll
        for (int i = 0; i < PASS; ++i) {
            const int t = tile * TT + ts + 8 * i, st = ts + 8 * i;
            float uu[V], dd[V], zz[V], yy[V], bias[V], xu[V], dc[V], sg[V];
            rd[i].get(dd);
            ry[i].get(yy);
#pragma unroll
            for (int v = 0; v < V; ++v) uu[v] = zz[v] = 0.f;
            if (!LITE) ru[i].get(uu);
            if (p.z != nullptr) rz[i].get(zz);
            lds<V>(sm.bias + cv, bias);
            if constexpr (V == 1) {
                softplus_full(dd[0] + bias[0], dd[0], sg[0]);
                dc[0] = p.z != nullptr ? yy[0] * silu_hw(zz[0]) : yy[0];
            } else {
#pragma unroll
                for (int v = 0; v < V; v += 2) {
                    float2 sp, s2, c2 = make_float2(yy[v], yy[v + 1]);
                    softplus2_full(make_float2(dd[v] + bias[v], dd[v + 1] + bias[v + 1]), sp, s2);
                    if (p.z != nullptr) {
                        const float2 z2 = make_float2(zz[v], zz[v + 1]);
                        c2 = __fmul2_rn(c2, __fmul2_rn(z2, sigmoid2_hw(z2)));
                    }
                    dd[v] = sp.x; dd[v + 1] = sp.y;
                    sg[v] = s2.x; sg[v + 1] = s2.y;
                    dc[v] = c2.x; dc[v + 1] = c2.y;
                }
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (t >= L) dd[v] = 0.f;
                if (LITE) sum_d[v] += dd[v];
                xu[v] = dd[v] * uu[v];
            }
            store_vec<float, V>(&sm.d[st][cv], dd);
            store_vec<float, V>(&sm.dc[st][cv], dc);
            if (!LITE) {
                store_vec<float, V>(&sm.xu[st][cv], xu);
                store_vec<float, V>(&sm.sg[st][cv], sg);
                ru[i].keep(&sm.u[st][cv]);
                if (p.z != nullptr) rz[i].keep(&sm.z[st][cv]);
                ry[i].keep(&sm.dy[st][cv]);
            }
        }
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            const int e = tid + kRevThreads * k, i = e / NP, n = e % NP;
            const float fb = to_f32(rB[k]), fc = to_f32(rC[k]);
#pragma unroll
            for (int o = 0; o < 4; ++o) {
                if (!LITE) sm.B[i][o][n ^ o] = fb;
                sm.C[i][o][n ^ o] = fc;
            }
        }
        float2 start[2][2];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int k = 0; k < 2; ++k) start[r][k] = rh[r][k];
        __syncthreads();
        if (tile > q.first) fetch(tile - 1);
        if (LITE) {
#pragma unroll
            for (int i = TT - 1; i >= 0; --i) {
                const float4 c4 = lds4(&sm.C[i][order][n0]);
                const float2 c2[2] = {make_float2(c4.x, c4.y), make_float2(c4.z, c4.w)};
                float2 d[2], dc[2];
                lds_pairs(&sm.d[i][cb], d);
                lds_pairs(&sm.dc[i][cb], dc);
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        ge[r][k] = __fmul2_rn(__ffma2_rn(dc[r], c2[k], ge[r][k]), decay2(d[r], A2[r][k]));
            }
            __syncthreads();
            continue;
        }
        auto forward = [&](int i, const float2 (&h)[2][2], float2 (&to)[2][2], float2 (&a)[2][2]) {
            const float4 b4 = lds4(&sm.B[i][order][n0]);
            const float2 b2[2] = {make_float2(b4.x, b4.y), make_float2(b4.z, b4.w)};
            float2 d[2], xu[2];
            lds_pairs(&sm.d[i][cb], d);
            lds_pairs(&sm.xu[i][cb], xu);
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                {
                    a[r][k] = decay2(d[r], A2[r][k]);
                    to[r][k] = __ffma2_rn(a[r][k], h[r][k], __fmul2_rn(xu[r], b2[k]));
                }
        };
        float2 mid[2][2], tile_dA[2][2];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                mid[r][k] = start[r][k];
                tile_dA[r][k] = both(0.f);
            }
#pragma unroll
        for (int i = 0; i < kHalf; ++i) {
            float2 a[2][2];
            forward(i, mid, mid, a);
        }
#pragma unroll 1
        for (int half = 1; half >= 0; --half) {
            float2 h[kHalf + 1][2][2], a[kHalf][2][2];
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int k = 0; k < 2; ++k) h[0][r][k] = half ? mid[r][k] : start[r][k];
#pragma unroll
            for (int i = 0; i < kHalf; ++i) forward(half * kHalf + i, h[i], h[i + 1], a[i]);
#pragma unroll
            for (int j = kHalf - 1; j >= 0; --j) {
                const int i = half * kHalf + j;
                const float4 b4 = lds4(&sm.B[i][order][n0]), c4 = lds4(&sm.C[i][order][n0]);
                const float2 b2[2] = {make_float2(b4.x, b4.y), make_float2(b4.z, b4.w)};
                const float2 c2[2] = {make_float2(c4.x, c4.y), make_float2(c4.z, c4.w)};
                float2 gB[2], gC[2];
                float sums[2][3];                       // dsu, sum kept A log2 e, C . h
                float2 d[2], xu[2], dc[2];
                lds_pairs(&sm.d[i][cb], d);
                lds_pairs(&sm.xu[i][cb], xu);
                lds_pairs(&sm.dc[i][cb], dc);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float2 dsu, kd, core;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float2 e = __ffma2_rn(dc[r], c2[k], ge[r][k]);
                        gB[k] = r == 0 ? __fmul2_rn(e, xu[r]) : __ffma2_rn(e, xu[r], gB[k]);
                        gC[k] = r == 0 ? __fmul2_rn(dc[r], h[j + 1][0][k]) : __ffma2_rn(dc[r], h[j + 1][1][k], gC[k]);
                        ge[r][k] = __fmul2_rn(e, a[j][r][k]);
                        const float2 kept = __fmul2_rn(ge[r][k], h[j][r][k]);
                        tile_dA[r][k] = __ffma2_rn(kept, d[r], tile_dA[r][k]);
                        dsu = k == 0 ? __fmul2_rn(e, b2[0]) : __ffma2_rn(e, b2[1], dsu);
                        core = k == 0 ? __fmul2_rn(c2[0], h[j + 1][r][0]) : __ffma2_rn(c2[1], h[j + 1][r][1], core);
                        kd = k == 0 ? __fmul2_rn(kept, A2[r][0]) : __ffma2_rn(kept, A2[r][1], kd);
                    }
                    sums[r][0] = dsu.x + dsu.y;
                    sums[r][1] = kd.x + kd.y;
                    sums[r][2] = core.x + core.y;
                }
                // dB, dC over the warp's channels: keep the first half, send the second
                constexpr int m1 = LPC == 16 ? 16 : 8, m0 = LPC == 4 ? 4 : 16;
                gB[0] = __fadd2_rn(gB[0], shfl2(gB[1], m1));
                gC[0] = __fadd2_rn(gC[0], shfl2(gC[1], m1));
                float *bc = sm.bc[warp][i] + n0;
                if constexpr (LPC == 16) {
                    *reinterpret_cast<float2 *>(bc + order) = gB[0];
                    *reinterpret_cast<float2 *>(bc + NP + order) = gC[0];
                } else {
                    const float2 s = __fadd2_rn(make_float2(gB[0].x, gC[0].x), shfl2(make_float2(gB[0].y, gC[0].y), m0));
                    if constexpr (LPC == 8) {
                        bc[order] = s.x;
                        bc[NP + order] = s.y;
                    } else {
                        const bool up = lane & 16;
                        bc[(up ? NP : 0) + order] = (up ? s.y : s.x) + __shfl_xor_sync(kFullMask, up ? s.x : s.y, 16);
                    }
                }
                // a channel's three sums over its lanes: bit 1 of the lane keeps one channel, then bit 0
                // one of dsu and the kept sum; C . h goes to both
                const bool up2 = lane & 2, up1 = lane & 1;
                float x[3];
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    x[k] = (up2 ? sums[1][k] : sums[0][k]) + __shfl_xor_sync(kFullMask, up2 ? sums[0][k] : sums[1][k], 2);
                float y = (up1 ? x[1] : x[0]) + __shfl_xor_sync(kFullMask, up1 ? x[0] : x[1], 1);
                x[2] += __shfl_xor_sync(kFullMask, x[2], 1);
#pragma unroll
                for (int m = 4; m < LPC; m <<= 1) {
                    y += __shfl_xor_sync(kFullMask, y, m);
                    x[2] += __shfl_xor_sync(kFullMask, x[2], m);
                }
                if (lane % LPC < 4) {
                    const int cc = cb + (lane >> 1 & 1);
                    *(up1 ? &sm.kd[i][cc] : &sm.dsu[i][cc]) = y;
                    if (!up1) sm.core[i][cc] = x[2];
                }
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int k = 0; k < 2; ++k) dA[r][k] = __fadd2_rn(dA[r][k], tile_dA[r][k]);
        __syncthreads();
        // each staged element's gradients
#pragma unroll
        for (int i = 0; i < PASS; ++i) {
            const int st = ts + 8 * i, t = tile * TT + st;
            if (t >= p.T) continue;
            float du[V], ddt[V], dz[V], uu[V], zz[V], yy[V], D[V], d[V], dc[V], sg[V], dsu[V], kd[V], core[V];
            lds<V>(&sm.d[st][cv], d);
            lds<V>(&sm.dc[st][cv], dc);
            lds<V>(&sm.sg[st][cv], sg);
            lds<V>(&sm.dsu[st][cv], dsu);
            lds<V>(&sm.kd[st][cv], kd);
            lds<V>(&sm.core[st][cv], core);
            lds<V>(sm.D + cv, D);
            load_vec<T, V>(&sm.u[st][cv], uu);
            load_vec<T, V>(&sm.dy[st][cv], yy);
#pragma unroll
            for (int v = 0; v < V; ++v) zz[v] = 0.f;
            if (p.z != nullptr) load_vec<T, V>(&sm.z[st][cv], zz);
            const bool on = t < L;
            if (p.z != nullptr) {
                if constexpr (V == 1) {
                    zz[0] = dsilu_hw(zz[0]);
                } else {
#pragma unroll
                    for (int v = 0; v < V; v += 2) {
                        const float2 q2 = dsilu2_hw(make_float2(zz[v], zz[v + 1]));
                        zz[v] = q2.x;
                        zz[v + 1] = q2.y;
                    }
                }
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                du[v] = on ? fmaf(dsu[v], d[v], D[v] * dc[v]) : 0.f;
                ddt[v] = on ? fmaf(dsu[v], uu[v], kd[v] * 0.69314718f) * sg[v] : 0.f;
                dz[v] = on ? yy[v] * fmaf(D[v], uu[v], core[v]) * zz[v] : 0.f;
                sum_D[v] += on ? dc[v] * uu[v] : 0.f;
                sum_b[v] += ddt[v];
            }
            const size_t at = row + (size_t)t * p.Cn;
            store_channels<T, V>(static_cast<T *>(p.du) + at, nv, VEC, du);
            store_channels<T, V>(static_cast<T *>(p.ddt) + at, nv, VEC, ddt);
            if (p.dz != nullptr) store_channels<T, V>(static_cast<T *>(p.dz) + at, nv, VEC, dz);
        }
        // the CTA's dB, dC of the tile: over its warps in ascending order
        for (int e = tid; e < TT * 2 * NP; e += kRevThreads) {
            const int i = e / (2 * NP), n = e % (2 * NP), tb = tile * TT + i;
            if (tb >= p.T || n % NP >= p.N) continue;
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kRevWarps; ++w) s += sm.bc[w][i][n];
            if (tb >= L) s = 0.f;
            p.part_bc[((((size_t)q.blk * p.Bn + q.b) * p.T + tb) * p.G + q.g) * (2 * p.N) + (n / NP) * p.N + n % NP] = s;
        }
        __syncthreads();
    }
    if (LITE) {
        store_mine(p.seg_state + ((size_t)q.seg * p.Bn + q.b) * states, ge);
        float *s = &sm.dsu[0][0];
#pragma unroll
        for (int v = 0; v < V; ++v) s[ts * CH + cv + v] = sum_d[v];
        __syncthreads();
        if (tid < q.nc) {
            float x = 0.f;
            for (int i = 0; i < 8; ++i) x += s[i * CH + tid];
            p.seg_sum[((size_t)q.seg * p.Bn + q.b) * p.Cn + q.c0 + tid] = x;
        }
        return;
    }
    if (p.segs == 1 && p.dh0 != nullptr) store_mine(p.dh0 + q.b * states, ge);
    for (int t = live * TT + ts; t < min(q.last * TT, p.T); t += 8) {
        const float zero[V] = {};
        const size_t at = row + (size_t)t * p.Cn;
        store_channels<T, V>(static_cast<T *>(p.du) + at, nv, VEC, zero);
        store_channels<T, V>(static_cast<T *>(p.ddt) + at, nv, VEC, zero);
        if (p.dz != nullptr) store_channels<T, V>(static_cast<T *>(p.dz) + at, nv, VEC, zero);
        float *part = p.part_bc + ((((size_t)q.blk * p.Bn + q.b) * p.T + t) * p.G + q.g) * (2 * p.N);
        for (int n = tid & 15; n < 2 * p.N; n += 16) part[n] = 0.f;
    }
    float *part = p.part_c + ((size_t)q.seg * p.Bn + q.b) * (p.N + 2) * p.Cn;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const float e[4] = {dA[r][0].x, dA[r][0].y, dA[r][1].x, dA[r][1].y};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int n = n0 + (k ^ order);
            if (n < p.N && cb + r < q.nc) part[(size_t)n * p.Cn + q.c0 + cb + r] = e[k];
        }
    }
    float *s = &sm.dsu[0][0];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        s[ts * CH + cv + v] = sum_D[v];
        s[(8 + ts) * CH + cv + v] = sum_b[v];
    }
    __syncthreads();
    for (int e = tid; e < 2 * CH; e += kRevThreads) {
        const int which = e / CH, cc = e % CH;
        if (cc >= q.nc) continue;
        float x = 0.f;
        for (int i = 0; i < 8; ++i) x += s[(which * 8 + i) * CH + cc];
        part[(size_t)(p.N + which) * p.Cn + q.c0 + cc] = x;
    }
}

// The last sums: dB, dC over the channel blocks of their group (the CTAs below n_bc), dA_log, dD and
// ddt_bias over the segments and batch rows (the others).
template <typename T>
__global__ void __launch_bounds__(256) scan_reduce_kernel(ScanParams p, int blocks, unsigned n_bc) {
    const bool bc = blockIdx.x < n_bc;
    const unsigned blk = bc ? blockIdx.x : blockIdx.x - n_bc;
    const size_t n = bc ? (size_t)p.Bn * p.T * p.G * 2 * p.N : (size_t)(p.N + 2) * p.Cn, i = (size_t)blk * 32 + threadIdx.x;
    const float s = slice_sum(bc ? p.part_bc : p.part_c, bc ? blocks : p.segs * p.Bn, n, blk);
    if (threadIdx.x >= 32 || i >= n) return;
    if (bc) {
        const size_t row = i / (2 * p.N);
        const int m = (int)(i % (2 * p.N));
        if (m < p.N) static_cast<T *>(p.dB)[row * p.N + m] = from_f32<T>(s);
        else static_cast<T *>(p.dC)[row * p.N + m - p.N] = from_f32<T>(s);
        return;
    }
    const int m = (int)(i / p.Cn), c = (int)(i % p.Cn);
    if (m < p.N) {
        const size_t o = (size_t)c * p.N + m;
        p.dA_log[o] = s * -expf(p.A_log[o]);
    } else if (m == p.N) {
        if (p.dD != nullptr) p.dD[c] = s;
    } else if (p.ddt_bias != nullptr) {
        p.ddt_bias[c] = s;
    }
}

namespace {

template <int LPC, typename T, bool VEC, bool LITE>
cudaError_t scan_bwd_one(const ScanParams &p, cudaStream_t s) {
    const cudaError_t e = allow_smem<scan_bwd_kernel<LPC, T, VEC, LITE>>((int)sizeof(BwdSmem<LPC, T>));
    if (e != cudaSuccess) return e;
    const dim3 grid(p.Bn * p.G * scan_blocks(p.Cn, p.G, p.N), p.segs);
    const char *name = LITE ? "scan_bwd_ends" : "scan_bwd";
    timing_mark(name, 0, s);
    scan_bwd_kernel<LPC, T, VEC, LITE><<<grid, kRevThreads, sizeof(BwdSmem<LPC, T>), s>>>(p);
    timing_mark(name, 1, s);
    return cudaGetLastError();
}

template <int LPC, typename T, bool VEC>
cudaError_t scan_bwd_prompt(const ScanParams &p, cudaStream_t s) {
    cudaError_t e;
    if (p.segs > 1) {
        if ((e = scan_bwd_one<LPC, T, VEC, true>(p, s)) != cudaSuccess) return e;
        if ((e = launch_scan_combine(p, p.dh_T, p.dh0, true, s)) != cudaSuccess) return e;
    }
    return scan_bwd_one<LPC, T, VEC, false>(p, s);
}

template <int LPC, typename T>
cudaError_t scan_bwd_launch(const ScanParams &p, cudaStream_t s) {
    cudaError_t e = scan_vec<T>(p, ScanGeo<LPC>::V) ? scan_bwd_prompt<LPC, T, true>(p, s) : scan_bwd_prompt<LPC, T, false>(p, s);
    if (e != cudaSuccess) return e;
    const size_t n = (size_t)p.Bn * p.T * p.G * 2 * p.N, m = (size_t)(p.N + 2) * p.Cn;
    const unsigned n_bc = (unsigned)((n + 31) / 32), n_c = (unsigned)((m + 31) / 32);
    timing_mark("scan_reduce", 0, s);
    scan_reduce_kernel<T><<<n_bc + n_c, 256, 0, s>>>(p, scan_blocks(p.Cn, p.G, p.N), n_bc);
    timing_mark("scan_reduce", 1, s);
    return cudaGetLastError();
}

template <typename T>
cudaError_t scan_bwd_lanes(const ScanParams &p, cudaStream_t s) {
    switch (scan_lanes(p.N)) {
        case 4: return scan_bwd_launch<4, T>(p, s);
        case 8: return scan_bwd_launch<8, T>(p, s);
        default: return scan_bwd_launch<16, T>(p, s);
    }
}

}  // namespace

cudaError_t launch_scan_bwd(const ScanParams &p, int dtype, cudaStream_t s) {
    return dtype == 0 ? scan_bwd_lanes<float>(p, s) : scan_bwd_lanes<__nv_bfloat16>(p, s);
}

}  // namespace gdn

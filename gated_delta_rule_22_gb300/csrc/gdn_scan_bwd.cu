// gdn_scan_bwd.cu -- selective state space scan, backward.
//
// With dcore = dy silu(z) and e_t the adjoint of h_t,
//     e_t = C_t dcore_t + a_{t+1} e_{t+1},  a = exp(d A)      (behind the last step: dh_T)
//     dC_t = sum_c dcore h_t,   dB_t = sum_c e d u,   dsu = sum_n e B,   kept = e a h_{t-1}
//     dd = sum_n kept A + dsu u,   ddt = dd sigmoid(dt + dt_bias),   du = dsu d + D dcore
//     dA_log = A sum kept d,   dD = sum dcore u,   dz = dy (C . h + D u) silu'(z),   dh0 = a_0 e_0
// The sums over c run over the channels that share B and C.
//
// A CTA walks its channels' tiles of 16 steps from the last to the first. In each it forms the 16
// states again from the tile's checkpoint, keeps them and their decays in registers, and sweeps
// back over them. What costs most is not that arithmetic (about 12 float32 operations per state and
// step) but its sums: per step, eight values (dB, dC of four states) over the warp's channels and three
// over a channel's lanes. Both exchange halves, so that each exchange also shortens what is left; for
// the first, lanes of different channels hold their four states in different order, chosen so that
// every lane keeps its first register and sends the others: no selects.
#include "gdn_scan.cuh"

namespace gdn {

namespace {

// The order of a lane's states: register k holds state n0 + (k ^ order).
template <int LPC>
__device__ __forceinline__ int state_order(int lane) {
    if (LPC == 4) return (lane >> 3 & 1) * 2 + (lane >> 2 & 1);
    if (LPC == 8) return (lane >> 3 & 1) * 2 + (lane >> 4 & 1);
    return (lane >> 4 & 1) * 2;
}

__device__ __forceinline__ float2 shfl2(float2 v, int m) {
    return make_float2(__shfl_xor_sync(kFullMask, v.x, m), __shfl_xor_sync(kFullMask, v.y, m));
}

// x + y with what the addition lost added to `lost`.
__device__ __forceinline__ void add_comp(float &x, float &lost, float y) {
    const float s = __fadd_rn(x, y), bb = __fadd_rn(s, -x);
    lost = __fadd_rn(lost, __fadd_rn(__fadd_rn(x, -__fadd_rn(s, -bb)), __fadd_rn(y, -bb)));
    x = s;
}

template <int LPC>
struct BwdSmem {
    using G = ScanGeo<LPC>;
    float4 in[kScanTile][G::CH];                  // d, d u, dcore, sigmoid(dt + dt_bias)
    float B[4][kScanTile][G::NP], C[4][kScanTile][G::NP];   // for each order of the states
    float4 out[kScanTile][G::CH];                 // dsu, sum kept A, C . h
    float bc[kScanWarps][kScanTile][2 * G::NP];   // a warp's dB, dC
};

}  // namespace

// LITE: the segment's start adjoint from a zero end and its sum of d, nothing else.
template <int LPC, typename T, bool VEC, bool LITE>
__global__ void __launch_bounds__(kScanThreads, 1) scan_bwd_kernel(ScanParams p) {
    using G = ScanGeo<LPC>;
    constexpr int CH = G::CH, NP = G::NP, V = G::V, KB = G::KB, TT = kScanTile;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    BwdSmem<LPC> &sm = *reinterpret_cast<BwdSmem<LPC> *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const ScanPlace q = scan_place<LPC>(p);
    if (q.first >= q.last) return;
    const int L = row_length(p.lens, q.b, p.T);
    const int ts = tid >> 4, cv = (tid & 15) * V, nv = q.nc - cv;
    const int ch = warp * G::CPW + lane / LPC, n0 = 4 * (lane % LPC), order = state_order<LPC>(lane);
    const bool live = ch < q.nc;
    const int c = q.c0 + (live ? ch : 0);
    const T *u = static_cast<const T *>(p.u) + (size_t)q.b * p.T * p.ldu + q.c0 + cv;
    const T *dt = static_cast<const T *>(p.dt) + (size_t)q.b * p.T * p.lddt + q.c0 + cv;
    const T *z = static_cast<const T *>(p.z) + (size_t)q.b * p.T * p.ldz + q.c0 + cv;
    const size_t row = (size_t)q.b * p.T * p.Cn + q.c0 + cv;      // packed [B, T, C] tensors
    const T *dy = static_cast<const T *>(p.dy) + row;
    const T *Bm = static_cast<const T *>(p.B) + (size_t)q.b * p.T * p.ldB + q.g * p.N;
    const T *Cm = static_cast<const T *>(p.C) + (size_t)q.b * p.T * p.ldC + q.g * p.N;
    const int tiles = (p.T + TT - 1) / TT;
    // this lane's four states of a row of N, in its order
    auto load_mine = [&](const float *r, float2 (&o)[2]) {
        float e[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int n = n0 + (k ^ order);
            e[k] = 0.f;
            if (n < p.N) e[k] = r[n];
        }
        o[0] = make_float2(e[0], e[1]);
        o[1] = make_float2(e[2], e[3]);
    };
    auto store_mine = [&](float *r, const float2 (&o)[2]) {
        const float e[4] = {o[0].x, o[0].y, o[1].x, o[1].y};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int n = n0 + (k ^ order);
            if (n < p.N) r[n] = e[k];
        }
    };
    Staged<T, V, VEC> ru, rd, rz, ry;
    T rB[KB], rC[KB];
    float2 rh[2];
    auto fetch = [&](int tile) {
        const int t = tile * TT + ts, n = t < L ? nv : 0;
        if (!LITE) ru.load(u + (size_t)t * p.ldu, n);
        rd.load(dt + (size_t)t * p.lddt, n);
        if (p.z != nullptr) rz.load(z + (size_t)t * p.ldz, n);
        ry.load(dy + (size_t)t * p.Cn, n);
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            const int e = tid + kScanThreads * k, tb = tile * TT + e / NP, n1 = e % NP;
            const bool ok = tb < L && n1 < p.N;
            rB[k] = rC[k] = from_f32<T>(0.f);
            if (!LITE && ok) rB[k] = Bm[(size_t)tb * p.ldB + n1];
            if (ok) rC[k] = Cm[(size_t)tb * p.ldC + n1];
        }
        if (!LITE) load_mine(p.ckpt + (((size_t)q.b * tiles + tile) * p.Cn + c) * p.N, rh);
    };
    fetch(q.last - 1);
    float2 A[2], ge[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    float dA[4] = {0.f, 0.f, 0.f, 0.f}, dA_lost[4] = {0.f, 0.f, 0.f, 0.f};
    float D[V], bias[V], sum_d[V], sum_D[V], sum_b[V];
    load_mine(p.A_log + (size_t)c * p.N, A);
    {
        float e[4] = {A[0].x, A[0].y, A[1].x, A[1].y};
#pragma unroll
        for (int k = 0; k < 4; ++k) e[k] = n0 + (k ^ order) < p.N ? -expf(e[k]) : 0.f;
        A[0] = make_float2(e[0], e[1]);
        A[1] = make_float2(e[2], e[3]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        D[v] = p.D != nullptr && v < nv ? p.D[q.c0 + cv + v] : 0.f;
        bias[v] = p.dt_bias != nullptr && v < nv ? p.dt_bias[q.c0 + cv + v] : 0.f;
        sum_d[v] = sum_D[v] = sum_b[v] = 0.f;
    }
    const size_t state_row = ((size_t)q.b * p.Cn + c) * p.N;
    if (!LITE && live) {
        if (p.segs > 1) load_mine(p.seg_state + (size_t)q.seg * p.Bn * p.Cn * p.N + state_row, ge);
        else if (p.dh_T != nullptr) load_mine(p.dh_T + state_row, ge);
    }
    for (int tile = q.last - 1; tile >= q.first; --tile) {
        const int t = tile * TT + ts;
        const Staged<T, V, VEC> cu = ru, cz = rz, cy = ry;
        {
            float uu[V], dd[V], zz[V], yy[V];
            if (!LITE) cu.get(uu);
            rd.get(dd);
            cz.get(zz);
            cy.get(yy);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float d, sg;
                softplus_full(dd[v] + bias[v], d, sg);
                if (t >= L) d = 0.f;
                if (LITE) sum_d[v] += d;
                sm.in[ts][cv + v] = make_float4(d, LITE ? 0.f : d * uu[v], p.z != nullptr ? yy[v] * silu_hw(zz[v]) : yy[v], sg);
            }
        }
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            const int e = tid + kScanThreads * k, i = e / NP, n = e % NP;
            const float fb = to_f32(rB[k]), fc = to_f32(rC[k]);
#pragma unroll
            for (int o = 0; o < 4; ++o) {
                if (!LITE) sm.B[o][i][n ^ o] = fb;
                sm.C[o][i][n ^ o] = fc;
            }
        }
        float2 hs[2] = {rh[0], rh[1]};
        __syncthreads();
        if (tile > q.first) fetch(tile - 1);
        float2 a[TT][2], h[TT + 1][2];
        h[0][0] = hs[0];
        h[0][1] = hs[1];
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            const float2 in = *reinterpret_cast<const float2 *>(&sm.in[i][ch]);
            float4 b4 = make_float4(0.f, 0.f, 0.f, 0.f);
            if (!LITE) b4 = *reinterpret_cast<const float4 *>(&sm.B[order][i][n0]);
            const float2 b2[2] = {make_float2(b4.x, b4.y), make_float2(b4.z, b4.w)};
            const float dl = in.x * kLog2e;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float2 x = __fmul2_rn(make_float2(dl, dl), A[k]);
                a[i][k] = make_float2(ex2(x.x), ex2(x.y));
                if (!LITE) h[i + 1][k] = __ffma2_rn(a[i][k], h[i][k], __fmul2_rn(make_float2(in.y, in.y), b2[k]));
            }
        }
        float2 tile_dA[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int i = TT - 1; i >= 0; --i) {
            const float4 in = sm.in[i][ch];
            const float2 dc = make_float2(in.z, in.z);
            const float4 c4 = *reinterpret_cast<const float4 *>(&sm.C[order][i][n0]);
            const float2 c2[2] = {make_float2(c4.x, c4.y), make_float2(c4.z, c4.w)};
            if (LITE) {
#pragma unroll
                for (int k = 0; k < 2; ++k) ge[k] = __fmul2_rn(__ffma2_rn(dc, c2[k], ge[k]), a[i][k]);
                continue;
            }
            const float4 b4 = *reinterpret_cast<const float4 *>(&sm.B[order][i][n0]);
            const float2 b2[2] = {make_float2(b4.x, b4.y), make_float2(b4.z, b4.w)};
            const float2 xu = make_float2(in.y, in.y), d2 = make_float2(in.x, in.x);
            float2 gB[2], gC[2], dsu2, kd2, core2;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float2 e = __ffma2_rn(dc, c2[k], ge[k]);
                gB[k] = __fmul2_rn(e, xu);
                gC[k] = __fmul2_rn(dc, h[i + 1][k]);
                ge[k] = __fmul2_rn(e, a[i][k]);
                const float2 kept = __fmul2_rn(ge[k], h[i][k]);
                tile_dA[k] = __ffma2_rn(kept, d2, tile_dA[k]);
                dsu2 = k == 0 ? __fmul2_rn(e, b2[0]) : __ffma2_rn(e, b2[1], dsu2);
                core2 = k == 0 ? __fmul2_rn(c2[0], h[i + 1][0]) : __ffma2_rn(c2[1], h[i + 1][1], core2);
                kd2 = k == 0 ? __fmul2_rn(kept, A[0]) : __ffma2_rn(kept, A[1], kd2);
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
            // dsu, kd and core over the channel's lanes: lane bits 1 and 0 choose which one is kept
            const float dsu = dsu2.x + dsu2.y, kd = kd2.x + kd2.y, core = core2.x + core2.y;
            const bool up2 = lane & 2, up1 = lane & 1;
            const float2 got = shfl2(up2 ? make_float2(dsu, kd) : make_float2(core, 0.f), 2);
            const float2 x = __fadd2_rn(up2 ? make_float2(core, 0.f) : make_float2(dsu, kd), got);
            float r = (up1 ? x.y : x.x) + __shfl_xor_sync(kFullMask, up1 ? x.x : x.y, 1);
#pragma unroll
            for (int m = 4; m < LPC; m <<= 1) r += __shfl_xor_sync(kFullMask, r, m);
            if (lane % LPC < 3) reinterpret_cast<float *>(&sm.out[i][ch])[lane % LPC] = r;
        }
        if (!LITE) {
            add_comp(dA[0], dA_lost[0], tile_dA[0].x);
            add_comp(dA[1], dA_lost[1], tile_dA[0].y);
            add_comp(dA[2], dA_lost[2], tile_dA[1].x);
            add_comp(dA[3], dA_lost[3], tile_dA[1].y);
        }
        __syncthreads();
        if (LITE) continue;
        // each staged element's gradients
        if (t < p.T) {
            float uu[V], zz[V], yy[V], du[V], ddt[V], dz[V];
            cu.get(uu);
            cz.get(zz);
            cy.get(yy);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float4 o = sm.out[ts][cv + v], in = sm.in[ts][cv + v];
                const bool on = t < L;
                du[v] = on ? fmaf(o.x, in.x, D[v] * in.z) : 0.f;
                ddt[v] = on ? fmaf(o.x, uu[v], o.y) * in.w : 0.f;
                dz[v] = on ? yy[v] * fmaf(D[v], uu[v], o.z) * dsilu_hw(zz[v]) : 0.f;
                sum_D[v] += on ? in.z * uu[v] : 0.f;
                sum_b[v] += ddt[v];
            }
            const size_t at = row + (size_t)t * p.Cn;
            store_channels<T, V>(static_cast<T *>(p.du) + at, nv, VEC, du);
            store_channels<T, V>(static_cast<T *>(p.ddt) + at, nv, VEC, ddt);
            if (p.dz != nullptr) store_channels<T, V>(static_cast<T *>(p.dz) + at, nv, VEC, dz);
        }
        // the CTA's dB, dC of the tile: over its warps in ascending order
        for (int e = tid; e < TT * 2 * NP; e += kScanThreads) {
            const int i = e / (2 * NP), n = e % (2 * NP), tb = tile * TT + i;
            if (tb >= p.T || n % NP >= p.N) continue;
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kScanWarps; ++w) s += sm.bc[w][i][n];
            p.part_bc[((((size_t)q.blk * p.Bn + q.b) * p.T + tb) * p.G + q.g) * (2 * p.N) + (n / NP) * p.N + n % NP] = s;
        }
        __syncthreads();
    }
    if (LITE) {
        if (live) store_mine(p.seg_state + (size_t)q.seg * p.Bn * p.Cn * p.N + state_row, ge);
        float *s = reinterpret_cast<float *>(sm.out);
#pragma unroll
        for (int v = 0; v < V; ++v) s[ts * CH + cv + v] = sum_d[v];
        __syncthreads();
        if (tid < q.nc) {
            float x = 0.f;
            for (int i = 0; i < TT; ++i) x += s[i * CH + tid];
            p.seg_sum[((size_t)q.seg * p.Bn + q.b) * p.Cn + q.c0 + tid] = x;
        }
        return;
    }
    if (p.segs == 1 && p.dh0 != nullptr && live) store_mine(p.dh0 + state_row, ge);
    float *part = p.part_c + ((size_t)q.seg * p.Bn + q.b) * (p.N + 2) * p.Cn;
    if (live) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int n = n0 + (k ^ order);
            if (n < p.N) part[(size_t)n * p.Cn + c] = dA[k] + dA_lost[k];
        }
    }
    float *s = reinterpret_cast<float *>(sm.out);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        s[ts * CH + cv + v] = sum_D[v];
        s[(TT + ts) * CH + cv + v] = sum_b[v];
    }
    __syncthreads();
    for (int e = tid; e < 2 * CH; e += kScanThreads) {
        const int which = e / CH, cc = e % CH;
        if (cc >= q.nc) continue;
        float x = 0.f;
        for (int i = 0; i < TT; ++i) x += s[(which * TT + i) * CH + cc];
        part[(size_t)(p.N + which) * p.Cn + q.c0 + cc] = x;
    }
}

// dB, dC: over the channel blocks of their group, in ascending order.
template <typename T>
__global__ void __launch_bounds__(256) scan_reduce_bc_kernel(ScanParams p, int blocks) {
    const size_t n = (size_t)p.Bn * p.T * p.G * 2 * p.N, i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    float s = 0.f;
    for (int k = 0; k < blocks; ++k) s += p.part_bc[(size_t)k * n + i];
    const size_t row = i / (2 * p.N);
    const int m = (int)(i % (2 * p.N));
    if (m < p.N) static_cast<T *>(p.dB)[row * p.N + m] = from_f32<T>(s);
    else static_cast<T *>(p.dC)[row * p.N + m - p.N] = from_f32<T>(s);
}

// dA_log, dD, ddt_bias: over the segments and batch rows.
__global__ void __launch_bounds__(256) scan_reduce_c_kernel(ScanParams p) {
    const size_t n = (size_t)(p.N + 2) * p.Cn, i = (size_t)blockIdx.x * 32 + threadIdx.x;
    const double s = slice_sum(p.part_c, p.segs * p.Bn, n);
    if (threadIdx.x >= 32 || i >= n) return;
    const int m = (int)(i / p.Cn), c = (int)(i % p.Cn);
    if (m < p.N) {
        const size_t o = (size_t)c * p.N + m;
        p.dA_log[o] = (float)(s * -(double)expf(p.A_log[o]));
    } else if (m == p.N) {
        if (p.dD != nullptr) p.dD[c] = (float)s;
    } else if (p.ddt_bias != nullptr) {
        p.ddt_bias[c] = (float)s;
    }
}

namespace {

template <int LPC, typename T, bool VEC, bool LITE>
cudaError_t scan_bwd_one(const ScanParams &p, cudaStream_t s) {
    const cudaError_t e = cudaFuncSetAttribute(scan_bwd_kernel<LPC, T, VEC, LITE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)sizeof(BwdSmem<LPC>));
    if (e != cudaSuccess) return e;
    const dim3 grid(p.Bn * p.G * scan_blocks(p.Cn, p.G, p.N), p.segs);
    const char *name = LITE ? "scan_bwd_ends" : "scan_bwd";
    timing_mark(name, 0, s);
    scan_bwd_kernel<LPC, T, VEC, LITE><<<grid, kScanThreads, sizeof(BwdSmem<LPC>), s>>>(p);
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
    timing_mark("scan_reduce", 0, s);
    scan_reduce_bc_kernel<T><<<(unsigned)((n + 255) / 256), 256, 0, s>>>(p, scan_blocks(p.Cn, p.G, p.N));
    timing_mark("scan_reduce", 1, s);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    timing_mark("scan_reduce", 0, s);
    scan_reduce_c_kernel<<<(unsigned)((m + 31) / 32), 256, 0, s>>>(p);
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

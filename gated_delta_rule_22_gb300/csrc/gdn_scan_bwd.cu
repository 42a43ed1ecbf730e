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
// back over them. Eight sums over the channels of a warp (dB, dC of four states) and three over a
// channel's lanes are reduced by exchanging halves, so that each exchange also shortens what is left.
#include "gdn_scan.cuh"

namespace gdn {

namespace {

// Sums eight values over the lanes of a warp that hold the same states of different channels (the
// lanes l, l + LPC, l + 2 LPC, ...): afterwards v[0 .. LPC / 4 - 1] hold the full sums of the value
// indices (l / LPC) * (LPC / 4) + i in bit order: halving from the top, as below.
template <int LPC>
__device__ __forceinline__ void channel_sum8(float (&v)[8], int lane) {
    int n = 8;
#pragma unroll
    for (int m = 16; m >= LPC; m >>= 1) {
        const bool upper = (lane & m) != 0;
        n >>= 1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i < n) {
                const float send = upper ? v[i] : v[i + n];
                const float keep = upper ? v[i + n] : v[i];
                v[i] = keep + __shfl_xor_sync(kFullMask, send, m);
            }
        }
    }
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
    float4 in[kScanTile][G::CH];                  // d, d u, dcore
    float B[kScanTile][G::NP], C[kScanTile][G::NP];
    float4 out[kScanTile][G::CH];                 // dsu, sum kept A, C . h
    float bc[kScanWarps][kScanTile][2 * G::NP];   // a warp's dB, dC
};

}  // namespace

// LITE: the segment's start adjoint from a zero end and its sum of d, nothing else.
template <int LPC, typename T, bool LITE>
__global__ void __launch_bounds__(kScanThreads, 1) scan_bwd_kernel(ScanParams p, bool vec) {
    using G = ScanGeo<LPC>;
    constexpr int CH = G::CH, NP = G::NP, V = G::V, KB = G::KB, TT = kScanTile;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    BwdSmem<LPC> &sm = *reinterpret_cast<BwdSmem<LPC> *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const ScanPlace q = scan_place<LPC>(p);
    if (q.first >= q.last) return;
    const int L = row_length(p.lens, q.b, p.T);
    const int ts = tid >> 4, cv = (tid & 15) * V, nv = q.nc - cv;
    const int ch = warp * G::CPW + lane / LPC, n0 = 4 * (lane % LPC);
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
    float A[4], ge[4] = {0.f, 0.f, 0.f, 0.f}, dA[4] = {0.f, 0.f, 0.f, 0.f}, dA_lost[4] = {0.f, 0.f, 0.f, 0.f};
    float D[V], bias[V], sum_d[V], sum_D[V], sum_b[V];
#pragma unroll
    for (int k = 0; k < 4; ++k) A[k] = n0 + k < p.N ? -expf(p.A_log[(size_t)c * p.N + n0 + k]) : 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        D[v] = p.D != nullptr && v < nv ? p.D[q.c0 + cv + v] : 0.f;
        bias[v] = p.dt_bias != nullptr && v < nv ? p.dt_bias[q.c0 + cv + v] : 0.f;
        sum_d[v] = sum_D[v] = sum_b[v] = 0.f;
    }
    const size_t state_row = ((size_t)q.b * p.Cn + c) * p.N;
    if (!LITE && live) {
        if (p.segs > 1) load_states(p.seg_state + (size_t)q.seg * p.Bn * p.Cn * p.N + state_row, n0, p.N, ge);
        else if (p.dh_T != nullptr) load_states(p.dh_T + state_row, n0, p.N, ge);
    }
    float ru[V], rd[V], rz[V], ry[V], rB[KB], rC[KB], rh[4];
    auto fetch = [&](int tile) {
        const int t = tile * TT + ts, n = t < L ? nv : 0;
        if (!LITE) load_channels<T, V>(u + (size_t)t * p.ldu, n, vec, ru);
        load_channels<T, V>(dt + (size_t)t * p.lddt, n, vec, rd);
        if (p.z != nullptr) load_channels<T, V>(z + (size_t)t * p.ldz, n, vec, rz);
        load_channels<T, V>(dy + (size_t)t * p.Cn, n, vec, ry);
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            const int e = tid + kScanThreads * k, tb = tile * TT + e / NP, n1 = e % NP;
            const bool ok = tb < L && n1 < p.N;
            if (!LITE) rB[k] = ok ? to_f32(Bm[(size_t)tb * p.ldB + n1]) : 0.f;
            rC[k] = ok ? to_f32(Cm[(size_t)tb * p.ldC + n1]) : 0.f;
        }
        if (!LITE) load_states(p.ckpt + (((size_t)q.b * tiles + tile) * p.Cn + c) * p.N, n0, p.N, rh);
    };
    fetch(q.last - 1);
    for (int tile = q.last - 1; tile >= q.first; --tile) {
        const int t = tile * TT + ts;
        float cu[V], cz[V], cy[V], cd[V], cs[V], hs[4];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float raw = rd[v] + bias[v];
            const float d = t < L ? softplus_full(raw) : 0.f;
            cu[v] = LITE ? 0.f : ru[v];
            cz[v] = p.z != nullptr ? rz[v] : 0.f;
            cy[v] = ry[v];
            cd[v] = d;
            cs[v] = raw;
            if (LITE) sum_d[v] += d;
            sm.in[ts][cv + v] = make_float4(d, LITE ? 0.f : d * ru[v], p.z != nullptr ? ry[v] * silu_hw(rz[v]) : ry[v], 0.f);
        }
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            const int e = tid + kScanThreads * k;
            if (!LITE) sm.B[e / NP][e % NP] = rB[k];
            sm.C[e / NP][e % NP] = rC[k];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) hs[k] = LITE ? 0.f : rh[k];
        __syncthreads();
        if (tile > q.first) fetch(tile - 1);
        float a[TT][4], h[TT + 1][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) h[0][k] = hs[k];
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            const float4 in = sm.in[i][ch];
            float4 b4 = make_float4(0.f, 0.f, 0.f, 0.f);
            if (!LITE) b4 = *reinterpret_cast<const float4 *>(&sm.B[i][n0]);
            const float bb[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                a[i][k] = ex2(in.x * (A[k] * kLog2e));
                if (!LITE) h[i + 1][k] = fmaf(a[i][k], h[i][k], in.y * bb[k]);
            }
        }
        float tile_dA[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = TT - 1; i >= 0; --i) {
            const float4 in = sm.in[i][ch];
            const float4 c4 = *reinterpret_cast<const float4 *>(&sm.C[i][n0]);
            const float cc[4] = {c4.x, c4.y, c4.z, c4.w};
            if (LITE) {
#pragma unroll
                for (int k = 0; k < 4; ++k) ge[k] = fmaf(in.z, cc[k], ge[k]) * a[i][k];
                continue;
            }
            const float4 b4 = *reinterpret_cast<const float4 *>(&sm.B[i][n0]);
            const float bb[4] = {b4.x, b4.y, b4.z, b4.w};
            float v8[8], dsu = 0.f, kd = 0.f, core = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float e = fmaf(in.z, cc[k], ge[k]);
                v8[k] = e * in.y;
                v8[4 + k] = in.z * h[i + 1][k];
                dsu = fmaf(e, bb[k], dsu);
                core = fmaf(cc[k], h[i + 1][k], core);
                ge[k] = e * a[i][k];
                const float kept = ge[k] * h[i][k];
                kd = fmaf(kept, A[k], kd);
                tile_dA[k] = fmaf(kept, in.x, tile_dA[k]);
            }
            channel_sum8<LPC>(v8, lane);
            // where the halving left them: value index from the lane bits, from the top
            if constexpr (LPC == 4) {
                const int idx = (lane >> 4 & 1) * 4 + (lane >> 3 & 1) * 2 + (lane >> 2 & 1);
                sm.bc[warp][i][(idx >> 2) * NP + n0 + (idx & 3)] = v8[0];
            } else if constexpr (LPC == 8) {
                const int idx = (lane >> 4 & 1) * 4 + (lane >> 3 & 1) * 2;
                sm.bc[warp][i][(idx >> 2) * NP + n0 + (idx & 3)] = v8[0];
                sm.bc[warp][i][(idx >> 2) * NP + n0 + (idx & 3) + 1] = v8[1];
            } else {
                const int idx = (lane >> 4 & 1) * 4;
                *reinterpret_cast<float4 *>(&sm.bc[warp][i][(idx >> 2) * NP + n0]) = make_float4(v8[0], v8[1], v8[2], v8[3]);
            }
            // dsu, kd and core over the channel's lanes: lane bits 1 and 0 choose which one is kept
            const bool up2 = lane & 2, up1 = lane & 1;
            const float s0 = __shfl_xor_sync(kFullMask, up2 ? dsu : core, 2), s1 = __shfl_xor_sync(kFullMask, up2 ? kd : 0.f, 2);
            float x0 = (up2 ? core : dsu) + s0, x1 = (up2 ? 0.f : kd) + s1;
            float r = (up1 ? x1 : x0) + __shfl_xor_sync(kFullMask, up1 ? x0 : x1, 1);
#pragma unroll
            for (int m = 4; m < LPC; m <<= 1) r += __shfl_xor_sync(kFullMask, r, m);
            if (lane % LPC < 3) reinterpret_cast<float *>(&sm.out[i][ch])[lane % LPC] = r;
        }
        if (!LITE) {
#pragma unroll
            for (int k = 0; k < 4; ++k) add_comp(dA[k], dA_lost[k], tile_dA[k]);
        }
        __syncthreads();
        if (LITE) continue;
        // each staged element's gradients
        if (t < p.T) {
            float du[V], ddt[V], dz[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float4 o = sm.out[ts][cv + v];      // dsu, sum kept A, C . h
                const float dcore = sm.in[ts][cv + v].z;
                const bool on = t < L;
                du[v] = on ? fmaf(o.x, cd[v], D[v] * dcore) : 0.f;
                ddt[v] = on ? fmaf(o.x, cu[v], o.y) * sigmoid_hw(cs[v]) : 0.f;
                dz[v] = on ? cy[v] * fmaf(D[v], cu[v], o.z) * dsilu_hw(cz[v]) : 0.f;
                sum_D[v] += on ? dcore * cu[v] : 0.f;
                sum_b[v] += ddt[v];
            }
            const size_t at = row + (size_t)t * p.Cn;
            store_channels<T, V>(static_cast<T *>(p.du) + at, nv, vec, du);
            store_channels<T, V>(static_cast<T *>(p.ddt) + at, nv, vec, ddt);
            if (p.dz != nullptr) store_channels<T, V>(static_cast<T *>(p.dz) + at, nv, vec, dz);
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
        if (live) store_states(p.seg_state + (size_t)q.seg * p.Bn * p.Cn * p.N + state_row, n0, p.N, ge);
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
    if (p.segs == 1 && p.dh0 != nullptr && live) store_states(p.dh0 + state_row, n0, p.N, ge);
    float *part = p.part_c + ((size_t)q.seg * p.Bn + q.b) * (p.N + 2) * p.Cn;
    if (live) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (n0 + k < p.N) part[(size_t)(n0 + k) * p.Cn + c] = dA[k] + dA_lost[k];
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

template <int LPC, typename T, bool LITE>
cudaError_t scan_bwd_one(const ScanParams &p, cudaStream_t s) {
    const cudaError_t e = cudaFuncSetAttribute(scan_bwd_kernel<LPC, T, LITE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)sizeof(BwdSmem<LPC>));
    if (e != cudaSuccess) return e;
    const dim3 grid(p.Bn * p.G * scan_blocks(p.Cn, p.G, p.N), p.segs);
    const char *name = LITE ? "scan_bwd_ends" : "scan_bwd";
    timing_mark(name, 0, s);
    scan_bwd_kernel<LPC, T, LITE><<<grid, kScanThreads, sizeof(BwdSmem<LPC>), s>>>(p, scan_vec<T>(p, ScanGeo<LPC>::V));
    timing_mark(name, 1, s);
    return cudaGetLastError();
}

template <int LPC, typename T>
cudaError_t scan_bwd_launch(const ScanParams &p, cudaStream_t s) {
    cudaError_t e;
    if (p.segs > 1) {
        if ((e = scan_bwd_one<LPC, T, true>(p, s)) != cudaSuccess) return e;
        if ((e = launch_scan_combine(p, p.dh_T, p.dh0, true, s)) != cudaSuccess) return e;
    }
    if ((e = scan_bwd_one<LPC, T, false>(p, s)) != cudaSuccess) return e;
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

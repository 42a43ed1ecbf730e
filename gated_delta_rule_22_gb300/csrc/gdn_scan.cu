// gdn_scan.cu -- selective state space scan, forward: prompts, the step of a single token, and the
// split of long sequences.
//
//     d = softplus(dt + dt_bias),  A = -exp(A_log)
//     h_t = exp(d A) h_{t-1} + d u B_t,   y_t = (C_t . h_t + D u) silu(z)
//
// Each state and step costs one exp2 and four float32 operations (d A log2 e, (d u) B, the update,
// the product with C), each channel and step 2 to 4 elements of memory traffic: with 16 states the
// exponentials bind, not the memory.
#include "gdn_scan.cuh"

namespace gdn {

// LITE: the segment's end state from a zero start and its sum of d, nothing else (first pass over a
// split sequence).
//
// Eight warps hold the states and do nothing but the recurrence; four more stage the tiles (loads a
// tile ahead, softplus) and finish the outputs. With as few channels as a layer has there are about
// two state warps per scheduler, which then have the helpers' work to hide their latencies, and no
// phases of their own that leave the recurrence idle. Two tiles are in flight; named barriers full[2]
// (staged) and done[2] (walked) hand them over.
template <int LPC, typename T, bool VEC, bool LITE>
__global__ void __launch_bounds__(kScanThreads + kScanHelpers, LITE ? 3 : 2) scan_fwd_kernel(ScanParams p) {
    using G = ScanGeo<LPC>;
    constexpr int CH = G::CH, NP = G::NP, V = G::V, TT = kScanTile, ALL = kScanThreads + kScanHelpers;
    constexpr int kFull = 1, kDone = 3;
    __shared__ __align__(16) float2 sdx[2][TT][CH];   // d, d u
    __shared__ __align__(16) float sB[2][TT][NP], sC[2][TT][NP];
    __shared__ float score[2][TT][G::SP];
    __shared__ __align__(16) T su[2][TT][CH], sz[2][TT][CH];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const ScanPlace q = scan_place<LPC>(p);
    if (q.first >= q.last) return;
    const int L = row_length(p.lens, q.b, p.T);
    if (tid >= kScanThreads) {
        constexpr int KB = NP * TT / kScanHelpers, PASS = TT * CH / V / kScanHelpers;
        // staged elements: steps ts and ts + 8 of a tile, V channels from cv
        const int h = tid - kScanThreads, ts = h >> 4, cv = (h & 15) * V, nv = q.nc - cv;
        const T *u = static_cast<const T *>(p.u) + (size_t)q.b * p.T * p.ldu + q.c0 + cv;
        const T *dt = static_cast<const T *>(p.dt) + (size_t)q.b * p.T * p.lddt + q.c0 + cv;
        const T *z = static_cast<const T *>(p.z) + (size_t)q.b * p.T * p.ldz + q.c0 + cv;
        T *y = static_cast<T *>(p.y) + (size_t)q.b * p.T * p.Cn + q.c0 + cv;
        const T *Bm = static_cast<const T *>(p.B) + (size_t)q.b * p.T * p.ldB + q.g * p.N;
        const T *Cm = static_cast<const T *>(p.C) + (size_t)q.b * p.T * p.ldC + q.g * p.N;
        Staged<T, V, VEC> ru[PASS], rd[PASS], rz[PASS];
        T rB[KB], rC[KB];
        auto fetch = [&](int tile) {
#pragma unroll
            for (int i = 0; i < PASS; ++i) {
                const int t = tile * TT + ts + 8 * i, n = t < L ? nv : 0;
                ru[i].load(u + (size_t)t * p.ldu, n);
                rd[i].load(dt + (size_t)t * p.lddt, n);
                if (!LITE && p.z != nullptr) rz[i].load(z + (size_t)t * p.ldz, n);
            }
#pragma unroll
            for (int k = 0; k < KB; ++k) {
                const int e = h + kScanHelpers * k, tb = tile * TT + e / NP, n1 = e % NP;
                const bool ok = tb < L && n1 < p.N;
                rB[k] = rC[k] = from_f32<T>(0.f);
                if (ok) rB[k] = Bm[(size_t)tb * p.ldB + n1];
                if (!LITE && ok) rC[k] = Cm[(size_t)tb * p.ldC + n1];
            }
        };
        float D[V], bias[V], sum_d[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            D[v] = p.D != nullptr && v < nv ? p.D[q.c0 + cv + v] : 0.f;
            bias[v] = p.dt_bias != nullptr && v < nv ? p.dt_bias[q.c0 + cv + v] : 0.f;
            sum_d[v] = 0.f;
        }
        auto stage = [&](int tile) {
            const int buf = tile & 1;
#pragma unroll
            for (int i = 0; i < PASS; ++i) {
                const int st = ts + 8 * i, t = tile * TT + st;
                float uu[V], dd[V];
                ru[i].get(uu);
                rd[i].get(dd);
                if constexpr (V == 1) {
                    dd[0] = softplus_full(dd[0] + bias[0]);
                } else {
#pragma unroll
                    for (int v = 0; v < V; v += 2) {
                        const float2 d = softplus2_full(make_float2(dd[v] + bias[v], dd[v + 1] + bias[v + 1]));
                        dd[v] = d.x;
                        dd[v + 1] = d.y;
                    }
                }
                if (t >= L)
#pragma unroll
                    for (int v = 0; v < V; ++v) dd[v] = 0.f;
                if constexpr (V == 1) {
                    sdx[buf][st][cv] = make_float2(dd[0], dd[0] * uu[0]);
                } else {
#pragma unroll
                    for (int v = 0; v < V; v += 2)
                        *reinterpret_cast<float4 *>(&sdx[buf][st][cv + v]) = make_float4(dd[v], dd[v] * uu[v], dd[v + 1], dd[v + 1] * uu[v + 1]);
                }
                if (LITE) {
#pragma unroll
                    for (int v = 0; v < V; ++v) sum_d[v] += dd[v];
                } else {
                    ru[i].keep(&su[buf][st][cv]);
                    if (p.z != nullptr) rz[i].keep(&sz[buf][st][cv]);
                }
            }
#pragma unroll
            for (int k = 0; k < KB; ++k) {
                const int e = h + kScanHelpers * k;
                sB[buf][e / NP][e % NP] = to_f32(rB[k]);
                if (!LITE) sC[buf][e / NP][e % NP] = to_f32(rC[k]);
            }
            if (tile + 1 < q.last) fetch(tile + 1);
            named_bar_arrive(kFull + buf, ALL);
        };
        fetch(q.first);
        stage(q.first);
        if (q.first + 1 < q.last) stage(q.first + 1);
        for (int tile = q.first; tile < q.last; ++tile) {
            const int buf = tile & 1;
            named_bar_sync(kDone + buf, ALL);
            if (!LITE) {
#pragma unroll
                for (int i = 0; i < PASS; ++i) {
                    const int st = ts + 8 * i, t = tile * TT + st;
                    if (t >= p.T) continue;
                    float o[V], uu[V], zz[V];
                    load_vec<T, V>(&su[buf][st][cv], uu);
#pragma unroll
                    for (int v = 0; v < V; ++v) o[v] = fmaf(D[v], uu[v], score[buf][st][cv + v]);
                    if (p.z != nullptr) {
                        load_vec<T, V>(&sz[buf][st][cv], zz);
#pragma unroll
                        for (int v = 0; v < V; ++v) o[v] *= silu_hw(zz[v]);
                    }
                    if (t >= L)
#pragma unroll
                        for (int v = 0; v < V; ++v) o[v] = 0.f;
                    store_channels<T, V>(y + (size_t)t * p.Cn, nv, VEC, o);
                }
            }
            if (tile + 2 < q.last) stage(tile + 2);
        }
        if (LITE) {
            // the sum of d over the segment: over a thread's tiles, then over its eight steps of a tile
#pragma unroll
            for (int v = 0; v < V; ++v) score[0][ts][cv + v] = sum_d[v];
            named_bar_sync(kDone + 2, kScanHelpers);
            for (int cc = h; cc < q.nc; cc += kScanHelpers) {
                float a = 0.f;
                for (int i = 0; i < 8; ++i) a += score[0][i][cc];
                p.seg_sum[((size_t)q.seg * p.Bn + q.b) * p.Cn + q.c0 + cc] = a;
            }
        }
        return;
    }
    // this lane's states: channel ch, states n0 .. n0 + 3
    const int ch = warp * G::CPW + lane / LPC, n0 = 4 * (lane % LPC);
    const bool live = ch < q.nc;
    const int c = q.c0 + (live ? ch : 0);
    float2 A2[2], h[2];
    {
        float e[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) e[k] = n0 + k < p.N ? -expf(p.A_log[(size_t)c * p.N + n0 + k]) * kLog2e : 0.f;
        A2[0] = make_float2(e[0], e[1]);
        A2[1] = make_float2(e[2], e[3]);
    }
    const size_t state_row = ((size_t)q.b * p.Cn + c) * p.N;
    {
        float e[4] = {0.f, 0.f, 0.f, 0.f};
        if (!LITE && live) {
            if (p.segs > 1) load_states(p.seg_state + (size_t)q.seg * p.Bn * p.Cn * p.N + state_row, n0, p.N, e);
            else if (p.h0 != nullptr) load_states(p.h0 + state_row, n0, p.N, e);
        }
        h[0] = make_float2(e[0], e[1]);
        h[1] = make_float2(e[2], e[3]);
    }
    const int tiles = (p.T + TT - 1) / TT;
    for (int tile = q.first; tile < q.last; ++tile) {
        const int buf = tile & 1;
        if (!LITE && p.ckpt != nullptr && live) {
            const float o[4] = {h[0].x, h[0].y, h[1].x, h[1].y};
            store_states(p.ckpt + (((size_t)q.b * tiles + tile) * p.Cn + c) * p.N, n0, p.N, o);
        }
        named_bar_sync(kFull + buf, ALL);
        // four steps at a time: what does not depend on the state (decays, d u B) is formed for the next
        // four before the chain of the present four, whose only latency is one multiply-add per step
        struct Group {
            float2 a[4][2], x[4][2], c[4][2];
        };
        auto prepare = [&](int i0, Group &o) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 dx = sdx[buf][i0 + i][ch];
                const float4 b4 = *reinterpret_cast<const float4 *>(&sB[buf][i0 + i][n0]);
                const float2 b2[2] = {make_float2(b4.x, b4.y), make_float2(b4.z, b4.w)};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    o.a[i][k] = decay2(dx.x, A2[k]);
                    o.x[i][k] = __fmul2_rn(make_float2(dx.y, dx.y), b2[k]);
                }
                if (!LITE) {
                    const float4 c4 = *reinterpret_cast<const float4 *>(&sC[buf][i0 + i][n0]);
                    o.c[i][0] = make_float2(c4.x, c4.y);
                    o.c[i][1] = make_float2(c4.z, c4.w);
                }
            }
        };
        Group now, then;
        prepare(0, now);
#pragma unroll
        for (int i0 = 0; i0 < TT; i0 += 4) {
            if (i0 + 4 < TT) prepare(i0 + 4, then);
            float core[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float2 sum;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    h[k] = __ffma2_rn(now.a[i][k], h[k], now.x[i][k]);
                    if (!LITE) sum = k == 0 ? __fmul2_rn(now.c[i][0], h[0]) : __ffma2_rn(now.c[i][1], h[1], sum);
                }
                if (!LITE) core[i] = sum.x + sum.y;
            }
            if (!LITE) {
                const float r = lane_sum4<LPC>(core, lane);
                if (lane % LPC < 4) score[buf][i0 + (lane & 3)][ch] = r;
            }
            now = then;
        }
        named_bar_arrive(kDone + buf, ALL);
    }
    const float out[4] = {h[0].x, h[0].y, h[1].x, h[1].y};
    if (LITE) {
        if (live) store_states(p.seg_state + (size_t)q.seg * p.Bn * p.Cn * p.N + state_row, n0, p.N, out);
    } else if (p.h_T != nullptr && live && q.seg == p.segs - 1) {
        store_states(p.h_T + state_row, n0, p.N, out);
    }
}

// One step (T = 1): a streaming pass over the states, bound by their bytes (read and written once). LPC
// lanes take one channel of four batch rows, so that A is formed once for four states; lane r forms
// row r's d and finishes its output. h_T may be h0.
template <int LPC, typename T>
__global__ void __launch_bounds__(256) scan_step_kernel(ScanParams p, bool vec) {
    const int lane = threadIdx.x & 31, j = threadIdx.x % LPC, n0 = 4 * j, mine = j & 3, base = lane & ~(LPC - 1);
    const int c = (int)((blockIdx.x * 256 + threadIdx.x) / LPC), b0 = blockIdx.y * 4;
    const bool live = c < p.Cn;
    const int cc = live ? c : 0, g = p.G == 1 ? 0 : cc / (p.Cn / p.G);
    float h[4][4], Bv[4][4], Cv[4][4];
    bool on[4];
    const size_t state = (size_t)p.Cn * p.N, first = (size_t)b0 * state + (size_t)cc * p.N + n0;
    const T *Bm = static_cast<const T *>(p.B) + (size_t)b0 * p.ldB + g * p.N + n0;
    const T *Cm = static_cast<const T *>(p.C) + (size_t)b0 * p.ldC + g * p.N + n0;
    if (vec && b0 + 4 <= p.Bn && p.lens == nullptr && p.h0 != nullptr && (p.N & 3) == 0 && n0 < p.N) {
        // four whole rows: all loads in flight at once
        Raw<T, 4> rb[4], rc[4];
        float4 rh[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) rh[r] = __ldcs(reinterpret_cast<const float4 *>(p.h0 + first + r * state));
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            rb[r] = load_raw<T, 4>(Bm + r * p.ldB);
            rc[r] = load_raw<T, 4>(Cm + r * p.ldC);
            on[r] = live;
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            unpack<T, 4>(rb[r], Bv[r]);
            unpack<T, 4>(rc[r], Cv[r]);
            h[r][0] = rh[r].x; h[r][1] = rh[r].y; h[r][2] = rh[r].z; h[r][3] = rh[r].w;
        }
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const bool row = live && b0 + r < p.Bn;
            on[r] = row && row_length(p.lens, b0 + r, 1) == 1;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const bool in = n0 + k < p.N;
                h[r][k] = Bv[r][k] = Cv[r][k] = 0.f;
                if (row && in && p.h0 != nullptr) h[r][k] = p.h0[first + r * state + k];
                if (on[r] && in) {
                    Bv[r][k] = to_f32(Bm[r * p.ldB + k]);
                    Cv[r][k] = to_f32(Cm[r * p.ldC + k]);
                }
            }
        }
    }
    const int bm = b0 + mine;
    const bool on_m = live && bm < p.Bn && row_length(p.lens, bm, 1) == 1;
    float u = 0.f, z = 0.f, d = 0.f, A2[4];
    if (on_m) {
        u = to_f32(static_cast<const T *>(p.u)[(size_t)bm * p.ldu + cc]);
        if (p.z != nullptr) z = to_f32(static_cast<const T *>(p.z)[(size_t)bm * p.ldz + cc]);
        d = softplus_full(to_f32(static_cast<const T *>(p.dt)[(size_t)bm * p.lddt + cc]) + (p.dt_bias != nullptr ? p.dt_bias[cc] : 0.f));
    }
    load_states(p.A_log + (size_t)cc * p.N, n0, p.N, A2);
#pragma unroll
    for (int k = 0; k < 4; ++k) A2[k] = n0 + k < p.N ? -expf(A2[k]) * kLog2e : 0.f;
    float core[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const float dr = __shfl_sync(kFullMask, d, base + r), xu = __shfl_sync(kFullMask, d * u, base + r);
        core[r] = 0.f;
        if (!on[r]) continue;                          // the same for all lanes of a channel
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            h[r][k] = fmaf(ex2(fmaf(A2[k], dr, kExp2Centre)), h[r][k], xu * Bv[r][k]);
            core[r] = fmaf(Cv[r][k], h[r][k], core[r]);
        }
    }
    const float sum = lane_sum4<LPC>(core, lane);
    if (!live) return;
    if (j < 4 && bm < p.Bn) {
        float y = 0.f;
        if (on_m) {
            y = sum + (p.D != nullptr ? p.D[cc] * u : 0.f);
            if (p.z != nullptr) y *= silu_hw(z);
        }
        static_cast<T *>(p.y)[(size_t)bm * p.Cn + cc] = from_f32<T>(y);
    }
    if (p.h_T == nullptr) return;
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (b0 + r < p.Bn) store_states(p.h_T + first - n0 + r * state, n0, p.N, h[r]);
}

__global__ void __launch_bounds__(256) scan_combine_kernel(ScanParams p, const float *start, float *out, bool reverse) {
    const size_t n = (size_t)p.Bn * p.Cn * p.N, i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const size_t bc = i / p.N;
    const float A2 = -expf(p.A_log[(bc % p.Cn) * p.N + i % p.N]) * kLog2e;
    float X = start != nullptr ? start[i] : 0.f;
    constexpr int U = 8;                               // segments loaded together
    for (int k0 = 0; k0 < p.segs; k0 += U) {
        float own[U], decay[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int s = reverse ? p.segs - 1 - k0 - k : k0 + k;
            if (k0 + k >= p.segs) break;
            own[k] = p.seg_state[(size_t)s * n + i];
            decay[k] = p.seg_sum[(size_t)s * p.Bn * p.Cn + bc];
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int s = reverse ? p.segs - 1 - k0 - k : k0 + k;
            if (k0 + k >= p.segs) break;
            p.seg_state[(size_t)s * n + i] = X;
            X = fmaf(ex2(A2 * decay[k]), X, own[k]);
        }
    }
    if (out != nullptr) out[i] = X;
}

cudaError_t launch_scan_combine(const ScanParams &p, const float *start, float *out, bool reverse, cudaStream_t s) {
    const size_t n = (size_t)p.Bn * p.Cn * p.N;
    timing_mark("scan_combine", 0, s);
    scan_combine_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(p, start, out, reverse);
    timing_mark("scan_combine", 1, s);
    return cudaGetLastError();
}

constexpr int kRoundsLow = 2, kRoundsHigh = 8;

int scan_lanes(int N) { return N <= 16 ? 4 : N <= 32 ? 8 : 16; }

int scan_blocks(int C, int G, int N) {
    const int ch = kScanThreads / scan_lanes(N), per = C / G;
    return (per + ch - 1) / ch;
}

// A split sequence is walked twice (the first pass costs the forward 0.65 of the second, the backward
// 0.2), so it is split only where its CTAs leave the SMs short of warps: the forward below half a CTA
// per SM, the backward below two. A segment has at least 4 (2) tiles: with few channels each tile is a
// latency of some microseconds, which shorter segments hide (3 x 333 steps of 518 x 11 states, forward
// and backward: 147 us with 8 tiles, 81 us with 2 to 4). Of the counts that give the SMs, which hold two
// CTAs each, kRoundsLow to kRoundsHigh rounds, the first that fills its last round to 95 percent, else the fullest.
void scan_split(ScanParams *p, bool bwd) {
    const long long ctas = (long long)p->Bn * p->G * scan_blocks(p->Cn, p->G, p->N);
    const int tiles = (p->T + kScanTile - 1) / kScanTile, slots = 304, most = tiles / (bwd ? 2 : 4);
    int segs = 1;
    if (ctas < (bwd ? 304 : 76) && tiles >= 16) {
        const int low = (int)((kRoundsLow * slots + ctas - 1) / ctas), high = (int)(kRoundsHigh * slots / ctas);
        double best = 0.0;
        segs = low < most ? low : most;
        for (int n = segs; n <= high && n <= most && best < 0.95; ++n) {
            const long long all = ctas * n, rounds = (all + slots - 1) / slots;
            const double full = (double)all / (double)(rounds * slots);
            if (full > best) {
                best = full;
                segs = n;
            }
        }
    }
    const int per = (tiles + segs - 1) / segs;
    p->seg_len = per * kScanTile;
    p->segs = (tiles + per - 1) / per;
}

namespace {

template <int LPC, typename T, bool VEC>
cudaError_t scan_fwd_prompt(const ScanParams &p, cudaStream_t s) {
    const dim3 grid(p.Bn * p.G * scan_blocks(p.Cn, p.G, p.N), p.segs);
    cudaError_t e;
    if (p.segs > 1) {
        timing_mark("scan_fwd_ends", 0, s);
        scan_fwd_kernel<LPC, T, VEC, true><<<grid, kScanThreads + kScanHelpers, 0, s>>>(p);
        timing_mark("scan_fwd_ends", 1, s);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        if ((e = launch_scan_combine(p, p.h0, nullptr, false, s)) != cudaSuccess) return e;
    }
    timing_mark("scan_fwd", 0, s);
    scan_fwd_kernel<LPC, T, VEC, false><<<grid, kScanThreads + kScanHelpers, 0, s>>>(p);
    timing_mark("scan_fwd", 1, s);
    return cudaGetLastError();
}

template <int LPC, typename T>
cudaError_t scan_fwd_launch(const ScanParams &p, cudaStream_t s) {
    if (p.T == 1 && p.ckpt == nullptr) {
        const size_t a = 4 * sizeof(T);
        const bool vec = p.N % 4 == 0 && p.ldB % 4 == 0 && p.ldC % 4 == 0 && (uintptr_t)p.B % a == 0 && (uintptr_t)p.C % a == 0;
        timing_mark("scan_step", 0, s);
        scan_step_kernel<LPC, T><<<dim3((unsigned)(((size_t)p.Cn * LPC + 255) / 256), (p.Bn + 3) / 4), 256, 0, s>>>(p, vec);
        timing_mark("scan_step", 1, s);
        return cudaGetLastError();
    }
    return scan_vec<T>(p, ScanGeo<LPC>::V) ? scan_fwd_prompt<LPC, T, true>(p, s) : scan_fwd_prompt<LPC, T, false>(p, s);
}

template <typename T>
cudaError_t scan_fwd_lanes(const ScanParams &p, cudaStream_t s) {
    switch (scan_lanes(p.N)) {
        case 4: return scan_fwd_launch<4, T>(p, s);
        case 8: return scan_fwd_launch<8, T>(p, s);
        default: return scan_fwd_launch<16, T>(p, s);
    }
}

}  // namespace

cudaError_t launch_scan_fwd(const ScanParams &p, int dtype, cudaStream_t s) {
    return dtype == 0 ? scan_fwd_lanes<float>(p, s) : scan_fwd_lanes<__nv_bfloat16>(p, s);
}

}  // namespace gdn

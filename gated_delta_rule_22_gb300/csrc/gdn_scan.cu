// gdn_scan.cu -- selective state space scan, forward: prompts, the step of a single token, and the
// split of long sequences.
//
//     d = softplus(dt + dt_bias),  A = -exp(A_log)
//     h_t = exp(d A) h_{t-1} + d u B_t,   y_t = (C_t . h_t + D u) silu(z)
//
// Each state and step costs one exp2 and four float32 operations (d A log2 e, (d u) B, the update,
// the product with C), each channel and step 2 to 4 elements of memory traffic: with 16 states the
// exponentials' time is the floor, not the memory's.
#include "gdn_scan.cuh"

namespace gdn {

template <int LPC, typename T>
struct FwdSmem {
    using G = ScanGeo<LPC>;
    static constexpr int CH = G::CH, NP = G::NP, TT = kScanTile;
    float4 dx[2][TT][CH / 2];                         // of two channels: d, d, d u, d u
    float B[2][TT][NP], C[2][TT][NP];
    float core[2][TT][G::SP];
    T u[2][TT][CH], z[2][TT][CH];
};

// LITE: the segment's end state from a zero start and its sum of d, nothing else (first pass over a
// split sequence).
//
// Four warps hold the states and do nothing but the recurrence; four more stage the tiles (loads a
// tile ahead, softplus) and finish the outputs, so that the recurrence has no phases in which it
// idles. Two tiles are in flight; named barriers full[2] (staged) and done[2] (walked) hand them over.
// A lane holds four states of two channels: what binds is shared memory, whose 16-byte loads take four
// cycles per warp however many lanes read the same address, and B and C then serve two channels. d and
// d u come in one load for both and are made pairs in registers: staged in pairs, or B and C twice (pairs
// over the channels), the loads grow by more than the moves cost (forward of 2 x 2048 steps 147 us
// against 138; of 4096 x 64 states 723 against 438).
//
// Measured on 2 x 2048 steps of 4096 channels x 16 states, bf16, with checkpoints: 134 us, against 153 with
// one channel per lane; 1 x 4096 steps, split, without checkpoints: 60 us for the ends, 90 for the outputs
// (float32: 142 us without checkpoints; 164 for the split).
// Not the exponentials bind (29 us at 32 per clock and SM) nor the memory (20 us, and 10 for
// checkpoints), but the loads from shared memory and the latency of one or two state warps per scheduler.
// CTAS per SM: three, with 80 registers, where there are more CTAs than two per SM (the split prompt
// takes 161 us in all instead of 167, 8 x 1024 steps of 8192 channels 356 instead of 366), else two (the
// 128 CTAs of the first case, one per SM at any rate, take 160 us instead of 134 with 80 registers).
template <int LPC, typename T, bool VEC, bool LITE, int CTAS>
__global__ void __launch_bounds__(kStateThreads + kScanHelpers, CTAS) scan_fwd_kernel(ScanParams p) {
    using G = ScanGeo<LPC>;
    constexpr int NP = G::NP, V = G::V, TT = kScanTile, ALL = kStateThreads + kScanHelpers;
    constexpr int kFull = 1, kDone = 3;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    FwdSmem<LPC, T> &sm = *reinterpret_cast<FwdSmem<LPC, T> *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const ScanPlace q = scan_place<LPC>(p);
    if (q.first >= q.last) return;
    const int L = row_length(p.lens, q.b, p.T);
    if (tid >= kStateThreads) {
        constexpr int KB = NP * TT / kScanHelpers, ROWS = kScanHelpers / 16, PASS = TT / ROWS;
        // staged elements: steps ts, ts + ROWS, ... of a tile, V channels from cv
        const int h = tid - kStateThreads, ts = h >> 4, cv = (h & 15) * V, nv = q.nc - cv;
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
                const int t = tile * TT + ts + ROWS * i, n = t < L ? nv : 0;
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
                const int st = ts + ROWS * i, t = tile * TT + st;
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
                    float *to = reinterpret_cast<float *>(&sm.dx[buf][st][cv / 2]) + (cv & 1);
                    to[0] = dd[0];
                    to[2] = dd[0] * uu[0];
                } else {
#pragma unroll
                    for (int v = 0; v < V; v += 2)
                        sm.dx[buf][st][(cv + v) / 2] = make_float4(dd[v], dd[v + 1], dd[v] * uu[v], dd[v + 1] * uu[v + 1]);
                }
                if (LITE) {
#pragma unroll
                    for (int v = 0; v < V; ++v) sum_d[v] += dd[v];
                } else {
                    ru[i].keep(&sm.u[buf][st][cv]);
                    if (p.z != nullptr) rz[i].keep(&sm.z[buf][st][cv]);
                }
            }
#pragma unroll
            for (int k = 0; k < KB; ++k) {
                const int e = h + kScanHelpers * k;
                sm.B[buf][e / NP][e % NP] = to_f32(rB[k]);
                if (!LITE) sm.C[buf][e / NP][e % NP] = to_f32(rC[k]);
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
                    const int st = ts + ROWS * i, t = tile * TT + st;
                    if (t >= p.T) continue;
                    float o[V], uu[V], zz[V];
                    load_vec<T, V>(&sm.u[buf][st][cv], uu);
#pragma unroll
                    for (int v = 0; v < V; ++v) o[v] = fmaf(D[v], uu[v], sm.core[buf][st][cv + v]);
                    if (p.z != nullptr) {
                        load_vec<T, V>(&sm.z[buf][st][cv], zz);
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
            // the sum of d over the segment: over a thread's tiles, then over the threads of a channel
#pragma unroll
            for (int v = 0; v < V; ++v) sm.core[0][ts][cv + v] = sum_d[v];
            named_bar_sync(kDone + 2, kScanHelpers);
            for (int cc = h; cc < q.nc; cc += kScanHelpers) {
                float a = 0.f;
                for (int i = 0; i < ROWS; ++i) a += sm.core[0][i][cc];
                p.seg_sum[((size_t)q.seg * p.Bn + q.b) * p.Cn + q.c0 + cc] = a;
            }
        }
        return;
    }
    // this lane's states: n0 .. n0 + 3 of channels ch and ch + 1, as pairs over the channels
    const int pr = warp * G::CPW + lane / LPC, ch = 2 * pr, n0 = 4 * (lane % LPC);
    const bool live[2] = {ch < q.nc, ch + 1 < q.nc};
    const int c[2] = {q.c0 + (live[0] ? ch : 0), q.c0 + (live[1] ? ch + 1 : 0)};
    const size_t row = (size_t)q.b * p.Cn * p.N, seg_row = (size_t)q.seg * p.Bn * p.Cn * p.N + row;
    auto load = [&](const float *rows, float2 (&o)[2][2]) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float e[4] = {0.f, 0.f, 0.f, 0.f};
            if (live[r]) load_states(rows + (size_t)c[r] * p.N, n0, p.N, e);
            o[r][0] = make_float2(e[0], e[1]);
            o[r][1] = make_float2(e[2], e[3]);
        }
    };
    auto store = [&](float *rows, const float2 (&o)[2][2]) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float e[4] = {o[r][0].x, o[r][0].y, o[r][1].x, o[r][1].y};
            if (live[r]) store_states(rows + (size_t)c[r] * p.N, n0, p.N, e);
        }
    };
    float2 A2[2][2], h[2][2];
    load(p.A_log, A2);
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int n = n0 + 2 * k;
            A2[r][k] = make_float2(n < p.N ? -expf(A2[r][k].x) * kLog2e : 0.f, n + 1 < p.N ? -expf(A2[r][k].y) * kLog2e : 0.f);
            h[r][k] = make_float2(0.f, 0.f);
        }
    if (!LITE) {
        if (p.segs > 1) load(p.seg_state + seg_row, h);
        else if (p.h0 != nullptr) load(p.h0 + row, h);
    }
    const int tiles = (p.T + TT - 1) / TT;
    for (int tile = q.first; tile < q.last; ++tile) {
        const int buf = tile & 1;
        if (!LITE && p.ckpt != nullptr) store(p.ckpt + ((size_t)q.b * tiles + tile) * p.Cn * p.N, h);
        named_bar_sync(kFull + buf, ALL);
        // what does not depend on the state (decays, d u B) is formed for the next step before the
        // present one's multiply-adds
        struct Step {
            float2 a[2][2], x[2][2];
        };
        auto prepare = [&](int i, Step &o) {
            const float4 dx = sm.dx[buf][i][pr], b4 = *reinterpret_cast<const float4 *>(&sm.B[buf][i][n0]);
            const float d[2] = {dx.x, dx.y}, x[2] = {dx.z, dx.w};
            const float2 b2[2] = {make_float2(b4.x, b4.y), make_float2(b4.z, b4.w)};
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    o.a[r][k] = decay2(d[r], A2[r][k]);
                    o.x[r][k] = __fmul2_rn(make_float2(x[r], x[r]), b2[k]);
                }
        };
        Step now, then;
        float2 core[4];
        prepare(0, now);
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            if (i + 1 < TT) prepare(i + 1, then);
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int k = 0; k < 2; ++k) h[r][k] = __ffma2_rn(now.a[r][k], h[r][k], now.x[r][k]);
            if (!LITE) {
                const float4 c4 = *reinterpret_cast<const float4 *>(&sm.C[buf][i][n0]);
                float2 sum[2];
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    sum[r] = __ffma2_rn(make_float2(c4.z, c4.w), h[r][1], __fmul2_rn(make_float2(c4.x, c4.y), h[r][0]));
                core[i & 3] = make_float2(sum[0].x + sum[0].y, sum[1].x + sum[1].y);
                if (i % 4 == 3) {
                    const float2 r = lane_sum4<LPC>(core, lane);
                    if (lane % LPC < 4) *reinterpret_cast<float2 *>(&sm.core[buf][i - 3 + (lane & 3)][ch]) = r;
                }
            }
            now = then;
        }
        named_bar_arrive(kDone + buf, ALL);
    }
    if (LITE) store(p.seg_state + seg_row, h);
    else if (p.h_T != nullptr && q.seg == p.segs - 1) store(p.h_T + row, h);
}

// One step (T = 1): a streaming pass over the states, bound by their bytes (read and written once). LPC
// lanes take one channel of four batch rows, so that A is formed once for four states; lane r forms
// row r's d and finishes its output. h_T may be h0. 64 rows of 4096 channels x 16 states: 10 us, 3.5
// TB/s (the states' 34 MB stay in L2 from step to step); by the prompt kernel, whose tiles would hold
// one step of 16, 41 us.
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
// per SM (1 x 4096 steps of 4096 channels x 16 states, 64 CTAs: 160 us split, 275 whole; 2 x 2048 steps,
// 128 CTAs: 169 split, 134 whole), the backward below two (the latter: 402 us split, 535 whole). A segment
// has at least 4 (2) tiles: with few channels each tile is a latency of some microseconds, which shorter
// segments hide (3 x 333 steps of 518 x 11 states, forward and backward: 147 us with 8 tiles, 81 us with 2
// to 4, 143 whole). Of the counts that give the SMs, which hold two
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

template <int LPC, typename T, bool VEC, bool LITE, int CTAS>
cudaError_t scan_fwd_one(const ScanParams &p, dim3 grid, cudaStream_t s) {
    constexpr int smem = (int)sizeof(FwdSmem<LPC, T>);
    if (smem > 48 * 1024) {
        const cudaError_t e = allow_smem<scan_fwd_kernel<LPC, T, VEC, LITE, CTAS>>(smem);
        if (e != cudaSuccess) return e;
    }
    const char *name = LITE ? "scan_fwd_ends" : "scan_fwd";
    timing_mark(name, 0, s);
    scan_fwd_kernel<LPC, T, VEC, LITE, CTAS><<<grid, kStateThreads + kScanHelpers, smem, s>>>(p);
    timing_mark(name, 1, s);
    return cudaGetLastError();
}
template <int LPC, typename T, bool VEC, bool LITE>
cudaError_t scan_fwd_ctas(const ScanParams &p, cudaStream_t s) {
    const dim3 grid(p.Bn * p.G * scan_blocks(p.Cn, p.G, p.N), p.segs);
    return (long long)grid.x * grid.y > 304 ? scan_fwd_one<LPC, T, VEC, LITE, 3>(p, grid, s) : scan_fwd_one<LPC, T, VEC, LITE, 2>(p, grid, s);
}

template <int LPC, typename T, bool VEC>
cudaError_t scan_fwd_prompt(const ScanParams &p, cudaStream_t s) {
    cudaError_t e;
    if (p.segs > 1) {
        if ((e = scan_fwd_ctas<LPC, T, VEC, true>(p, s)) != cudaSuccess) return e;
        if ((e = launch_scan_combine(p, p.h0, nullptr, false, s)) != cudaSuccess) return e;
    }
    return scan_fwd_ctas<LPC, T, VEC, false>(p, s);
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

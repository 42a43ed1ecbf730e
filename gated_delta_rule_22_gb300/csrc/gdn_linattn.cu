// gdn_linattn.cu -- linear attention with a constant decay for each value head: the single step, the
// step-by-step form of prompts and gradients (float32; bf16 of a few steps or at unaligned addresses), the sums of
// sweeps' float32 outputs, and copies that TMA can read. (gdn_linattn_chunk.cu holds the chunked form.)
//
//     S_t = g S_{t-1} + v_t k_t^T,   y_t = S_t q_t
//     dq_t = S_t^T dy_t;   R_t = g R_{t+1} + dy_t q_t^T,   dk_t = R_t^T v_t,   dv_t = R_t k_t,   dS0 = g R_0
//
// Forward and gradients are the same sweep (LinattnSweep in gdn_layer.cuh) over other operands, so that one
// kernel computes them all.
//
// Measured: one step of 64 rows of 32 heads of 128 x 128, 43 us, 6.2 TB/s of state; two to four steps, step by step, 151 to 155 (the
// state in pieces of 8 bytes, by small CTAs). Step by step in float32, 8 x 1024 steps of 32 heads of 128 x 128: 860 to 890 us, 19
// TFLOP/s of the two products of a step. Few rows are bound by the latency of a step's sums over lanes, 135 ns: 1 x 1024 steps of
// 8 heads 136 us, in segments 74. bf16 at addresses that TMA cannot read, 4 x 1024 of 32 heads: 537 us, in chunks 49. The large
// CTAs' form of dims above 128 spills 312 bytes of a thread in bf16.
#include "gdn_layer.cuh"

namespace gdn {

namespace {

constexpr int kStepThreads = 256;
constexpr int kStepRowsPerThread = 4;

constexpr int kWalkTile = kLinattnTile;                 // steps staged at once

constexpr int kSumThreads = 256;

}  // namespace

// ---- one step: a pass over the state, every element read once and written once. LPR lanes share a state
// row (lane j holds columns V j + V LPR m), kStepRowsPerThread rows each, all loaded before the first is used.
template <typename T, int V, int LPR, int NP>
__global__ void __launch_bounds__(kStepThreads) linattn_step_kernel(const LinattnParams p) {
    constexpr int RPT = kStepRowsPerThread, SLOTS = kStepThreads / LPR;
    const LinattnSweep &w = p.sweep[0];
    const int lane = threadIdx.x % LPR, slot = threadIdx.x / LPR;
    const int h = blockIdx.y, b = blockIdx.z, hk = h / (p.Hv / p.Hk), Dk = p.Dk, Dv = p.Dv;
    const size_t head = (size_t)b * p.Hv + h;
    const bool on = row_length(p.lens, b, 1) > 0;
    const int row0 = blockIdx.x * SLOTS * RPT + slot;
    const float *S0 = w.init == nullptr ? nullptr : w.init + head * Dv * Dk;
    float s[RPT][NP][V];
#pragma unroll
    for (int r = 0; r < RPT; ++r)
#pragma unroll
        for (int m = 0; m < NP; ++m) {
            const int row = row0 + r * SLOTS, col = (m * LPR + lane) * V;
#pragma unroll
            for (int i = 0; i < V; ++i) s[r][m][i] = 0.f;
            if (S0 != nullptr && row < Dv && col < Dk) load_vec<float, V>(S0 + (size_t)row * Dk + col, s[r][m]);
        }
    if (on) {
        const T *q = static_cast<const T *>(w.a) + (size_t)b * w.lda + (size_t)hk * Dk;
        const T *k = static_cast<const T *>(w.b) + (size_t)b * w.ldb + (size_t)hk * Dk;
        const T *v = static_cast<const T *>(w.c) + (size_t)b * w.ldc + (size_t)h * Dv;
        const float g = p.g[h];
        float kk[NP][V], qq[NP][V];
#pragma unroll
        for (int m = 0; m < NP; ++m)
#pragma unroll
            for (int i = 0; i < V; ++i) {              // q and k may lie at any address
                const int col = (m * LPR + lane) * V + i;
                kk[m][i] = col < Dk ? to_f32(k[col]) : 0.f;
                qq[m][i] = col < Dk ? to_f32(q[col]) : 0.f;
            }
#pragma unroll
        for (int r = 0; r < RPT; ++r) {
            const int row = row0 + r * SLOTS;
            const float c = row < Dv ? to_f32(v[row]) : 0.f;
            float y = 0.f;
#pragma unroll
            for (int m = 0; m < NP; ++m)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    s[r][m][i] = fmaf(g, s[r][m][i], c * kk[m][i]);
                    y = fmaf(s[r][m][i], qq[m][i], y);
                }
#pragma unroll
            for (int m = LPR / 2; m >= 1; m >>= 1) y += __shfl_xor_sync(kFullMask, y, m);
            if (lane == 0 && row < Dv) static_cast<T *>(w.out)[head * Dv + row] = from_f32<T>(y);
        }
    } else if (lane == 0) {
#pragma unroll
        for (int r = 0; r < RPT; ++r)
            if (row0 + r * SLOTS < Dv) static_cast<T *>(w.out)[head * Dv + row0 + r * SLOTS] = from_f32<T>(0.f);
    }
    if (w.last == nullptr) return;
#pragma unroll
    for (int r = 0; r < RPT; ++r)
#pragma unroll
        for (int m = 0; m < NP; ++m) {
            const int row = row0 + r * SLOTS, col = (m * LPR + lane) * V;
            if (row < Dv && col < Dk) store_vec<float, V>(w.last + (head * Dv + row) * Dk + col, s[r][m]);
        }
}

// ---- step by step. A warp holds ROWS rows of the state X [Dc][Db] in registers, lane l the columns
// 2 l + 64 m and the next (pairs, for the packed instructions); a CTA holds ROWS WARPS rows of one sweep,
// head and batch row and stages some steps of a, b and c in shared memory as float32, the next tile's
// elements in registers meanwhile. A step is three packed instructions per pair of state elements; the outputs
// of four steps are summed over the lanes together, 31 shuffles in five rounds.
// STATE: the segments' end states from zero, nothing else.
template <typename T, int E2, int WARPS, int ROWS, bool STATE>
__global__ void __launch_bounds__(32 * WARPS) linattn_walk_kernel(const LinattnParams p, int blocks0, int blocks1) {
    constexpr int W = 64 * E2;                          // staged columns of a and b
    constexpr int kWalkThreads = 32 * WARPS, kWalkBlock = WARPS * ROWS;     // threads, state rows of a CTA
    static_assert(kWalkThreads % kWalkBlock == 0, "whole steps of zeros at once");
    constexpr int LA = kWalkTile * W / kWalkThreads, LC = kWalkTile * kWalkBlock / kWalkThreads;
    __shared__ __align__(16) float sa[kWalkTile][W], sb[kWalkTile][W], sc[kWalkTile][kWalkBlock];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr bool SEGMENTS = WARPS == 4;               // (the large CTAs take whole rows)
    const int segs = !SEGMENTS ? 1 : STATE ? p.segs - 1 : p.segs, seg = SEGMENTS ? blockIdx.x % segs : 0, x = SEGMENTS ? blockIdx.x / segs : blockIdx.x;
    const int which = x < blocks0 ? 0 : x < blocks0 + blocks1 ? 1 : 2;
    const LinattnSweep &w = p.sweep[which];
    const int block = x - (which == 0 ? 0 : which == 1 ? blocks0 : blocks0 + blocks1);
    const int h = blockIdx.y, b = blockIdx.z, hk = h / (p.Hv / p.Hk), T_ = p.T;
    const int Db = w.Db, Dc = w.Dc, e0 = block * kWalkBlock, row0 = e0 + warp * ROWS;
    const int n = row_length(p.lens, b, T_);
    const float g = p.g[h];
    const size_t head = (size_t)b * p.Hv + h;
    const T *a_ = static_cast<const T *>(w.a) + (size_t)b * T_ * w.lda + (size_t)(w.a_keys ? hk : h) * Db;
    const T *b_ = static_cast<const T *>(w.b) + (size_t)b * T_ * w.ldb + (size_t)(w.b_keys ? hk : h) * Db;
    const T *c_ = static_cast<const T *>(w.c) + (size_t)b * T_ * w.ldc + (size_t)(w.c_keys ? hk : h) * Dc + e0;
    // the state
    float2 s[ROWS][E2];
    auto place = [&](int r, int m, int i) {             // of an element of the state in init and last
        const int row = row0 + r, col = 2 * lane + 64 * m + i;
        return w.init_t ? (head * Db + col) * Dc + row : (head * Dc + row) * Db + col;
    };
    auto inside = [&](int r, int m, int i) { return row0 + r < Dc && 2 * lane + 64 * m + i < Db; };
    const bool pairs = !w.init_t && Db % 2 == 0;        // of a row's elements in init and last, aligned to 8 bytes
    const int tiles = (n + kWalkTile - 1) / kWalkTile;
    const int first_tile = SEGMENTS ? seg * p.seg_chunks : 0;                                       // in the order of the sweep
    const int last_tile = SEGMENTS ? min(first_tile + p.seg_chunks, tiles) : tiles;
    if (STATE && last_tile >= tiles) return;            // (nothing follows)
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
        for (int m = 0; m < E2; ++m) {
            if (STATE) {
                s[r][m] = make_float2(0.f, 0.f);
                continue;
            }
            if (pairs) {
                s[r][m] = w.init != nullptr && inside(r, m, 0) ? *reinterpret_cast<const float2 *>(w.init + place(r, m, 0)) : make_float2(0.f, 0.f);
                continue;
            }
            s[r][m].x = w.init != nullptr && inside(r, m, 0) ? w.init[place(r, m, 0)] : 0.f;
            s[r][m].y = w.init != nullptr && inside(r, m, 1) ? w.init[place(r, m, 1)] : 0.f;
        }
    auto state_at = [&](int of, int r, int m, int i) -> float & {          // of the state behind segment `of`
        return w.states[(((size_t)of * p.B + b) * p.Hv + h) * Dc * Db + (size_t)(row0 + r) * Db + 2 * lane + 64 * m + i];
    };
    if (SEGMENTS && !STATE && seg > 0 && first_tile < tiles) {      // through the earlier segments
        const int before = w.rev ? n - (tiles - first_tile) * kWalkTile - 1 : first_tile * kWalkTile;
        const float decay = exp2f(before == 0 ? 0.f : before * log2f(g));
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
#pragma unroll
            for (int m = 0; m < E2; ++m) {
                if (inside(r, m, 0)) s[r][m].x = fmaf(decay, s[r][m].x, state_at(seg - 1, r, m, 0));
                if (inside(r, m, 1)) s[r][m].y = fmaf(decay, s[r][m].y, state_at(seg - 1, r, m, 1));
            }
    }
    T ra[LA], rb[LA], rc[LC];
    auto fetch = [&](int tile) {
        const int t0 = tile * kWalkTile;
#pragma unroll
        for (int i = 0; i < LA; ++i) {
            const int t = t0 + (tid + i * kWalkThreads) / W, col = (tid + i * kWalkThreads) % W;
            const bool ok = t < n && col < Db;
            if (!STATE) ra[i] = ok ? a_[(size_t)t * w.lda + col] : from_f32<T>(0.f);
            rb[i] = ok ? b_[(size_t)t * w.ldb + col] : from_f32<T>(0.f);
        }
#pragma unroll
        for (int i = 0; i < LC; ++i) {
            const int t = t0 + (tid + i * kWalkThreads) / kWalkBlock, row = (tid + i * kWalkThreads) % kWalkBlock;
            rc[i] = t < n && e0 + row < Dc ? c_[(size_t)t * w.ldc + row] : from_f32<T>(0.f);
        }
    };
    // outputs: a row of a value head, or (keys of their own) of its key head
    const size_t out_step = (size_t)p.Hv * Dc;          // where the heads are summed later, and where Hk == Hv
    const size_t out0 = (size_t)b * T_ * out_step + (size_t)h * Dc;
    auto put = [&](int t, int row, float x) {
        const size_t at = out0 + (size_t)t * out_step + row;
        if (w.sums) w.part[at] = x;
        else static_cast<T *>(w.out)[at] = from_f32<T>(x);
    };
    if (first_tile < last_tile) fetch(w.rev ? tiles - 1 - first_tile : first_tile);
    bool first = w.rev && seg == 0;                     // backwards the first step does not decay the state
    for (int it = first_tile; it < last_tile; ++it) {
        const int tile = w.rev ? tiles - 1 - it : it, t0 = tile * kWalkTile, steps = min(kWalkTile, n - t0);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < LA; ++i) {
            const int j = tid + i * kWalkThreads;
            if (!STATE) sa[j / W][j % W] = to_f32(ra[i]);
            sb[j / W][j % W] = to_f32(rb[i]);
        }
#pragma unroll
        for (int i = 0; i < LC; ++i) {
            const int j = tid + i * kWalkThreads;
            sc[j / kWalkBlock][j % kWalkBlock] = to_f32(rc[i]);
        }
        __syncthreads();
        if (it + 1 < last_tile) fetch(w.rev ? tile - 1 : tile + 1);
        if (row0 >= Dc) continue;                       // (a warp without rows stages only)
        auto step = [&](int k, float *y) {
            const int i = w.rev ? steps - 1 - k : k;
            const float gs = first ? 1.f : g;
            const float2 g2 = make_float2(gs, gs);
            first = false;
            float2 av[E2], bv[E2];
#pragma unroll
            for (int m = 0; m < E2; ++m) {
                av[m] = STATE ? make_float2(0.f, 0.f) : *reinterpret_cast<const float2 *>(&sa[i][2 * lane + 64 * m]);
                bv[m] = *reinterpret_cast<const float2 *>(&sb[i][2 * lane + 64 * m]);
            }
            float c[ROWS];
#pragma unroll
            for (int r = 0; r < ROWS; r += 4) *reinterpret_cast<float4 *>(c + r) = *reinterpret_cast<const float4 *>(&sc[i][warp * ROWS + r]);
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                const float2 c2 = make_float2(c[r], c[r]);
                float2 acc = make_float2(0.f, 0.f);
#pragma unroll
                for (int m = 0; m < E2; ++m) {
                    s[r][m] = __ffma2_rn(g2, s[r][m], __fmul2_rn(c2, bv[m]));
                    if (!STATE) acc = __ffma2_rn(s[r][m], av[m], acc);
                }
                y[r] = acc.x + acc.y;
            }
        };
        for (int k = 0; k < steps; k += 4) {           // the sums of four steps are formed together
            float y[4 * ROWS];
            if (k + 4 <= steps) {
#pragma unroll
                for (int u = 0; u < 4; ++u) step(k + u, y + u * ROWS);
            } else {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (k + u < steps) step(k + u, y + u * ROWS);
                    else
#pragma unroll
                        for (int r = 0; r < ROWS; ++r) y[u * ROWS + r] = 0.f;
                }
            }
            if (STATE) continue;
            const float sum = transpose_reduce<4 * ROWS>(y, lane);
            constexpr int SHARE = 32 / (4 * ROWS);     // lanes with the same sum
            const int at = lane / SHARE, ku = k + at / ROWS, row = row0 + at % ROWS;
            if (lane % SHARE == 0 && ku < steps && row < Dc) put(t0 + (w.rev ? steps - 1 - ku : ku), row, sum);
        }
    }
    if (STATE) {
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
#pragma unroll
            for (int m = 0; m < E2; ++m) {
                if (inside(r, m, 0)) state_at(seg, r, m, 0) = s[r][m].x;
                if (inside(r, m, 1)) state_at(seg, r, m, 1) = s[r][m].y;
            }
        return;
    }
    if (e0 + tid % kWalkBlock < Dc) {                   // zeros behind the row, by turns
        constexpr int ZEROS = kWalkThreads / kWalkBlock;
        for (long long t = n + (long long)seg * ZEROS + tid / kWalkBlock; t < T_; t += segs * ZEROS) put((int)t, e0 + tid % kWalkBlock, 0.f);
    }
    if (w.last != nullptr && (!SEGMENTS || seg == (tiles > 0 ? (tiles - 1) / p.seg_chunks : 0))) {
        const float gl = w.rev && n > 0 ? g : 1.f;
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
#pragma unroll
            for (int m = 0; m < E2; ++m) {
                if (pairs) {
                    if (inside(r, m, 0)) *reinterpret_cast<float2 *>(w.last + place(r, m, 0)) = make_float2(gl * s[r][m].x, gl * s[r][m].y);
                    continue;
                }
                if (inside(r, m, 0)) w.last[place(r, m, 0)] = gl * s[r][m].x;
                if (inside(r, m, 1)) w.last[place(r, m, 1)] = gl * s[r][m].y;
            }
    }
}

// ---- outputs from the sweeps' float32 ones: planes (blocks of Db) and the value heads of a key head, added in
// ascending order
template <typename T, int V>
__global__ void __launch_bounds__(kSumThreads) linattn_sum_kernel(const LinattnParams p) {
    const LinattnSum &w = p.sum[blockIdx.y];
    T *out = static_cast<T *>(w.out);
    const int pieces = w.D / V, add = w.group * w.planes;
    const size_t n = (size_t)p.B * p.T * w.heads * pieces;
    for (size_t i = (size_t)blockIdx.x * kSumThreads + threadIdx.x; i < n; i += (size_t)gridDim.x * kSumThreads) {
        const size_t head = i / pieces;                 // (batch row, step, head)
        const float *x = w.part + head * w.group * w.pitch + (i - head * pieces) * V;
        float s[V];
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = 0.f;
#pragma unroll 4
        for (int r = 0; r < add; ++r) {
            float e[V];
            load_vec<float, V>(x + (r % w.planes) * w.plane + (size_t)(r / w.planes) * w.pitch, e);
#pragma unroll
            for (int v = 0; v < V; ++v) s[v] += e[v];
        }
        store_vec<T, V>(out + i * V, s);
    }
}

// ---- rows that TMA can read, from rows that it cannot: eight elements of a padded row by a thread
__global__ void __launch_bounds__(kSumThreads) linattn_copy_kernel(const LinattnParams p) {
    const LinattnCopy &w = p.copy[blockIdx.y];
    const int pieces = w.pitch / 8;
    const size_t n = (size_t)p.B * p.T * w.H * pieces;
    for (size_t i = (size_t)blockIdx.x * kSumThreads + threadIdx.x; i < n; i += (size_t)gridDim.x * kSumThreads) {
        const size_t head = i / pieces, row = head / w.H;
        const int c0 = (int)(i - head * pieces) * 8;
        const unsigned short *in = static_cast<const unsigned short *>(w.in) + row * w.ld + (head - row * w.H) * w.D;
        uint32_t x[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) x[c] = c0 + c < w.D ? in[c0 + c] : 0u;
        static_cast<uint4 *>(w.out)[i] = make_uint4(x[0] | x[1] << 16, x[2] | x[3] << 16, x[4] | x[5] << 16, x[6] | x[7] << 16);
    }
}

cudaError_t launch_linattn_copies(const LinattnParams &p, cudaStream_t s) {
    size_t n = 0;
    for (int i = 0; i < p.copies; ++i) {
        const size_t m = (size_t)p.B * p.T * p.copy[i].H * (p.copy[i].pitch / 8);
        n = m > n ? m : n;
    }
    const size_t ctas = (n + kSumThreads - 1) / kSumThreads;
    timing_mark("linattn_copy", 0, s);
    linattn_copy_kernel<<<dim3((unsigned)(ctas < 152 * 32 ? ctas : 152 * 32), p.copies), kSumThreads, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    timing_mark("linattn_copy", 1, s);
    return e;
}

template <typename T>
static cudaError_t launch_step_t(const LinattnParams &p, cudaStream_t s) {
    auto run = [&](auto kernel, int lpr) {
        const int rows = kStepThreads / lpr * kStepRowsPerThread;
        kernel<<<dim3((p.Dv + rows - 1) / rows, p.Hv, p.B), kStepThreads, 0, s>>>(p);
    };
    if (p.Dk % 4 != 0) {
        if (p.Dk <= 32) run(linattn_step_kernel<T, 1, 32, 1>, 32);
        else if (p.Dk <= 128) run(linattn_step_kernel<T, 1, 32, 4>, 32);
        else run(linattn_step_kernel<T, 1, 32, 8>, 32);
    } else if (p.Dk <= 32) run(linattn_step_kernel<T, 4, 8, 1>, 8);
    else if (p.Dk <= 64) run(linattn_step_kernel<T, 4, 16, 1>, 16);
    else if (p.Dk <= 128) run(linattn_step_kernel<T, 4, 32, 1>, 32);
    else run(linattn_step_kernel<T, 4, 32, 2>, 32);
    return cudaGetLastError();
}

cudaError_t launch_linattn_step(const LinattnParams &p, int dtype, cudaStream_t s) {
    timing_mark("linattn_step", 0, s);
    const cudaError_t e = dtype == 0 ? launch_step_t<float>(p, s) : launch_step_t<__nv_bfloat16>(p, s);
    timing_mark("linattn_step", 1, s);
    return e;
}

template <typename T>
static cudaError_t launch_sums_t(const LinattnParams &p, cudaStream_t s) {
    size_t n = 0;
    bool vec = true;
    for (int i = 0; i < p.sums; ++i) {
        const size_t m = (size_t)p.B * p.T * p.sum[i].heads * p.sum[i].D;
        n = m > n ? m : n;
        vec = vec && p.sum[i].D % 4 == 0 && p.sum[i].pitch % 4 == 0;
    }
    const size_t ctas = (n / (vec ? 4 : 1) + kSumThreads - 1) / kSumThreads;
    const dim3 grid((unsigned)(ctas < 152 * 32 ? ctas : 152 * 32), p.sums);
    if (vec) linattn_sum_kernel<T, 4><<<grid, kSumThreads, 0, s>>>(p);
    else linattn_sum_kernel<T, 1><<<grid, kSumThreads, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_linattn_sums(const LinattnParams &p, int dtype, cudaStream_t s) {
    timing_mark("linattn_sums", 0, s);
    const cudaError_t e = dtype == 0 ? launch_sums_t<float>(p, s) : launch_sums_t<__nv_bfloat16>(p, s);
    timing_mark("linattn_sums", 1, s);
    return e;
}

// ---- what the segments up to each leave, from what each leaves: E_s += g^(steps of s) E_{s-1}. All segments here but
// the first hold whole tiles only.
__global__ void __launch_bounds__(kSumThreads) linattn_walk_join_kernel(const LinattnParams p) {
    const int b = blockIdx.z, h = blockIdx.y, which = blockIdx.x % p.sweeps, n = p.Dk * p.Dv;
    const int tiles = (row_length(p.lens, b, p.T) + kWalkTile - 1) / kWalkTile;
    const float decay = exp2f(p.seg_chunks * kWalkTile * log2f(p.g[h]));
    const size_t step = (size_t)p.B * p.Hv * n;
    for (int i = blockIdx.x / p.sweeps * kSumThreads + threadIdx.x; i < n; i += gridDim.x / p.sweeps * kSumThreads) {
        float *E = p.sweep[which].states + ((size_t)b * p.Hv + h) * n + i, sum = 0.f;
        for (int s = 0; s < p.segs - 1 && (s + 1) * p.seg_chunks < tiles; ++s, E += step) *E = sum = fmaf(decay, sum, *E);
    }
}

template <typename T, int WARPS, int ROWS, bool STATE>
static cudaError_t launch_walk_w(const LinattnParams &p, cudaStream_t s) {
    int blocks[3] = {0, 0, 0}, widest = 1;
    for (int i = 0; i < p.sweeps; ++i) {
        blocks[i] = (p.sweep[i].Dc + WARPS * ROWS - 1) / (WARPS * ROWS);
        widest = p.sweep[i].Db > widest ? p.sweep[i].Db : widest;
    }
    const dim3 grid((blocks[0] + blocks[1] + blocks[2]) * (STATE ? p.segs - 1 : p.segs), p.Hv, p.B);
    if (widest <= 64) linattn_walk_kernel<T, 1, WARPS, ROWS, STATE><<<grid, 32 * WARPS, 0, s>>>(p, blocks[0], blocks[1]);
    else if (widest <= 128) linattn_walk_kernel<T, 2, WARPS, ROWS, STATE><<<grid, 32 * WARPS, 0, s>>>(p, blocks[0], blocks[1]);
    else linattn_walk_kernel<T, 4, WARPS, ROWS, STATE><<<grid, 32 * WARPS, 0, s>>>(p, blocks[0], blocks[1]);
    return cudaGetLastError();
}

// CTAs of eight warps of eight rows share what is staged; of four warps of four rows where that would leave SMs idle
// or where reading the state is the work (float32, 1024 steps of 8 heads of 128 x 128: 142 us before segments, 259 with the
// large ones; of 4 x 32 heads 565 and 443; bf16, 64 x 32 heads: 2 steps 148 and 159 us).
static bool walk_small(const LinattnParams &p) {
    long long ctas = 0;
    for (int i = 0; i < p.sweeps; ++i) ctas += (p.sweep[i].Dc + 63) / 64;
    return ctas * p.Hv * p.B < 152 || p.T < 16;
}

// Segments of a row, where the small CTAs leave room for more of them (two to four on an SM, by their registers): as
// many as fill it, of 32 steps at least. float32, 1024 steps of 128 x 128, whole and in segments: 4 heads 136 and 40 us,
// 16 heads 136 and 124, 24 heads (two segments) 185 and 175; 128 steps of 8 heads 20.8 and 19.4.
void linattn_step_segments(LinattnParams *p) {
    const int tiles = (p->T + kWalkTile - 1) / kWalkTile;
    long long ctas = 0;
    int widest = 1;
    for (int i = 0; i < p->sweeps; ++i) {
        ctas += (p->sweep[i].Dc + 15) / 16;
        widest = p->sweep[i].Db > widest ? p->sweep[i].Db : widest;
    }
    ctas *= (long long)p->Hv * p->B;
    long long segs = walk_small(*p) ? 152 * (widest <= 64 ? 4 : widest <= 128 ? 3 : 2) / ctas : 1;
    if (segs > tiles / 2) segs = tiles / 2;
    if (segs < 2) segs = 1;
    p->seg_chunks = (int)((tiles + segs - 1) / segs);
    p->segs = (tiles + p->seg_chunks - 1) / p->seg_chunks;
}

template <typename T>
static cudaError_t launch_walk_t(const LinattnParams &p, cudaStream_t s) {
    if (!walk_small(p)) return launch_walk_w<T, 8, 8, false>(p, s);
    if (p.segs > 1) {
        cudaError_t e = launch_walk_w<T, 4, 4, true>(p, s);
        if (e == cudaSuccess && p.segs > 2) {
            const int ctas = (p.Dk * p.Dv + kSumThreads - 1) / kSumThreads;
            linattn_walk_join_kernel<<<dim3(p.sweeps * ctas, p.Hv, p.B), kSumThreads, 0, s>>>(p);
            e = cudaGetLastError();
        }
        if (e != cudaSuccess) return e;
    }
    return launch_walk_w<T, 4, 4, false>(p, s);
}

cudaError_t launch_linattn_steps(const LinattnParams &p, int dtype, cudaStream_t s) {
    timing_mark("linattn_walk", 0, s);
    cudaError_t e = dtype == 0 ? launch_walk_t<float>(p, s) : launch_walk_t<__nv_bfloat16>(p, s);
    timing_mark("linattn_walk", 1, s);
    if (e == cudaSuccess && p.sums > 0) e = launch_linattn_sums(p, dtype, s);
    return e;
}

}  // namespace gdn

// gdn_layer.cuh -- parameter blocks, launchers and device helpers of the layer operators: the
// short causal convolution, the selective state space scan, the linear attention with a decay, the
// group norm, the norms around a block and the projection (internal; not part of the C ABI).
#pragma once

#include "gdn_common.cuh"

#include <atomic>

namespace gdn {

enum { kActNone = 0, kActSilu = 1, kActGelu = 2 };

// ---- shared with the C ABI's first file (gdn_api.cu)
void api_clear_error();
int api_cuda_status(cudaError_t e);
int api_device_status_address(int **out);
// Tensor map of `planes` row-major bf16 [rows][cols] arrays with `ld` elements between rows (planes
// rows * ld apart), 128-byte swizzle; what lies outside an array reads as zero. box_blocks = 0: 3-D
// {cols, rows, planes}, box {64, box_rows, 1}. Else (cols a multiple of 64) 4-D {64, rows, cols / 64,
// planes}, box {64, box_rows, box_blocks, 1}: box_blocks neighbouring boxes of 64 columns by one copy.
int api_planes_map(CUtensorMap *map, const void *ptr, uint64_t cols, uint64_t rows, uint64_t planes, uint64_t ld, int box_rows,
                   int box_blocks);
// Tensor map of a bf16 [B][T][H][D] array with `ld` elements between steps: 4-D {D, H, T, B}, box {64, 1,
// box_t, 1}, 128-byte swizzle; what lies outside reads as zero.
int api_heads_map(CUtensorMap *map, const void *ptr, int B, int T, int H, int D, long long ld, int box_t);

// ---- parameter blocks
struct ConvParams {
    const void *x, *s0, *dy, *ds_T;
    const float *w, *bias;
    const int *lens;
    void *y, *s_T, *dx, *ds0;
    float *dw, *dbias;
    float *part;            // backward: [slices][W + 1][C] partial sums of dw and dbias
    long long ldx;
    int B, T, C, W, act;
};

struct ScanParams {
    const void *u, *dt, *B, *C, *z, *dy;
    const float *A_log, *D, *dt_bias, *h0, *dh_T;
    const int *lens;
    void *y, *du, *ddt, *dB, *dC, *dz;
    float *h_T, *ckpt, *dA_log, *dD, *ddt_bias, *dh0;
    // sequence split: per (segment, b) the end state from a zero start (or, backward, the start
    // adjoint from a zero end) [segs][B][C][N], turned in place into each segment's incoming state
    // (adjoint), and the segment's sum of d [segs][B][C]
    float *seg_state, *seg_sum;
    float *part_bc;         // backward: [channel blocks of a group][B][T][G][2 N] partial dB, dC
    float *part_c;          // backward: [segs][B][N + 2][C] partial dA, dD, ddt_bias
    long long ldu, lddt, ldz, ldB, ldC;
    int Bn, T, Cn, N, G, segs, seg_len;   // seg_len: steps per segment, a multiple of kScanTile
};

struct NormParams {
    const void *x, *z, *dy;
    const float *w, *b;
    const float *stats_in;
    void *y, *dx, *dz;
    float *stats, *dw, *db;
    float *part;            // backward: [slices][2][G D] partial sums of dw and db
    long long ldx, ldz;
    int M, G, D, act, center, slices;
    float eps;
};

struct LinearParams {
    const void *x, *W, *bias, *res, *pre_in, *dy;
    void *y, *pre, *dx, *dW, *dbias;
    char *ws;               // linear_fwd_workspace / linear_bwd_workspace bytes
    int *status;
    long long ldx, ldw, ldres;
    int M, N, K, act;
};

// One sweep of the linear attention: over the steps of a row, in order or (rev) backwards, with a state
// X of [Dc][Db], started from init:
//     X <- g X + outer(c_t, b_t)  (rev: the first step does not decay init),   out_t = X a_t
// The forward is one, and so is each gradient: dq is (dy, v, k), dk backwards (v, dy, q), dv backwards
// (k, q, dy), for (a, b, c).
struct LinattnSweep {
    const void *a, *b, *c;
    const float *init;         // the state before the first step taken; null: zeros
    float *last;               // the state behind the last (rev: decayed once more); null: not wanted
    void *out;                 // [B][T][heads][Dc] in the call's type, the heads those of c
    float *part;               // (sums) float32 outputs by value head instead, [blocks of Db][B][T][Hv][Dc], to be added
                               // or written to rows that are no multiples of 8
    long long lda, ldb, ldc;   // elements between steps
    int a_keys, b_keys, c_keys;   // the operand's heads are key heads
    int Db, Dc, rev;
    int init_t;                // init lies transposed, [Db][Dc]
    int sums;                  // out is formed from part (LinattnSum)
    int a_map, b_map, c_map;   // tensor maps of the operands
    int Db_of, Dc_of;          // the dims of init, last and out: Db and Dc, which the chunked form pads to multiples of 8
    float *states;             // step by step: what the segments up to each but the last leave, [segs - 1][B][Hv][Dc][Db]
};

// A sweep's outputs from its float32 ones: the sum over `planes` and `group` value heads, in ascending order.
struct LinattnSum {
    const float *part;         // [planes][B][T][heads][group][pitch]
    void *out;                 // [B][T][heads][D]
    size_t plane;
    int planes, group, heads, D, pitch;
};

// A bf16 operand that TMA cannot read (rows or strides that are no multiples of 8), copied to rows padded with zeros.
struct LinattnCopy {
    const void *in;            // [B][T][H][D], ld elements between steps
    void *out;                 // [B][T][H][pitch]
    long long ld;
    int H, D, pitch;
};

struct LinattnMaps { CUtensorMap map[4]; };   // q, k, v, dy

struct LinattnParams {
    LinattnSweep sweep[3];
    LinattnSum sum[3];
    LinattnCopy copy[4];
    int sweeps, sums, copies;
    const float *g;
    const int *lens;
    int *status;
    int B, T, Hk, Hv, Dk, Dv;
    // A row is taken in `segs` segments of seg_chunks chunks (step by step: of seg_chunks tiles of kLinattnTile steps).
    // seg_state: chunked form, what the segments up to each but the last leave, from a zero state: [CTAs /
    // segs][segs - 1][128][128]
    int segs, seg_chunks;
    float *seg_state;
};

constexpr int kLinattnChunk = 128;   // steps of a chunk
constexpr int kLinattnTile = 16;     // steps staged at once, step by step

struct ResnormParams {
    const void *x, *h, *z, *dy, *dr;
    const float *scale, *w_post, *w_pre, *stats_in;
    void *r, *y, *dx, *dh, *dz;
    float *stats, *dscale, *dw_post, *dw_pre;
    float *part;               // backward: [ctas][2][D] partial sums of what dscale and dw_post are made of, and of dw_pre
    float *part_z;             // backward, more than one unit for a row of z: [units][D] partial sums of dz before act'(z)
    long long ldx, ldh, ldz;
    int M, D, gate_rows, act, post, pre;
    int unit, per_gate, units, ctas;   // backward: rows of a unit, units of a row of z, units, CTAs that take them
    float eps;
};

constexpr int kScanTile = 16;   // steps between the scan's checkpoints, and of one staged tile
constexpr int kLinearFewRows = 32;   // rows that the projection's forward streams on the CUDA cores where TMA cannot read

// ---- geometry shared by the launchers and the size queries
int conv_bwd_slices(const ConvParams &p);
int scan_lanes(int N);                              // lanes that share one channel's states
int scan_blocks(int C, int G, int N);               // channel blocks of one group
void scan_split(ScanParams *p, bool bwd);           // chooses segs and seg_len
int norm_bwd_slices(int M, int G, int D, int dtype);
void resnorm_units(ResnormParams *p, int dtype);   // chooses unit, per_gate, units and ctas
size_t linear_fwd_workspace(const LinearParams &p, int dtype);
size_t linear_bwd_workspace(const LinearParams &p, int dtype);

// ---- launchers (dtype: 0 float32, 1 bfloat16)
cudaError_t launch_conv_fwd(const ConvParams &p, int dtype, cudaStream_t s);
cudaError_t launch_conv_bwd(const ConvParams &p, int dtype, cudaStream_t s);
cudaError_t launch_scan_fwd(const ScanParams &p, int dtype, cudaStream_t s);
cudaError_t launch_scan_bwd(const ScanParams &p, int dtype, cudaStream_t s);
cudaError_t launch_norm_fwd(const NormParams &p, int dtype, cudaStream_t s);
cudaError_t launch_norm_bwd(const NormParams &p, int dtype, cudaStream_t s);
cudaError_t launch_linattn_step(const LinattnParams &p, int dtype, cudaStream_t s);    // T = 1, the forward's sweep
cudaError_t launch_linattn_steps(const LinattnParams &p, int dtype, cudaStream_t s);   // all sweeps, then their sums
size_t linattn_segments(LinattnParams *p);                                             // chooses segs and seg_chunks; the states of seg_state
void linattn_step_segments(LinattnParams *p);                                          // the same, step by step
cudaError_t launch_linattn_chunks(const LinattnParams &p, const LinattnMaps &maps, cudaStream_t s);
cudaError_t launch_linattn_copies(const LinattnParams &p, cudaStream_t s);
cudaError_t launch_linattn_sums(const LinattnParams &p, int dtype, cudaStream_t s);
cudaError_t launch_resnorm_fwd(const ResnormParams &p, int dtype, cudaStream_t s);
cudaError_t launch_resnorm_bwd(const ResnormParams &p, int dtype, cudaStream_t s);
// These return a GDN_* code (they encode tensor maps).
int launch_linear_fwd(const LinearParams &p, int dtype, cudaStream_t s);
int launch_linear_bwd(const LinearParams &p, int dtype, cudaStream_t s);

// Raises a kernel's limit of dynamic shared memory, once per device (the call costs about a
// microsecond, as much as a third of a launch).
template <auto Kernel>
inline cudaError_t allow_smem(int bytes) {
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// ---- device helpers
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 1 / (1 + exp(-x)) from the hardware's exp2 and reciprocal: a relative error of a few 2^-23, and for
// negative x of |x| 2^-24 more, as the product x log2 e is rounded (20 x 2^-23 at -40, where the value
// itself is 4e-18). An exponent that overflows gives 1 / inf = 0.
__device__ __forceinline__ float sigmoid_hw(float x) { return rcp(1.f + ex2(-x * kLog2e)); }
__device__ __forceinline__ float2 sigmoid2_hw(float2 x) {
    const float2 e = __fmul2_rn(x, make_float2(-kLog2e, -kLog2e));
    const float2 d = __fadd2_rn(make_float2(ex2(e.x), ex2(e.y)), make_float2(1.f, 1.f));
    return make_float2(rcp(d.x), rcp(d.y));
}
__device__ __forceinline__ float silu_hw(float x) { return x * sigmoid_hw(x); }
__device__ __forceinline__ float dsilu_hw(float x) {
    const float s = sigmoid_hw(x);
    return s * fmaf(x, 1.f - s, 1.f);
}
__device__ __forceinline__ float gelu_f(float x) { return 0.5f * x * (1.f + erff(x * 0.70710678f)); }
__device__ __forceinline__ float dgelu_f(float x) {
    return fmaf(x, 0.3989422804f * ex2(-0.5f * kLog2e * x * x), 0.5f * (1.f + erff(x * 0.70710678f)));
}
// softplus(x) = max(x, 0) + log1p(exp(-|x|)), and the logistic function of x from the same exponential.
// exp(-|x|): the product with log2 e is carried to twice float32 (Dekker's two-term product, by fused
// multiply-adds), so that the hardware's exp2 sees no rounded argument. log1p(e) for e in [0, 1]: 2 atanh(e / (2 + e)) by the series of atanh, whose
// argument, a quotient with one Newton correction by its remainder, is at most 1/3 (seven terms:
// 1.4e-8 relative), with full relative accuracy for small e.
__device__ __forceinline__ void softplus_full(float x, float &sp, float &sg) {
    const float ax = fminf(fabsf(x), 200.f), hi = -ax * kLog2e;
    const float lo = fmaf(-ax, 1.925963033e-8f, fmaf(-ax, kLog2e, -hi));
    float e = ex2(hi);
    e = fmaf(e, lo * 0.69314718f, e);
    const float d = 2.f + e, r = rcp(d);
    float s = e * r;
    s = fmaf(r, fmaf(-s, d, e), s);
    const float q = s * s;
    float f = fmaf(q, 1.f / 13.f, 1.f / 11.f);
    f = fmaf(q, f, 1.f / 9.f);
    f = fmaf(q, f, 1.f / 7.f);
    f = fmaf(q, f, 1.f / 5.f);
    f = fmaf(q, f, 1.f / 3.f);
    f = fmaf(q, f, 1.f);
    sp = fmaf(2.f * s, f, x <= 0.f ? 0.f : x);      // a NaN stays one
    const float r1 = rcp(1.f + e);
    sg = x >= 0.f ? r1 : e * r1;
}
// The same for two values at once (packed instructions).
__device__ __forceinline__ float2 softplus2_full(float2 x, float2 &e) {
    const float2 ax = make_float2(fminf(fabsf(x.x), 200.f), fminf(fabsf(x.y), 200.f));
    const float2 l = make_float2(-kLog2e, -kLog2e), hi = __fmul2_rn(ax, l);
    const float2 lo = __ffma2_rn(ax, make_float2(-1.925963033e-8f, -1.925963033e-8f), __ffma2_rn(ax, l, make_float2(-hi.x, -hi.y)));
    e = make_float2(ex2(hi.x), ex2(hi.y));
    e = __ffma2_rn(e, __fmul2_rn(lo, make_float2(0.69314718f, 0.69314718f)), e);
    const float2 d = __fadd2_rn(e, make_float2(2.f, 2.f)), r = make_float2(rcp(d.x), rcp(d.y));
    float2 s = __fmul2_rn(e, r);
    s = __ffma2_rn(r, __ffma2_rn(make_float2(-s.x, -s.y), d, e), s);
    const float2 q = __fmul2_rn(s, s);
    float2 f = __ffma2_rn(q, make_float2(1.f / 13.f, 1.f / 13.f), make_float2(1.f / 11.f, 1.f / 11.f));
    f = __ffma2_rn(q, f, make_float2(1.f / 9.f, 1.f / 9.f));
    f = __ffma2_rn(q, f, make_float2(1.f / 7.f, 1.f / 7.f));
    f = __ffma2_rn(q, f, make_float2(1.f / 5.f, 1.f / 5.f));
    f = __ffma2_rn(q, f, make_float2(1.f / 3.f, 1.f / 3.f));
    f = __ffma2_rn(q, f, make_float2(1.f, 1.f));
    return __ffma2_rn(__fadd2_rn(s, s), f, make_float2(x.x <= 0.f ? 0.f : x.x, x.y <= 0.f ? 0.f : x.y));
}
__device__ __forceinline__ float2 softplus2_full(float2 x) {
    float2 e;
    return softplus2_full(x, e);
}
// softplus and the logistic function
__device__ __forceinline__ void softplus2_full(float2 x, float2 &sp, float2 &sg) {
    float2 e;
    sp = softplus2_full(x, e);
    const float2 d = __fadd2_rn(e, make_float2(1.f, 1.f)), r = make_float2(rcp(d.x), rcp(d.y));
    sg = __fmul2_rn(r, make_float2(x.x >= 0.f ? 1.f : e.x, x.y >= 0.f ? 1.f : e.y));
}
__device__ __forceinline__ float softplus_full(float x) {
    float sp, sg;
    softplus_full(x, sp, sg);
    return sp;
}

// V consecutive elements as float, from an address aligned to V elements
template <typename T, int V>
__device__ __forceinline__ void load_vec(const T *p, float (&o)[V]) {
    constexpr int BYTES = V * (int)sizeof(T);
    if constexpr (sizeof(T) == 4) {
        if constexpr (BYTES == 16) {
            const float4 x = *reinterpret_cast<const float4 *>(p);
            o[0] = x.x; o[1] = x.y; o[2] = x.z; o[3] = x.w;
        } else if constexpr (BYTES == 8) {
            const float2 x = *reinterpret_cast<const float2 *>(p);
            o[0] = x.x; o[1] = x.y;
        } else {
            static_assert(V == 1, "vector width");
            o[0] = to_f32(*p);
        }
    } else {
        if constexpr (BYTES == 16) {
            const uint4 x = *reinterpret_cast<const uint4 *>(p);
            const uint32_t r[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                o[2 * i] = __uint_as_float(r[i] << 16);
                o[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
            }
        } else if constexpr (BYTES == 8) {
            const uint2 x = *reinterpret_cast<const uint2 *>(p);
            o[0] = __uint_as_float(x.x << 16); o[1] = __uint_as_float(x.x & 0xffff0000u);
            o[2] = __uint_as_float(x.y << 16); o[3] = __uint_as_float(x.y & 0xffff0000u);
        } else if constexpr (BYTES == 4) {
            const uint32_t x = *reinterpret_cast<const uint32_t *>(p);
            o[0] = __uint_as_float(x << 16); o[1] = __uint_as_float(x & 0xffff0000u);
        } else {
            static_assert(V == 1, "vector width");
            o[0] = to_f32(*p);
        }
    }
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T *p, const float (&o)[V]) {
    constexpr int BYTES = V * (int)sizeof(T);
    if constexpr (V == 1) {
        *p = from_f32<T>(o[0]);
    } else if constexpr (sizeof(T) == 4) {
        if constexpr (BYTES == 16) *reinterpret_cast<float4 *>(p) = make_float4(o[0], o[1], o[2], o[3]);
        else *reinterpret_cast<float2 *>(p) = make_float2(o[0], o[1]);
    } else {
        if constexpr (BYTES == 16)
            *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]),
                                                       pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7]));
        else if constexpr (BYTES == 8)
            *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]));
        else *reinterpret_cast<uint32_t *>(p) = pack_bf16(o[0], o[1]);
    }
}

// V consecutive elements as they lie in memory, and as floats: loads that are started ahead hold
// the fewest registers.
template <int BYTES>
struct RawType;
template <>
struct RawType<16> { using type = uint4; };
template <>
struct RawType<8> { using type = uint2; };
template <>
struct RawType<4> { using type = uint32_t; };
template <>
struct RawType<2> { using type = unsigned short; };
template <typename T, int V>
using Raw = typename RawType<V * (int)sizeof(T)>::type;

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load_raw(const T *p) { return *reinterpret_cast<const Raw<T, V> *>(p); }
template <typename T, int V>
__device__ __forceinline__ void unpack(const Raw<T, V> &r, float (&o)[V]) {
    load_vec<T, V>(reinterpret_cast<const T *>(&r), o);
}

// x + y in float32, what the addition lost added to `lost` (two-sum).
__device__ __forceinline__ void add_comp(float &x, float &lost, float y) {
    const float s = __fadd_rn(x, y), bb = __fadd_rn(s, -x);
    lost = __fadd_rn(lost, __fadd_rn(__fadd_rn(x, -__fadd_rn(s, -bb)), __fadd_rn(y, -bb)));
    x = s;
}

// Sum over the slices of partial sums part[slice][n] of column block * 32 + threadIdx.x % 32, for a CTA
// of 256 threads: eight threads take every eighth slice of a column, then their sums are added in
// order. Compensated float32: as exact as float64 here, whose rate on this GPU is a sixty-fourth. Valid
// in the first 32 threads.
__device__ __forceinline__ float slice_sum(const float *part, int slices, size_t n, unsigned block) {
    __shared__ float2 sums[8][32];
    const int col = threadIdx.x & 31, lane = threadIdx.x >> 5;
    const size_t i = (size_t)block * 32 + col;
    float a = 0.f, lost = 0.f;
    if (i < n)
#pragma unroll 4
        for (int s = lane; s < slices; s += 8) add_comp(a, lost, part[(size_t)s * n + i]);
    sums[lane][col] = make_float2(a, lost);
    __syncthreads();
    if (lane == 0)
#pragma unroll
        for (int k = 1; k < 8; ++k) {
            add_comp(a, lost, sums[k][col].x);
            lost += sums[k][col].y;
        }
    return lost == lost ? a + lost : a;            // a sum that is infinite has lost infinity - infinity
}

// Valid steps of batch row b.
__device__ __forceinline__ int row_length(const int *lens, int b, int T) {
    return lens == nullptr ? T : min(max(lens[b], 0), T);
}

}  // namespace gdn

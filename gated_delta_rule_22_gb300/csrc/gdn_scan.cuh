// gdn_scan.cuh -- what the selective state space scan's forward and backward kernels share
// (internal; not part of the C ABI).
//
// Layout of the work. The states of two channels lie on LPC neighbouring lanes (4, 8 or 16), four
// states of each channel on a lane, so that N up to 16, 32 or 64 states take one pass; a CTA holds CH =
// 256 / LPC channels of one group of one batch row and walks the steps in tiles of 16. The
// per-step inputs of a tile (d, d u, B, C and in the backward the cotangent) are staged in shared
// memory as float32: each is read by every lane that needs it as a broadcast, softplus is computed
// once per channel and step, and the global accesses of the channels-last tensors stay wide.
#pragma once

#include "gdn_layer.cuh"

namespace gdn {

constexpr int kScanThreads = 256;     // lanes of a CTA's channels at four states each
constexpr int kStateThreads = 128;    // of the forward that hold states: two channels each
constexpr int kScanHelpers = 128;     // of the forward that stage inputs and finish outputs

__device__ __forceinline__ void named_bar_arrive(int id, int n) {
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory");
}

template <int LPC>
struct ScanGeo {
    static constexpr int CH = kScanThreads / LPC;           // channels per CTA
    static constexpr int CPW = 32 / LPC;                    // channels per warp
    static constexpr int NP = 4 * LPC;                      // states per channel, padded
    static constexpr int V = CH * kScanTile / kScanThreads; // staged elements per thread (4, 2, 1)
    static constexpr int SP = CH + CPW;                     // pitch of a row of sums: no bank conflicts
};

// a = exp(d A) as exp2(d A log2 e). Near 1, where a state remembers 1 / (d |A|) steps, the hardware's
// exp2 is low by 1.8e-8 to 2.6e-8 on average (measured on [-0.1, -0.001]); a bias adds up over all of
// those steps, so the argument carries its opposite: the error of dA_log halves, at no cost.
constexpr float kExp2Centre = 2.5e-8f;
__device__ __forceinline__ float2 decay2(float2 d, float2 A2) {
    const float2 x = __ffma2_rn(d, A2, make_float2(kExp2Centre, kExp2Centre));
    return make_float2(ex2(x.x), ex2(x.y));
}
__device__ __forceinline__ float2 decay2(float d, float2 A2) { return decay2(make_float2(d, d), A2); }

// V staged elements as they were loaded. VEC: one access of V elements where all of them exist; the
// others one by one. They are turned into floats only where they are used, a tile later: an instruction
// that needs them earlier would wait for memory.
template <typename T, int V, bool VEC>
struct Staged {
    Raw<T, V> raw;
    __device__ __forceinline__ void load(const T *p, int n) {
        raw = Raw<T, V>();
        if (n > 0) raw = load_raw<T, V>(p);
    }
    __device__ __forceinline__ void get(float (&o)[V]) const { unpack<T, V>(raw, o); }
    __device__ __forceinline__ void keep(T *p) const { *reinterpret_cast<Raw<T, V> *>(p) = raw; }
};
template <typename T, int V>
struct Staged<T, V, false> {
    T e[V];
    __device__ __forceinline__ void load(const T *p, int n) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            e[v] = from_f32<T>(0.f);
            if (v < n) e[v] = p[v];
        }
    }
    __device__ __forceinline__ void get(float (&o)[V]) const {
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = to_f32(e[v]);
    }
    __device__ __forceinline__ void keep(T *p) const {
#pragma unroll
        for (int v = 0; v < V; ++v) p[v] = e[v];
    }
};
template <typename T, int V>
__device__ __forceinline__ void store_channels(T *p, int n, bool vec, const float (&o)[V]) {
    if (vec && n >= V) {
        store_vec<T, V>(p, o);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v < n) p[v] = from_f32<T>(o[v]);
    }
}

// The four states from position n0 on of a row of N float32 states (zeros past N).
__device__ __forceinline__ void load_states(const float *p, int n0, int N, float (&o)[4]) {
    if ((N & 3) == 0 && n0 < N) {
        const float4 x = *reinterpret_cast<const float4 *>(p + n0);
        o[0] = x.x; o[1] = x.y; o[2] = x.z; o[3] = x.w;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = n0 + k < N ? p[n0 + k] : 0.f;
    }
}
__device__ __forceinline__ void store_states(float *p, int n0, int N, const float (&o)[4]) {
    if ((N & 3) == 0) {
        if (n0 < N) *reinterpret_cast<float4 *>(p + n0) = make_float4(o[0], o[1], o[2], o[3]);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (n0 + k < N) p[n0 + k] = o[k];
    }
}

__device__ __forceinline__ float2 shfl2(float2 v, int m) {
    return make_float2(__shfl_xor_sync(kFullMask, v.x, m), __shfl_xor_sync(kFullMask, v.y, m));
}

// Sums four values (steps i0 .. i0 + 3) over the LPC lanes of a channel by exchanging halves: the
// lanes with lane % 4 = j get the sum of value j.
template <int LPC>
__device__ __forceinline__ float lane_sum4(const float (&v)[4], int lane) {
    const bool up2 = lane & 2, up1 = lane & 1;
    const float a = (up2 ? v[2] : v[0]) + __shfl_xor_sync(kFullMask, up2 ? v[0] : v[2], 2);
    const float b = (up2 ? v[3] : v[1]) + __shfl_xor_sync(kFullMask, up2 ? v[1] : v[3], 2);
    float r = (up1 ? b : a) + __shfl_xor_sync(kFullMask, up1 ? a : b, 1);
#pragma unroll
    for (int m = 4; m < LPC; m <<= 1) r += __shfl_xor_sync(kFullMask, r, m);
    return r;
}

template <int LPC>
__device__ __forceinline__ float2 lane_sum4(const float2 (&v)[4], int lane) {
    const bool up2 = lane & 2, up1 = lane & 1;
    const float2 a = __fadd2_rn(up2 ? v[2] : v[0], shfl2(up2 ? v[0] : v[2], 2));
    const float2 b = __fadd2_rn(up2 ? v[3] : v[1], shfl2(up2 ? v[1] : v[3], 2));
    float2 r = __fadd2_rn(up1 ? b : a, shfl2(up1 ? a : b, 1));
#pragma unroll
    for (int m = 4; m < LPC; m <<= 1) r = __fadd2_rn(r, shfl2(r, m));
    return r;
}

// The CTA's place: channels c0 .. c0 + nc of group g of batch row b, segment seg of the steps.
struct ScanPlace {
    int b, g, blk, c0, nc, seg, first, last;   // first, last: the segment's tiles [first, last)
};
template <int LPC>
__device__ __forceinline__ ScanPlace scan_place(const ScanParams &p) {
    constexpr int CH = ScanGeo<LPC>::CH;
    const int per = p.Cn / p.G, blocks = (per + CH - 1) / CH;
    ScanPlace q;
    q.seg = blockIdx.y;
    q.blk = blockIdx.x % blocks;
    const int bg = blockIdx.x / blocks;
    q.g = bg % p.G;
    q.b = bg / p.G;
    q.c0 = q.g * per + q.blk * CH;
    q.nc = min(CH, per - q.blk * CH);
    const int tiles = (p.T + kScanTile - 1) / kScanTile;
    q.first = q.seg * (p.seg_len / kScanTile);
    q.last = min(q.first + p.seg_len / kScanTile, tiles);
    return q;
}

// Whether V-wide accesses of the channels-last tensors are aligned everywhere.
template <typename T>
inline bool scan_vec(const ScanParams &p, int V) {
    const size_t a = V * sizeof(T);
    const int per = p.Cn / p.G;
    return per % V == 0 && p.ldu % V == 0 && p.lddt % V == 0 && p.ldz % V == 0 && (uintptr_t)p.u % a == 0 &&
           (uintptr_t)p.dt % a == 0 && (uintptr_t)p.z % a == 0;
}

// Turns the segments' end states (or start adjoints) into their incoming ones: in segment order
// (reverse: from the last), in = X, X = exp(A sum d) X + own. start may be null (zeros); the last X
// goes to `out` if not null.
cudaError_t launch_scan_combine(const ScanParams &p, const float *start, float *out, bool reverse, cudaStream_t s);

}  // namespace gdn

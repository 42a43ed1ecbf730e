// gdn_scan.cuh -- what the selective state space scan's forward and backward kernels share
// (internal; not part of the C ABI).
//
// Layout of the work. The states of one channel lie on LPC neighbouring lanes (4, 8 or 16), four
// states on each, so that N up to 16, 32 or 64 states take one pass; a CTA of 8 warps holds
// CH = 256 / LPC channels of one group of one batch row and walks the steps in tiles of 16. The
// per-step inputs of a tile (d, d u, B, C and in the backward the cotangent) are staged in shared
// memory as float32: each is read by every lane that needs it as a broadcast, softplus is computed
// once per channel and step, and the global accesses of the channels-last tensors stay wide.
#pragma once

#include "gdn_layer.cuh"

namespace gdn {

constexpr int kScanThreads = 256;
constexpr int kScanWarps = kScanThreads / 32;

template <int LPC>
struct ScanGeo {
    static constexpr int CH = kScanThreads / LPC;           // channels per CTA
    static constexpr int CPW = 32 / LPC;                    // channels per warp
    static constexpr int NP = 4 * LPC;                      // states per channel, padded
    static constexpr int V = CH * kScanTile / kScanThreads; // staged elements per thread (4, 2, 1)
    static constexpr int KB = NP * kScanTile / kScanThreads;// staged elements of B (of C) per thread
};

// V elements from channel position p on; those past `n` are zero.
template <typename T, int V>
__device__ __forceinline__ void load_channels(const T *p, int n, bool vec, float (&o)[V]) {
    if (vec && n >= V) {
        load_vec<T, V>(p, o);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = v < n ? to_f32(p[v]) : 0.f;
    }
}
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

// Sum over the LPC lanes of a channel.
template <int LPC>
__device__ __forceinline__ float lane_sum(float x) {
#pragma unroll
    for (int m = LPC / 2; m >= 1; m >>= 1) x += __shfl_xor_sync(kFullMask, x, m);
    return x;
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

// gdn_linear.cu -- matrix product with bias, activation and residual, and its gradients, on the
// tcgen05 tensor cores.
//
//     pre = x W^T + bias,  y = act(pre) + res
//     dpre = dy act'(pre),  dx = dpre W,  dW = dpre^T x,  dbias = sum_m dpre
//
// All three products are D[m][n] = sum_k A(m, k) B(n, k) with each operand either K-major (its rows
// are m or n, as x, W in the forward) or MN-major (its rows are k, as W in dx, dpre and x in dW):
// the tensor cores read both from what one TMA box puts into shared memory, so that nothing is
// transposed in memory.
//
// float32 operands are held as three bf16 terms (x = x0 + x1 + x2 exactly, each term the rest rounded to
// nearest: |x1| <= 2^-8 |x|, |x2| <= 2^-17 |x|, of either sign); six of the nine products of terms are
// summed, smallest first, by walking K once per product: the dropped ones are together below 2^-23.9 of
// the product, of either sign. Outputs that infinities make NaN on the way are formed again in float32.
// 2048 x 4096 x 8192 takes 0.8 ms, 0.085 of it for the terms: 173 TFLOP/s, where the CUDA cores' float32
// arithmetic ends at 75.
//
// Measured in bf16, 8192 x 2048 x 8192 with a residual: 153 us in short bursts, 1.80 PFLOP/s; 173 under
// the power cap when it runs on and on, 1.59 PFLOP/s (cuBLAS, measured the same ways, on a square case:
// 1.95 and 1.7). 16 x 8192 x 2048: 9 us, 3.7 TB/s of weights; 16 x 8192 x 8192: 27 us, 4.9 TB/s.
#include "gdn.h"
#include "gdn_layer.cuh"
#include "gdn_umma.cuh"

#include <algorithm>

namespace gdn {

namespace {

constexpr int kBM = 128, kBK = 64, kMaxBN = 256, kStages = 5;   // per CTA of a pair: 128 rows, 64 deep
constexpr int kPairs = 76;                          // pairs of SMs
constexpr int kEpiWarps = 8, kGemmThreads = 96 + 32 * kEpiWarps;   // + two fetching warps, one issuing
constexpr int kChunk = 32, kEpiPitch = kChunk + 4;  // columns an epilogue warp takes at once; floats per staged row
constexpr int kBox = 64 * kBK * 2;                  // one TMA box: 64 rows x 128 bytes
constexpr int kStageBytes = 4 * kBox;               // two boxes of A, two of B
constexpr size_t kGemmSmem = 1024 + (size_t)kStages * kStageBytes + kEpiWarps * 32 * kEpiPitch * 4 + 256;
constexpr int kBiasSlices = 128;
// K blocks per run of the tensor cores' accumulator, whose additions truncate: a sum of one sign loses some
// 1e-7 of itself per product of 16 (measured: 2.4 % over 4e6 rows). Each run's sum is added in float32
// with rounding. float32: short runs, added in registers, keep the error at that of float32
// arithmetic. bf16: a run of 4096 products loses at most some 4e-4, a fifth of the output's rounding; only
// K above 65536 takes more than one, added in the workspace, which costs (dW of 32768 x 2048 x 2048 cut
// into two runs: 169 us, 153 in one).
template <typename T>
constexpr int kRun = sizeof(T) == 4 ? 4 : 1024;

size_t up256(size_t n) { return (n + 255) / 256 * 256; }
int up8(int n) { return (n + 7) / 8 * 8; }

// The six products of the float32 terms (A's, B's), smallest first; bf16 has the last alone.
__constant__ signed char kTermA[6] = {0, 2, 1, 0, 1, 0}, kTermB[6] = {2, 0, 1, 1, 0, 0};

// What a pair of CTAs computes at once: rows m0 .. m0 + 255, columns n0 .. n0 + BN - 1. Items are
// numbered: whole tiles of 256 columns (within a panel of columns the columns first); then the tiles
// of an incomplete last round, cut into halves of 128 columns where that lets every pair take at most
// one; then the tiles of the last, narrower columns, of as many columns as are left (in 32s).
template <typename T>
constexpr int kTileN = sizeof(T) == 4 ? 128 : kMaxBN;   // columns of a whole tile

struct GemmParams {
    const void *bias, *res;
    void *out, *pre;
    float *partial;             // bf16, more than one run: the sum of the earlier ones, [32 rows][32 columns] in the lanes' order
    int *status;
    long long ldres;
    int M, N, kblocks, run, act;   // run: K blocks per accumulation
    int chunks;                 // partial: 32-column chunks of a row of tiles
    int mt, nt, panel;          // tiles along m and n (of 256 columns), n tiles walked together
    int whole, halves, edge;    // whole tiles, half tiles, columns of the edge tiles
    int light, light_edges;     // the first pair of those with the fewest other items, and the edge tiles that go to these alone
    int vec;                    // 16-byte accesses of out, pre and res are aligned
    int a_blocks, b_blocks;     // MN-major operands of whole 64-column blocks
    const __nv_bfloat16 *a, *b; // float32: the operands' terms, planes of rows of lda (ldb) elements, K terms deep
    size_t a_plane, b_plane;
    long long lda, ldb;
    int K;
};

// One output of a float32 product by a warp, in float32 arithmetic on the CUDA cores, for outputs that
// the six products made NaN: an infinity by a zero or opposite second or third term is not an infinity
// by the value. The sum ends early where it is NaN. Meant for few outputs: 2048 x 4096 x 8192 takes 0.78 ms
// where all sums are finite, 14 ms where everything is NaN, 0.34 s with an infinity in every row of x.
template <bool A_MN, bool B_MN>
__device__ __forceinline__ float dot_of_terms(const GemmParams &p, int m, int n) {
    const int lane = threadIdx.x & 31;
    auto value = [](const __nv_bfloat16 *t, size_t plane) {
        return __bfloat162float(t[0]) + (__bfloat162float(t[plane]) + __bfloat162float(t[2 * plane]));
    };
    float s = 0.f;
    for (int k0 = 0; k0 < p.K && !__any_sync(kFullMask, s != s); k0 += 32 * 8)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const size_t k = k0 + 32 * i + lane;
            if (k >= p.K) break;
            s = fmaf(value(p.a + (A_MN ? k * p.lda + m : m * p.lda + k), p.a_plane), value(p.b + (B_MN ? k * p.ldb + n : n * p.ldb + k), p.b_plane), s);
        }
    return warp_sum(s);
}

// The n-th item of a pair of CTAs; false behind its last. Whole and half tiles go round; so do the edge
// tiles, but the first ones only among the pairs that would otherwise end a round earlier.
template <int TN>
__device__ __forceinline__ bool item_of(const GemmParams &p, int n, int &m0, int &n0, int &BN) {
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1, main = p.whole + p.halves;
    int i = pair + n * pairs;
    if (i >= main) {
        const int k = n - (pair < main ? (main - pair + pairs - 1) / pairs : 0), lights = pairs - p.light;   // its k-th edge tile
        int e = p.edge > 0 ? 0 : p.mt, first = 0;
        if (pair >= p.light) {
            first = (p.light_edges - (pair - p.light) + lights - 1) / lights;      // its share of the first ones
            if (k < first) e = pair - p.light + k * lights;
        }
        if (k >= first) e += p.light_edges + pair + (k - first) * pairs;
        m0 = e * 2 * kBM;
        n0 = p.nt * TN;
        BN = p.edge;
        return e < p.mt;
    }
    BN = TN;
    const int t = i >= p.whole ? p.whole + (i - p.whole) / 2 : i;
    const int per = p.panel * p.mt, q = t / per, r = t % per, w = min(p.panel, p.nt - q * p.panel);
    m0 = r / w * 2 * kBM;
    n0 = (q * p.panel + r % w) * TN;
    if (i >= p.whole) {
        BN = TN / 2;
        n0 += (i - p.whole) % 2 * BN;
    }
    return true;
}

// ---- a pair of CTAs (cta_group::2): products issued by the even one read both CTAs' shared memory and
// write both CTAs' tensor memory
__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t leader_addr(const void *p) {      // the even CTA's copy of a shared variable
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(0));
    return a;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// a TMA load into this CTA's shared memory whose bytes count on a barrier of either CTA of the pair
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}
// One operand's tile of a stage: `boxes` boxes of 64 rows (or columns) from mn, K from k0. The number of
// copies is what counts: each costs its warp a few hundred cycles, so a tile is one copy wherever a
// map can describe it (an MN-major array of whole 64-column blocks: both boxes at once; `half` is the
// map of one box).
template <bool MN>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap *map, const CUtensorMap *half, bool blocks, int boxes,
                                          uint32_t bar, int mn, int k0, int term) {
    if (!MN) {
        tma_load_pair(dst, boxes == 2 ? map : half, bar, k0, mn, term);
    } else if (blocks) {
        tma_load_pair(dst, boxes == 2 ? map : half, bar, 0, k0, mn / 64, term);
    } else {
        tma_load_pair(dst, half, bar, mn, k0, term);
        if (boxes == 2) tma_load_pair(dst + kBox, half, bar, mn + 64, k0, term);
    }
}
__device__ __forceinline__ void pair_tmem_alloc(uint32_t *slot, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(ncols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void pair_umma_bf16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, bool accumulate,
                                               uint32_t lead) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"((uint32_t)accumulate), "r"(lead)
        : "memory");
}
// completion of the earlier products arrives once on both CTAs' copies of `bar`
__device__ __forceinline__ void pair_commit(uint64_t *bar, uint32_t lead) {
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
        " @q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %2;\n}" ::"r"(
            smem_addr(bar)),
        "r"(lead), "h"((unsigned short)3)
        : "memory");
}

// 128-byte swizzled operand descriptors. K-major: rows of 64 K elements, 8-row atoms 1024 bytes
// apart. MN-major: rows are K, 64 M/N elements wide; 8-row atoms 1024 bytes apart along K, the next
// 64 M/N elements one box (8192 bytes) further.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t start, bool mn) {
    return umma_sdesc(start, mn ? 8192u : 16u, 1024u) | (uint64_t)2 << 61;
}

__device__ __forceinline__ float act_rt(int act, float x) {
    return act == kActSilu ? silu_hw(x) : act == kActGelu ? gelu_f(x) : x;
}

}  // namespace

// A pair of CTAs shares each tile: CTA r holds rows 128 r .. 128 r + 127 of A's 256 and half of B's
// columns, so that each operand element is fetched into one SM only: with 128 x 256 tiles of single
// CTAs the tiles' way from L2 (27 TB/s at full rate) was the bound, 1.36 PFLOP/s. In each CTA warps 0
// and 2 fetch (TMA, kStages deep), warp 1 of the even CTA issues the products into one of two accumulators
// in tensor memory, and warps 3-10 turn the other one into output under the products of the next tile.
template <bool A_MN, bool B_MN, typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads, 1)
gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA_half,
            const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmB_half, const GemmParams p) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    float *stage_out = reinterpret_cast<float *>(smem + kStages * kStageBytes);
    uint64_t *bars = reinterpret_cast<uint64_t *>(stage_out + kEpiWarps * 32 * kEpiPitch);
    uint64_t *full = bars, *empty = bars + kStages, *acc_full = bars + 2 * kStages, *acc_empty = acc_full + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_empty + 2);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cta_rank();
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + i, 1);
            mbar_init(acc_empty + i, 2 * kEpiWarps);
        }
        fence_mbar_init();
        tma_prefetch_map(A_MN && !p.a_blocks ? &tmA_half : &tmA);
    }
    if (warp == 1) pair_tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    constexpr int TN = kTileN<T>, TERMS = sizeof(T) == 4 ? 6 : 1;
    griddep_launch();
    griddep_wait();                                // the set-up above ran under the previous kernel's end
    if (warp == 0 || warp == 2) {                  // one fetches A, the other B
        uint32_t it = 0;
        bool ok = true;
        if (lane == 0) {
            int st = 0;
            uint32_t phase = 1;
            int m0, n0, BN;
            for (int i = 0; ok && item_of<TN>(p, i, m0, n0, BN); ++i) {
                const int boxes = (BN / 2 + 63) / 64, am = m0 + rank * kBM, bn = n0 + rank * (BN / 2);
                for (int kr = 0; kr < p.kblocks && ok; kr += p.run)
                for (int term = 6 - TERMS; term < 6 && ok; ++term) {
                    const int ta = kTermA[term], tb = kTermB[term];
                    for (int k = kr; k < min(kr + p.run, p.kblocks); ++k, ++it) {
                        if (!(ok = mbar_wait(empty + st, phase))) {
                            report_status(p.status, kStatusTimeout);
                            break;
                        }
                        const uint32_t a = smem_addr(smem) + st * kStageBytes, bar = leader_addr(full + st);
                        if (warp == 0) {
                            if (rank == 0) mbar_expect_tx(full + st, 2 * (2 + boxes) * kBox);
                            load_tile<A_MN>(a, &tmA, &tmA_half, p.a_blocks, 2, bar, am, k * kBK, ta);
                        } else {
                            load_tile<B_MN>(a + 2 * kBox, &tmB, &tmB_half, p.b_blocks, boxes, bar, bn, k * kBK, tb);
                        }
                        if (++st == kStages) {
                            st = 0;
                            phase ^= 1;
                        }
                    }
                }
            }
            // copies that nothing has waited for (only after a wait ran out) land before the CTA ends
            if (!ok && rank == 0)
                for (uint32_t i = it < kStages ? 0 : it - kStages; i < it; ++i) mbar_wait(full + i % kStages, i / kStages & 1);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            const uint32_t lead = elect_one_sync();
            uint32_t n_tile = 0, phase = 0;
            int st = 0;
            bool ok = true;
            int m0, n0, BN;
            for (int i = 0; ok && item_of<TN>(p, i, m0, n0, BN); ++i) {
                const uint32_t idesc = umma_idesc_t(1, 2 * kBM, BN, A_MN, B_MN);
                for (int kr = 0; kr < p.kblocks && ok; kr += p.run, ++n_tile) {
                    const int acc = n_tile & 1, steps = min(p.run, p.kblocks - kr) * TERMS;
                    ok = mbar_wait(acc_empty + acc, (n_tile / 2 & 1) ^ 1);
                    tc_fence_after();
                    for (int s = 0; s < steps; ++s) {
                        ok = ok && mbar_wait(full + st, phase);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t base = smem_addr(smem) + st * kStageBytes;
                        uint64_t a = sw128_desc(base, A_MN), b = sw128_desc(base + 2 * kBox, B_MN);
#pragma unroll
                        for (int k = 0; k < kBK / 16; ++k) {
                            pair_umma_bf16(tmem + acc * kMaxBN, a, b, idesc, s > 0 || k > 0, lead);
                            a += A_MN ? 2048 >> 4 : 32 >> 4;
                            b += B_MN ? 2048 >> 4 : 32 >> 4;
                        }
                        pair_commit(empty + st, lead);
                        if (++st == kStages) {
                            st = 0;
                            phase ^= 1;
                        }
                    }
                    if (ok) pair_commit(acc_full + acc, lead);
                }
            }
            if (!ok && lane == 0) report_status(p.status, kStatusTimeout);
        }
    } else {
        const int quarter = warp & 3, half = (warp - 3) >> 2;      // tensor-memory lanes; chunks in turn
        float *mine = stage_out + (warp - 3) * 32 * kEpiPitch;
        const T *bias = static_cast<const T *>(p.bias), *res = static_cast<const T *>(p.res);
        T *out = static_cast<T *>(p.out), *pre = static_cast<T *>(p.pre);
        constexpr int V = 16 / sizeof(T), LPR = kChunk / V, RPP = 32 / LPR;   // columns per lane, lanes per row, rows per pass
        constexpr int CW = TN / (2 * kChunk);          // chunks of a tile per warp
        const int lr = lane / LPR, lc = lane % LPR * V;
        uint32_t n_tile = 0;
        bool ok = true, odd = false;               // odd: float32, a NaN among this lane's sums
        int m0, n0, BN;
        for (int i = 0; ok && item_of<TN>(p, i, m0, n0, BN); ++i) {
            const int row0 = m0 + rank * kBM + 32 * quarter, chunks = BN / kChunk;
            // the residual and bias of a chunk, loaded a chunk ahead
            Raw<T, V> next_res[LPR], next_bias;
            auto fetch = [&](int c) {
                const int col = n0 + c * kChunk + lc;
                const bool in = p.vec && c < chunks && col < p.N;
                next_bias = Raw<T, V>();
                if (in && bias != nullptr) next_bias = load_raw<T, V>(bias + col);
                if (res == nullptr) return;
#pragma unroll
                for (int h = 0; h < LPR; ++h) {
                    const int row = row0 + h * RPP + lr;
                    if (in && row < p.M) next_res[h] = load_raw<T, V>(res + (size_t)row * p.ldres + col);
                }
            };
            fetch(half);
            float sum[sizeof(T) == 4 ? CW : 1][kChunk];    // float32: the sum of the runs so far
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int k = 0; k < CW; ++k)
#pragma unroll
                    for (int j = 0; j < kChunk; ++j) sum[k][j] = 0.f;
            }
            uint32_t src = 0, drained = 0;
            auto begin_run = [&]() {
                const int acc = n_tile & 1;
                if (!mbar_wait(acc_full + acc, n_tile / 2 & 1)) {
                    if (lane == 0) report_status(p.status, kStatusTimeout);
                    return false;
                }
                ++n_tile;
                tc_fence_after();
                src = tmem + ((uint32_t)(32 * quarter) << 16) + acc * kMaxBN;
                drained = leader_addr(acc_empty + acc);
                return true;
            };
            auto end_run = [&]() {                     // this warp's last read of the accumulator is over
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_cluster(drained);
            };
            auto read = [&](int c, float2 (&v)[kChunk / 2]) {
                tmem_ld16(src + c * kChunk, *reinterpret_cast<float2(*)[8]>(v));
                tmem_ld16(src + c * kChunk + 16, *reinterpret_cast<float2(*)[8]>(v + 8));
            };
            if constexpr (sizeof(T) == 4) {
                for (int kr = p.run; kr < p.kblocks && ok; kr += p.run) {      // all runs but the last
                    if (!(ok = begin_run())) break;
#pragma unroll
                    for (int k = 0; k < CW; ++k) {
                        if (half + 2 * k >= chunks) continue;
                        float2 v[kChunk / 2];
                        read(half + 2 * k, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < kChunk / 2; ++j) {
                            sum[k][2 * j] += v[j].x;
                            sum[k][2 * j + 1] += v[j].y;
                        }
                    }
                    end_run();
                }
            }
            auto partial_at = [&](int c) {
                return reinterpret_cast<float4 *>(p.partial) + ((size_t)(row0 >> 5) * p.chunks + (n0 / kChunk + c)) * (kChunk * 8) + lane;
            };
            if constexpr (sizeof(T) == 2) {
                for (int kr = p.run; kr < p.kblocks && ok; kr += p.run) {
                    if (!(ok = begin_run())) break;
#pragma unroll 1
                    for (int c = half; c < chunks; c += 2) {
                        float2 v[kChunk / 2];
                        read(c, v);
                        tmem_wait_ld();
                        float4 *at = partial_at(c);
#pragma unroll
                        for (int j = 0; j < kChunk / 4; ++j) {
                            float4 x = make_float4(v[2 * j].x, v[2 * j].y, v[2 * j + 1].x, v[2 * j + 1].y);
                            if (kr > p.run) {
                                const float4 y = at[32 * j];
                                x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
                            }
                            at[32 * j] = x;
                        }
                    }
                    end_run();
                }
            }
            if (!ok || !(ok = begin_run())) break;
            if (half >= chunks) {
                end_run();
                continue;
            }
            float2 ahead[kChunk / 2];
            read(half, ahead);
            // one chunk; `acc` the float32 sum of the earlier runs
            auto finish = [&](int c, const float *acc) {
                tmem_wait_ld();
                // through shared memory, so that neighbouring lanes hold neighbouring columns
#pragma unroll
                for (int j = 0; j < kChunk / 4; ++j) {
                    float4 x = make_float4(ahead[2 * j].x, ahead[2 * j].y, ahead[2 * j + 1].x, ahead[2 * j + 1].y);
                    if constexpr (sizeof(T) == 4) {
                        x.x += acc[4 * j]; x.y += acc[4 * j + 1]; x.z += acc[4 * j + 2]; x.w += acc[4 * j + 3];
                        odd |= x.x != x.x || x.y != x.y || x.z != x.z || x.w != x.w;
                    } else if (p.partial != nullptr) {
                        const float4 y = partial_at(c)[32 * j];
                        x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
                    }
                    *reinterpret_cast<float4 *>(mine + lane * kEpiPitch + 4 * j) = x;
                }
                if (c + 2 < chunks) read(c + 2, ahead);
                else end_run();
                Raw<T, V> now_res[LPR], now_bias = next_bias;
#pragma unroll
                for (int h = 0; h < LPR; ++h) now_res[h] = next_res[h];
                fetch(c + 2);
                __syncwarp();
                const int col0 = n0 + c * kChunk;
                if (p.vec) {
                    float bs[V];
                    unpack<T, V>(now_bias, bs);
#pragma unroll
                    for (int h = 0; h < LPR; ++h) {
                        const int r = h * RPP + lr, col = col0 + lc;
                        const size_t row = row0 + r;
                        if (row >= p.M || col >= p.N) continue;
                        float o[V], e[V];
#pragma unroll
                        for (int j = 0; j < V / 4; ++j) {
                            const float4 x = *reinterpret_cast<const float4 *>(mine + r * kEpiPitch + lc + 4 * j);
                            o[4 * j] = x.x; o[4 * j + 1] = x.y; o[4 * j + 2] = x.z; o[4 * j + 3] = x.w;
                        }
#pragma unroll
                        for (int j = 0; j < V; ++j) o[j] += bs[j];
                        if (pre != nullptr) store_vec<T, V>(pre + row * p.N + col, o);
                        if (p.act == kActSilu) {
#pragma unroll
                            for (int j = 0; j < V; ++j) o[j] = silu_hw(o[j]);
                        } else if (p.act == kActGelu) {
#pragma unroll
                            for (int j = 0; j < V; ++j) o[j] = gelu_f(o[j]);
                        }
                        if (res != nullptr) {
                            unpack<T, V>(now_res[h], e);
#pragma unroll
                            for (int j = 0; j < V; ++j) o[j] = __fadd_rn(o[j], e[j]);
                        }
                        store_vec<T, V>(out + row * p.N + col, o);
                    }
                } else {
                    const int col = col0 + lane;
                    const float b = bias != nullptr && col < p.N ? to_f32(bias[col]) : 0.f;
                    constexpr int U = 8;               // rows whose residuals are loaded together
#pragma unroll 1
                    for (int r0 = 0; r0 < 32 && row0 + r0 < p.M && col < p.N; r0 += U) {
                        const size_t at = (size_t)(row0 + r0) * p.N + col;
                        const int rows = min(U, p.M - row0 - r0);
                        T e[U];
                        if (res != nullptr)
#pragma unroll
                            for (int r = 0; r < U; ++r)
                                if (r < rows) e[r] = res[(size_t)(row0 + r0 + r) * p.ldres + col];
#pragma unroll
                        for (int r = 0; r < U; ++r) {
                            if (r >= rows) break;
                            float o = mine[(r0 + r) * kEpiPitch + lane] + b;
                            if (pre != nullptr) pre[at + (size_t)r * p.N] = from_f32<T>(o);
                            o = act_rt(p.act, o);
                            if (res != nullptr) o = __fadd_rn(o, to_f32(e[r]));
                            out[at + (size_t)r * p.N] = from_f32<T>(o);
                        }
                    }
                }
                __syncwarp();
            };
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int k = 0; k < CW; ++k)
                    if (half + 2 * k < chunks) finish(half + 2 * k, sum[k]);
            } else {
#pragma unroll 1
                for (int c = half; c < chunks; c += 2) finish(c, nullptr);
            }
        }
        if constexpr (sizeof(T) == 4) {
            // the warp's NaN outputs once more (nothing waits for this with a limit: the products are over)
            if (__any_sync(kFullMask, odd && ok))
                for (int i = 0; item_of<TN>(p, i, m0, n0, BN); ++i)
                    for (int c = half; c < BN / kChunk; c += 2)
                        for (int r = 0; r < 32; ++r) {
                            const int row = m0 + rank * kBM + 32 * quarter + r, col = n0 + c * kChunk + lane;
                            const bool in = row < p.M && col < p.N;
                            const float is = in ? out[(size_t)row * p.N + col] : 0.f;
                            for (unsigned nan = __ballot_sync(kFullMask, is != is); nan != 0; nan &= nan - 1) {
                                const int who = __ffs(nan) - 1;
                                float o = dot_of_terms<A_MN, B_MN>(p, row, col - lane + who);
                                if (lane != who) continue;
                                if (bias != nullptr) o += bias[col];
                                if (pre != nullptr) pre[(size_t)row * p.N + col] = o;
                                o = act_rt(p.act, o);
                                if (res != nullptr) o = __fadd_rn(o, res[(size_t)row * p.ldres + col]);
                                out[(size_t)row * p.N + col] = o;
                            }
                        }
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();                                // the pair's products and arrivals are over
    tc_fence_after();
    if (warp == 1) pair_tmem_dealloc(tmem, 512);
}

// ---- few rows (decode): a stream over the weights
//
// With up to 64 rows the product is bound by the bytes of W. It is computed the other way round, D[n][m]
// = W x^T: 128 rows of W are the tensor cores' M, the rows of x (padded to 16, 32 or 64) their N. The
// CTAs of a cluster share one tile of W's rows, each with its part of K, so that every SM streams; their
// partial sums meet in shared memory (cluster rank order) and each CTA finishes its share of the rows.
constexpr int kTokThreads = 64 + 128;

template <int MP>
struct TokGeo {
    static constexpr int kStage = 2 * kBox + MP * kBK * 2;
    static constexpr int kDepth = MP == 16 ? 6 : MP == 32 ? 5 : 4;      // two CTAs' stages fit one SM
    static constexpr size_t kSmem = 1024 + (size_t)kDepth * kStage + 256;
    static_assert(128 * MP * 4 <= kDepth * kStage, "the partial sums take the stages' place");
};

struct TokenParams {
    const void *bias, *res;
    void *out, *pre;
    int *status;
    long long ldres;
    int M, N, kblocks, per, act;     // per: K blocks of one CTA
};

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_addr(bar))
        : "memory");
}

template <int MP>
__global__ void __launch_bounds__(kTokThreads) linear_token_kernel(const __grid_constant__ CUtensorMap tmW,
                                                                   const __grid_constant__ CUtensorMap tmX, const TokenParams p) {
    using T = __nv_bfloat16;
    using G = TokGeo<MP>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    float *partial = reinterpret_cast<float *>(smem);               // [MP][128], over the stages
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + G::kDepth * G::kStage);
    uint64_t *full = bars, *empty = bars + G::kDepth, *done = empty + G::kDepth;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int splits = gridDim.x, rank = blockIdx.x, n0 = blockIdx.y * 128;
    const int k_first = rank * p.per, steps = max(min(p.per, p.kblocks - k_first), 0);
    if (threadIdx.x == 0) {
        for (int i = 0; i < G::kDepth; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        mbar_init(done, 1);
        fence_mbar_init();
        tma_prefetch_map(&tmW);
        tma_prefetch_map(&tmX);
    }
    if (warp == 1) tmem_alloc(tmem_slot, MP < 32 ? 32 : MP);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (warp == 0) {
        if (lane == 0) {
            bool ok = true;
            int s = 0;
            for (; s < steps; ++s) {
                const int st = s % G::kDepth;
                if (!(ok = mbar_wait(empty + st, (s / G::kDepth & 1) ^ 1))) break;
                unsigned char *w = smem + st * G::kStage;
                mbar_expect_tx(full + st, G::kStage);
                tma_load_3d(w, &tmW, full + st, (k_first + s) * kBK, n0, 0);
                tma_load_3d(w + 2 * kBox, &tmX, full + st, (k_first + s) * kBK, 0, 0);
            }
            if (!ok) {                            // what was started lands before the CTA ends
                report_status(p.status, kStatusTimeout);
                for (int i = s < G::kDepth ? 0 : s - G::kDepth; i < s; ++i) mbar_wait(full + i % G::kDepth, i / G::kDepth & 1);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        const uint32_t lead = elect_one_sync();
        const uint32_t idesc = umma_idesc(1, 128, MP);
        bool ok = true;
        for (int s = 0; s < steps; ++s) {
            const int st = s % G::kDepth;
            if (!(ok = mbar_wait(full + st, s / G::kDepth & 1))) break;
            tc_fence_after();
            const uint32_t base = smem_addr(smem) + st * G::kStage;
            uint64_t a = sw128_desc(base, false), b = sw128_desc(base + 2 * kBox, false);
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k) {
                umma_bf16_w(tmem, a, b, idesc, s > 0 || k > 0, lead);
                a += 32 >> 4;
                b += 32 >> 4;
            }
            umma_commit_w(empty + st, lead);
        }
        if (ok) umma_commit_w(done, lead);
        else if (lane == 0) report_status(p.status, kStatusTimeout);
    } else {
        const int quarter = warp & 3;
        bool ok = true;
        if (steps > 0 && !(ok = mbar_wait(done, 0)) && lane == 0) report_status(p.status, kStatusTimeout);
        tc_fence_after();
        // every product has read its stage: the partial sums go there, [m][row of W]
#pragma unroll
        for (int c = 0; c < MP; c += 16) {
            float2 v[8];
            if (steps > 0 && ok) {
                tmem_ld16(tmem + ((uint32_t)(32 * quarter) << 16) + c, v);
                tmem_wait_ld();
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = make_float2(0.f, 0.f);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                partial[(c + 2 * j) * 128 + 32 * quarter + lane] = v[j].x;
                partial[(c + 2 * j + 1) * 128 + 32 * quarter + lane] = v[j].y;
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    cluster_sync();
    const int rows = 128 / splits, mine = rank * rows;
    const T *bias = static_cast<const T *>(p.bias), *res = static_cast<const T *>(p.res);
    for (int e = threadIdx.x; e < rows * p.M; e += kTokThreads) {
        const int r = mine + e % rows, m = e / rows, n = n0 + r;
        if (n >= p.N) continue;
        const uint32_t at = smem_addr(partial + m * 128 + r);
        float v = 0.f;
        for (int k = 0; k < splits; ++k) {
            uint32_t remote;
            float x;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(at), "r"(k));
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(remote));
            v += x;
        }
        if (bias != nullptr) v += to_f32(bias[n]);
        const size_t o = (size_t)m * p.N + n;
        if (p.pre != nullptr) static_cast<T *>(p.pre)[o] = from_f32<T>(v);
        v = act_rt(p.act, v);
        if (res != nullptr) v = __fadd_rn(v, to_f32(res[(size_t)m * p.ldres + n]));
        static_cast<T *>(p.out)[o] = from_f32<T>(v);
    }
    __syncthreads();                              // the loop above leaves warps divided; the cluster's barrier is for whole ones
    cluster_sync();                               // nobody leaves while its partial sums are read
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, MP < 32 ? 32 : MP);
    }
}

// Few rows of float32, or of bf16 that TMA cannot read in place: the same stream on the CUDA cores. A
// warp takes four rows of W and a slice of K, with MT rows of x at a time; `slices` warps of a CTA share
// four rows of W.
template <typename T, int V, int MT>
__global__ void __launch_bounds__(256) linear_stream_kernel(const T *x, long long ldx, const T *W, long long ldw, const T *bias,
                                                            const T *res, long long ldres, T *out, T *pre, int M, int N, int K,
                                                            int act, int slices) {
    __shared__ float sums[8][4][MT];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = warp / slices, slice = warp % slices;
    const int n0 = (blockIdx.x * (8 / slices) + group) * 4, m0 = blockIdx.y * MT;
    const int steps = (K + 32 * V - 1) / (32 * V), per = (steps + slices - 1) / slices;
    float acc[4][MT];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[r][m] = 0.f;
    Raw<T, V> next[4];
    auto fetch = [&](int s) {
        const int k = (s * 32 + lane) * V;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            next[r] = Raw<T, V>();
            if (k < K && n0 + r < N) next[r] = load_raw<T, V>(W + (size_t)(n0 + r) * ldw + k);
        }
    };
    const int first = slice * per, last = min(first + per, steps);
    if (first < last) fetch(first);
    for (int s = first; s < last; ++s) {
        float w[4][V];
#pragma unroll
        for (int r = 0; r < 4; ++r) unpack<T, V>(next[r], w[r]);
        if (s + 1 < last) fetch(s + 1);
        const int k = (s * 32 + lane) * V;
        if (k >= K) continue;
#pragma unroll
        for (int m = 0; m < MT; ++m) {                 // rows past the last repeat it: no branch in the stream
            float e[V];
            load_vec<T, V>(x + (size_t)min(m0 + m, M - 1) * ldx + k, e);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int v = 0; v < V; ++v) acc[r][m] = fmaf(w[r][v], e[v], acc[r][m]);
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const float t = warp_sum(acc[r][m]);
            if (lane == 0) sums[warp][r][m] = t;
        }
    __syncthreads();
    for (int e = threadIdx.x; e < 8 / slices * 4 * MT; e += 256) {
        const int g = e / (4 * MT), r = e % 4, m = e / 4 % MT, n = (blockIdx.x * (8 / slices) + g) * 4 + r;
        if (n >= N || m0 + m >= M) continue;
        float v = 0.f;
        for (int k = 0; k < slices; ++k) v += sums[g * slices + k][r][m];
        if (bias != nullptr) v += to_f32(bias[n]);
        const size_t o = (size_t)(m0 + m) * N + n;
        if (pre != nullptr) pre[o] = from_f32<T>(v);
        v = act_rt(act, v);
        if (res != nullptr) v = __fadd_rn(v, to_f32(res[(size_t)(m0 + m) * ldres + n]));
        out[o] = from_f32<T>(v);
    }
}

// x as bf16 operand rows of `cols8` elements: a copy (bf16) or three terms (float32), planes of
// [rows][cols8]. What lies past the `cols` columns is never read.
__device__ __forceinline__ void split3(float x, __nv_bfloat16 (&t)[3]) {
    // the largest values, which would round to infinity, are cut
    t[0] = fabsf(x) < 0x1.ffp127f ? __float2bfloat16_rn(x) : __float2bfloat16_rz(x);
    const float r = x - __bfloat162float(t[0]);
    const bool fine = r - r == 0.f;                // an infinity or NaN stays in the first term
    t[1] = __float2bfloat16_rn(fine ? r : 0.f);
    t[2] = __float2bfloat16_rn(fine ? r - __bfloat162float(t[1]) : 0.f);
}
// V elements of a row, as the operand's planes from `out` on (`plane` elements apart)
template <typename T, int V>
__device__ __forceinline__ void store_operand(__nv_bfloat16 *out, size_t plane, const float (&x)[V]) {
    if constexpr (sizeof(T) == 2) {
        store_vec<__nv_bfloat16, V>(out, x);
    } else {
        __nv_bfloat16 t[V][3];
#pragma unroll
        for (int v = 0; v < V; ++v) split3(x[v], t[v]);
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            float e[V];                                // exact: terms are bf16
#pragma unroll
            for (int v = 0; v < V; ++v) e[v] = __bfloat162float(t[v][i]);
            store_vec<__nv_bfloat16, V>(out + i * plane, e);
        }
    }
}
template <typename T, int V>
__global__ void __launch_bounds__(256) linear_pack_kernel(const T *x, long long ld, __nv_bfloat16 *out, int rows, int cols, int cols8) {
    griddep_launch();
    griddep_wait();
    const int c = (blockIdx.x * 256 + threadIdx.x) * V;
    if (c >= cols) return;
    const size_t plane = (size_t)rows * cols8;
    int r = blockIdx.y;
    constexpr int U = 4;                               // rows in flight per thread
    for (; r + (U - 1) * (int)gridDim.y < rows; r += U * gridDim.y) {
        Raw<T, V> in[U];
#pragma unroll
        for (int i = 0; i < U; ++i) in[i] = load_raw<T, V>(x + (size_t)(r + i * gridDim.y) * ld + c);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            float e[V];
            unpack<T, V>(in[i], e);
            store_operand<T, V>(out + (size_t)(r + i * gridDim.y) * cols8 + c, plane, e);
        }
    }
    for (; r < rows; r += gridDim.y) {
        float e[V];
        load_vec<T, V>(x + (size_t)r * ld + c, e);
        store_operand<T, V>(out + (size_t)r * cols8 + c, plane, e);
    }
}

// dpre = dy act'(pre) as an operand (null: dy is used as it is), and each slice of rows' column sums.
// The rounding of dpre to bf16 is the operand format's; the bias sums take it before that. A CTA takes
// 64 V columns and four rows at a time.
template <typename T, int V>
__global__ void __launch_bounds__(256) linear_dpre_kernel(const T *dy, const T *pre, __nv_bfloat16 *dpre, float *part, int M,
                                                          int N, int N8, int act) {
    __shared__ float sums[4][64 * V];
    griddep_launch();
    griddep_wait();
    const int cg = threadIdx.x & 63, rl = threadIdx.x >> 6, n = (blockIdx.x * 64 + cg) * V;
    float s[V] = {};
    if (n < N) {
        const size_t plane = (size_t)M * N8;
        const int step = 4 * gridDim.y;
        Raw<T, V> next_d = Raw<T, V>(), next_p = Raw<T, V>();
        auto fetch = [&](int m) {
            if (m >= M) return;
            next_d = load_raw<T, V>(dy + (size_t)m * N + n);
            if (act != kActNone) next_p = load_raw<T, V>(pre + (size_t)m * N + n);
        };
        int m = blockIdx.y * 4 + rl;
        fetch(m);
        for (; m < M; m += step) {
            float d[V], q[V];
            unpack<T, V>(next_d, d);
            unpack<T, V>(next_p, q);
            fetch(m + step);
            if (act == kActSilu) {
#pragma unroll
                for (int v = 0; v < V; ++v) d[v] *= dsilu_hw(q[v]);
            } else if (act == kActGelu) {
#pragma unroll
                for (int v = 0; v < V; ++v) d[v] *= dgelu_f(q[v]);
            }
            if (dpre != nullptr) store_operand<T, V>(dpre + (size_t)m * N8 + n, plane, d);
#pragma unroll
            for (int v = 0; v < V; ++v) s[v] += d[v];
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) sums[rl][cg * V + v] = s[v];
    __syncthreads();
    for (int i = threadIdx.x; i < 64 * V; i += 256) {
        const int c = blockIdx.x * 64 * V + i;
        if (c < N) part[(size_t)blockIdx.y * N + c] = (sums[0][i] + sums[1][i]) + (sums[2][i] + sums[3][i]);
    }
}

template <typename T>
__global__ void __launch_bounds__(256) linear_dbias_kernel(const float *part, T *dbias, int slices, int N) {
    griddep_launch();
    griddep_wait();
    const int n = blockIdx.x * 32 + threadIdx.x;
    const float s = slice_sum(part, slices, N, blockIdx.x);
    if (threadIdx.x < 32 && n < N) dbias[n] = from_f32<T>(s);
}

namespace {

// Room for an operand's copy: float32 terms always, bf16 where TMA cannot read it in place (rows not
// a multiple of 16 bytes apart) or might not be able to (a slice or a single row, whose address may be
// unaligned).
size_t pack_bytes(long long rows, int cols, long long ld, int dtype) {
    if (dtype == 0) return up256((size_t)3 * rows * up8(cols) * 2);
    return ld % 8 != 0 || ld != cols || rows == 1 ? up256((size_t)rows * up8(cols) * 2) : 0;
}

struct Operand {
    const void *p;
    long long ld;
    int rows, cols;
};

// The operand as TMA can read it, copied to ws where it has to be.
int pack(const Operand &in, Operand *out, char *ws, int dtype, cudaStream_t s) {
    *out = in;
    if (dtype != 0 && in.ld % 8 == 0 && (uintptr_t)in.p % 16 == 0) return 0;
    __nv_bfloat16 *to = reinterpret_cast<__nv_bfloat16 *>(ws);
    const int cols8 = up8(in.cols);
    timing_mark("linear_pack", 0, s);
    auto launch = [&](auto kernel, auto *src, int V) {
        const int cols = (in.cols / V + 255) / 256, most = (kPairs * 2 * 16 + cols - 1) / cols;
        return launch_pdl(kernel, dim3(cols, in.rows < most ? in.rows : most), dim3(256), 0, s, src, in.ld, to, in.rows, in.cols, cols8);
    };
    cudaError_t e;
    if (dtype == 0) {
        const float *src = static_cast<const float *>(in.p);
        if (in.cols % 4 == 0 && in.ld % 4 == 0 && (uintptr_t)in.p % 16 == 0) e = launch(linear_pack_kernel<float, 4>, src, 4);
        else e = launch(linear_pack_kernel<float, 1>, src, 1);
    } else {
        const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(in.p);
        if (in.cols % 2 == 0 && in.ld % 2 == 0 && (uintptr_t)in.p % 4 == 0) e = launch(linear_pack_kernel<__nv_bfloat16, 2>, src, 2);
        else e = launch(linear_pack_kernel<__nv_bfloat16, 1>, src, 1);
    }
    timing_mark("linear_pack", 1, s);
    out->p = to;
    out->ld = cols8;
    return api_cuda_status(e);
}

struct Epilogue {
    const void *bias, *res;
    long long ldres;
    int act;
    void *out, *pre;
    float *partial;             // partial_bytes
};

// Sums of a product's earlier runs (bf16).
size_t partial_bytes(long long M, long long N, long long K, int dtype) {
    if (dtype == 0 || K <= (long long)kRun<__nv_bfloat16> * kBK) return 0;
    return (size_t)((M + 2 * kBM - 1) / (2 * kBM) * (2 * kBM)) * ((N + 127) / 128 * 128) * 4;
}

template <bool A_MN, bool B_MN, typename T>
int gemm(const char *name, const Operand &A, const Operand &B, int M, int N, int K, const Epilogue &e, int *status, cudaStream_t s) {
    GemmParams p = {};
    p.bias = e.bias; p.res = e.res; p.ldres = e.ldres; p.act = e.act; p.out = e.out; p.pre = e.pre; p.status = status;
    p.M = M; p.N = N; p.K = K;
    p.a = static_cast<const __nv_bfloat16 *>(A.p); p.lda = A.ld; p.a_plane = (size_t)A.rows * A.ld;
    p.b = static_cast<const __nv_bfloat16 *>(B.p); p.ldb = B.ld; p.b_plane = (size_t)B.rows * B.ld;
    p.kblocks = (K + kBK - 1) / kBK;
    const int planes = sizeof(T) == 4 ? 3 : 1;
    p.run = p.kblocks < kRun<T> ? p.kblocks : kRun<T>;
    p.partial = sizeof(T) == 2 && p.kblocks > p.run ? e.partial : nullptr;
    constexpr int TN = kTileN<T>;
    // a product with an odd number of columns left gets narrower tiles at the end
    p.mt = (M + 2 * kBM - 1) / (2 * kBM);
    p.nt = N / TN;
    const int unit = B_MN && B.cols % 64 == 0 ? 128 : 32;   // each CTA's half starts on a 64-column block
    p.edge = (N % TN + unit - 1) / unit * unit;
    p.chunks = (p.nt * TN + p.edge) / kChunk;
    // panels of 8 tiles of columns: a round's tiles then share rows of both operands in L2 (8192 x 2048 x
    // 8192: 171 us sustained with panels of 8, 181 of 1; the products of a gradient of 4100 x 2056 x 2040,
    // with edge tiles dealt round as well, 39 and 38 us against 53 and 62)
    p.panel = p.nt < 8 ? (p.nt > 0 ? p.nt : 1) : 8;
    const long long tiles = (long long)p.mt * p.nt;
    const int last = (int)(tiles % kPairs);            // tiles of an incomplete last round
    if (tiles > 0x3fffffffLL) return GDN_ERR_UNSUPPORTED_SHAPE;
    // halves, where each pair then takes at most one: 155 us instead of 164 for 8192 x 2048 x 8192, whose
    // fourth round has 28 tiles
    p.halves = TN == kMaxBN && last > 0 && last <= kPairs / 2 ? 2 * last : 0;
    p.whole = (int)tiles - p.halves / 2;
    const int items = p.whole + p.halves + (p.edge > 0 ? p.mt : 0), pairs = items < kPairs ? items : kPairs;
    // an edge tile costs about (its columns + 64) / 320 of a whole one: that many fit into a round
    p.light = (p.whole + p.halves) % pairs;
    const int room = (pairs - p.light) * (320 / (p.edge + 64));
    p.light_edges = p.edge == 0 ? 0 : p.mt < room ? p.mt : room;
    const int V = 16 / (int)sizeof(T);
    p.vec = N % V == 0 && (uintptr_t)e.res % 16 == 0 && e.ldres % V == 0;
    CUtensorMap tm[4] = {};                            // A, one box of A, B, one box of B: those in use
    const bool a_blocks = A_MN && A.cols % 64 == 0, b_blocks = B_MN && B.cols % 64 == 0;
    const bool a_boxes = A_MN && !a_blocks, b_boxes = B_MN && !b_blocks;
    const bool use[4] = {!a_boxes, a_boxes, !b_boxes && (p.whole > 0 || p.edge > 128),
                         b_boxes || p.halves > 0 || (p.edge > 0 && p.edge <= 128) || TN <= 128};
    p.a_blocks = a_blocks;
    p.b_blocks = b_blocks;
    int rc;
    for (int i = 0; i < 4; ++i) {
        const Operand &o = i < 2 ? A : B;
        const bool mn = i < 2 ? A_MN : B_MN, blocks = i < 2 ? a_blocks : b_blocks;
        const int boxes = 2 - i % 2;
        if (use[i] && (rc = api_planes_map(&tm[i], o.p, o.cols, o.rows, planes, o.ld, mn ? kBK : 64 * boxes, blocks ? boxes : 0)) != 0)
            return rc;
    }
    cudaError_t err = allow_smem<gemm_kernel<A_MN, B_MN, T>>((int)kGemmSmem);
    if (err != cudaSuccess) return api_cuda_status(err);
    timing_mark(name, 0, s);
    err = launch_pdl(gemm_kernel<A_MN, B_MN, T>, dim3(2 * pairs), dim3(kGemmThreads), kGemmSmem, s, tm[0],
                     tm[1], tm[2], tm[3], p);
    timing_mark(name, 1, s);
    return api_cuda_status(err);
}

constexpr int kNotTaken = 1;

template <int MP>
int token_launch(const LinearParams &p, cudaStream_t s) {
    using G = TokGeo<MP>;
    TokenParams t = {p.bias, p.res, p.y, p.pre, p.status, p.ldres, p.M, p.N, (p.K + kBK - 1) / kBK, 0, p.act};
    const int tiles = (p.N + 127) / 128;
    // at most two CTAs per SM, at least two K blocks each (64 rows, 8192 x 2048: 13 us, 27 by one CTA per tile)
    int splits = 8;
    while (splits > 1 && (tiles * splits > 4 * kPairs || t.kblocks < 2 * splits)) splits /= 2;
    while ((t.kblocks + splits - 1) / splits > kRun<__nv_bfloat16>) splits *= 2;     // up to 8: see token_any
    t.per = (t.kblocks + splits - 1) / splits;
    CUtensorMap w, x;
    int rc;
    if ((rc = api_planes_map(&w, p.W, p.K, p.N, 1, p.ldw, 128, 0)) != 0) return rc;
    if ((rc = api_planes_map(&x, p.x, p.K, p.M, 1, p.ldx, MP, 0)) != 0) return rc;
    cudaError_t e = allow_smem<linear_token_kernel<MP>>((int)G::kSmem);
    if (e != cudaSuccess) return api_cuda_status(e);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(splits, tiles);
    cfg.blockDim = kTokThreads;
    cfg.dynamicSmemBytes = G::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = splits;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    timing_mark("linear_token", 0, s);
    e = cudaLaunchKernelEx(&cfg, linear_token_kernel<MP>, w, x, t);
    timing_mark("linear_token", 1, s);
    return api_cuda_status(e);
}

template <typename T, int V, int MT>
int stream_launch(const LinearParams &p, cudaStream_t s) {
    const int groups = (p.N + 3) / 4, steps = (p.K + 32 * V - 1) / (32 * V);
    int slices = 1;                                    // warps per four rows: until there are 16 warps per SM
    while (slices < 8 && groups * slices < 2 * kPairs * 16 && steps >= 4 * slices) slices *= 2;
    const int per = 8 / slices;
    timing_mark("linear_stream", 0, s);
    linear_stream_kernel<T, V, MT><<<dim3((groups + per - 1) / per, (p.M + MT - 1) / MT), 256, 0, s>>>(
        static_cast<const T *>(p.x), p.ldx, static_cast<const T *>(p.W), p.ldw, static_cast<const T *>(p.bias),
        static_cast<const T *>(p.res), p.ldres, static_cast<T *>(p.y), static_cast<T *>(p.pre), p.M, p.N, p.K, p.act, slices);
    timing_mark("linear_stream", 1, s);
    return api_cuda_status(cudaGetLastError());
}
template <typename T, int V>
int stream_rows(const LinearParams &p, cudaStream_t s) {
    return p.M <= 2 ? stream_launch<T, V, 2>(p, s) : p.M <= 4 ? stream_launch<T, V, 4>(p, s)
         : p.M <= 8 ? stream_launch<T, V, 8>(p, s) : stream_launch<T, V, 16>(p, s);
}

// The decode forms: bf16 rows that TMA reads in place, up to 64 of them, on the tensor cores (weights of
// 8192 x 2048: 16 rows 9 us, 18 by the tiles of 256 rows; 64 rows 13 us, 15); else, up to 32 (beyond that
// packing W for the tensor cores costs less than streaming it more than twice), on the CUDA cores (float32
// weights of the same size: 16 rows 51 us, 79 packed; 32 rows 83 us, 81).
template <typename T>
int token_any(const LinearParams &p, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    const uintptr_t at = (uintptr_t)p.x | (uintptr_t)p.W;
    const bool short_runs = p.K <= 8 * kRun<__nv_bfloat16> * kBK;      // of each of a cluster's CTAs
    if (sizeof(T) == 2 && p.M <= 64 && short_runs && p.ldx % 8 == 0 && p.ldw % 8 == 0 && at % 16 == 0)
        return p.M <= 16 ? token_launch<16>(p, s) : p.M <= 32 ? token_launch<32>(p, s) : token_launch<64>(p, s);
    if (p.M > kLinearFewRows) return kNotTaken;
    const bool vec = p.K % V == 0 && p.ldx % V == 0 && p.ldw % V == 0 && at % 16 == 0;
    return vec ? stream_rows<T, V>(p, s) : stream_rows<T, 1>(p, s);
}

template <typename T>
int fwd_any(const LinearParams &p, int dtype, cudaStream_t s) {
    const int few = token_any<T>(p, s);
    if (few != kNotTaken) return few;
    Operand x = {p.x, p.ldx, p.M, p.K}, w = {p.W, p.ldw, p.N, p.K};
    char *ws = p.ws;
    int rc;
    if ((rc = pack(x, &x, ws, dtype, s)) != 0) return rc;
    ws += pack_bytes(p.M, p.K, p.ldx, dtype);
    if ((rc = pack(w, &w, ws, dtype, s)) != 0) return rc;
    float *partial = reinterpret_cast<float *>(ws + pack_bytes(p.N, p.K, p.ldw, dtype));
    return gemm<false, false, T>("linear_fwd", x, w, p.M, p.N, p.K, {p.bias, p.res, p.ldres, p.act, p.y, p.pre, partial}, p.status, s);
}

template <typename T>
int bwd_any(const LinearParams &p, int dtype, cudaStream_t s) {
    Operand x = {p.x, p.ldx, p.M, p.K}, w = {p.W, p.ldw, p.N, p.K}, d = {p.dy, p.N, p.M, p.N};
    char *ws = p.ws;
    float *part = reinterpret_cast<float *>(ws);
    ws += up256((size_t)kBiasSlices * p.N * 4);
    const bool own_dpre = dtype == 0 || p.act != kActNone || p.N % 8 != 0;
    int rc;
    if (own_dpre || p.dbias != nullptr) {
        __nv_bfloat16 *to = own_dpre ? reinterpret_cast<__nv_bfloat16 *>(ws) : nullptr;
        constexpr int V = 16 / (int)sizeof(T);
        const T *dy = static_cast<const T *>(p.dy), *pre = static_cast<const T *>(p.pre_in);
        const int slices = (p.M + 3) / 4 < kBiasSlices ? (p.M + 3) / 4 : kBiasSlices;
        timing_mark("linear_dpre", 0, s);
        auto launch = [&](auto kernel, int v) {
            return launch_pdl(kernel, dim3((p.N + 64 * v - 1) / (64 * v), slices), dim3(256), 0, s, dy, pre, to, part, p.M, p.N, up8(p.N), p.act);
        };
        cudaError_t e = p.N % V == 0 ? launch(linear_dpre_kernel<T, V>, V) : launch(linear_dpre_kernel<T, 1>, 1);
        timing_mark("linear_dpre", 1, s);
        if ((rc = api_cuda_status(e)) != 0) return rc;
        if (to != nullptr) d = {to, up8(p.N), p.M, p.N};
        if (p.dbias != nullptr) {
            timing_mark("linear_dbias", 0, s);
            e = launch_pdl(linear_dbias_kernel<T>, dim3((p.N + 31) / 32), dim3(256), 0, s, part, static_cast<T *>(p.dbias), slices, p.N);
            timing_mark("linear_dbias", 1, s);
            if ((rc = api_cuda_status(e)) != 0) return rc;
        }
    }
    if (own_dpre) ws += up256((size_t)(dtype == 0 ? 3 : 1) * p.M * up8(p.N) * 2);
    // the two products' partial sums take the same place, one after the other
    float *partial = reinterpret_cast<float *>(ws + pack_bytes(p.N, p.K, p.ldw, dtype) + pack_bytes(p.M, p.K, p.ldx, dtype));
    if (p.dx != nullptr) {
        if ((rc = pack(w, &w, ws, dtype, s)) != 0) return rc;
        if ((rc = gemm<false, true, T>("linear_dx", d, w, p.M, p.K, p.N, {nullptr, nullptr, 0, kActNone, p.dx, nullptr, partial}, p.status, s)) != 0)
            return rc;
    }
    ws += pack_bytes(p.N, p.K, p.ldw, dtype);
    if (p.dW != nullptr) {
        if ((rc = pack(x, &x, ws, dtype, s)) != 0) return rc;
        rc = gemm<true, true, T>("linear_dw", d, x, p.N, p.K, p.M, {nullptr, nullptr, 0, kActNone, p.dW, nullptr, partial}, p.status, s);
        if (rc != 0) return rc;
    }
    return 0;
}

}  // namespace

size_t linear_fwd_workspace(const LinearParams &p, int dtype) {
    if (p.M <= kLinearFewRows) return 0;
    return pack_bytes(p.M, p.K, p.ldx, dtype) + pack_bytes(p.N, p.K, p.ldw, dtype) + partial_bytes(p.M, p.N, p.K, dtype);
}

size_t linear_bwd_workspace(const LinearParams &p, int dtype) {
    const bool own_dpre = dtype == 0 || p.act != kActNone || p.N % 8 != 0;
    return up256((size_t)kBiasSlices * p.N * 4) + (own_dpre ? up256((size_t)(dtype == 0 ? 3 : 1) * p.M * up8(p.N) * 2) : 0) +
           pack_bytes(p.M, p.K, p.ldx, dtype) + pack_bytes(p.N, p.K, p.ldw, dtype) +
           std::max(partial_bytes(p.M, p.K, p.N, dtype), partial_bytes(p.N, p.K, p.M, dtype));
}

int launch_linear_fwd(const LinearParams &p, int dtype, cudaStream_t s) {
    return dtype == 0 ? fwd_any<float>(p, dtype, s) : fwd_any<__nv_bfloat16>(p, dtype, s);
}

int launch_linear_bwd(const LinearParams &p, int dtype, cudaStream_t s) {
    return dtype == 0 ? bwd_any<float>(p, dtype, s) : bwd_any<__nv_bfloat16>(p, dtype, s);
}

}  // namespace gdn

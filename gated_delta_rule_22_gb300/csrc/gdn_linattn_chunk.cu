// gdn_linattn_chunk.cu -- the sweeps of the linear attention with a decay (LinattnSweep in gdn_layer.cuh),
// bf16, in chunks of 128 steps on the tcgen05 tensor cores.
//
// For a chunk of L valid steps with incoming state Z [Dc][Db] (forward; local steps i, m = 0 .. L - 1):
//     out_i = sum_{m <= i} g^(i-m) (a_i . b_m) c_m + g^(i+1) Z a_i
//     Z'    = g^L Z + sum_m g^(L-1-m) c_m b_m^T
// Backwards, with Z the adjoint that the later steps leave behind, decayed up to the step in front of them:
//     out_i = sum_{m >= i} g^(m-i) (a_i . b_m) c_m + g^(L-1-i) Z a_i,    Z' = g^L Z + sum_m g^(m+1) c_m b_m^T
// Every exponent is at least 0, so that no decay, however strong, divides by an underflow.
//
// A CTA takes one sweep of one (batch row, value head), one block of up to 128 columns of Db and of Dc (the
// sweep is linear in b's columns and splits over c's; blocks of Db are added in float32 afterwards), and a
// segment of the chunks. Four products of 128 x 128 x 128 per chunk, their operands as TMA brings them:
//     P = a b^T        both K-major                  -> tensor memory; its decayed, masked bf16 copy P~ takes its place
//     O1 = P~ c        P~ from tensor memory, c MN-major
//     O2 = a Z^T       Z as bf16 in shared memory
//     U = c^T b~       both MN-major; b~_m = g^(L-1-m) b_m takes b's place once P has read it
// out = O1 + g^(i+1) O2 is formed in float32, and the state is kept in registers, Z' = g^L Z + U, so that the
// truncating additions of the tensor cores never run over more than a chunk.
// Rounded to bf16 besides the outputs: Z as an operand, and either b~ or P~ (the other one has two terms, 16 bits):
// each a relative 2^-9 of terms of either sign, so that a chunk's own steps add one rounding to that of the
// output and earlier steps at most two. b~ is the one rounded, since U then needs nothing but b's place and the
// chain from state to state is short; where the state leaves the call and the chunk still counts in it by
// 2^-12, b~ has two terms (by 1 / 8: three, 24 bits), which take the places of a and Z once O2 has read them.
//
// Warps 0-7 mask P, warps 8-11 write outputs, warps 12-19 hold the state (each four half of its columns); one warp
// fetches (two chunks deep), two issue products: P and O1, and O2 and U, so that neither chain waits for the other.
//
// A chunk takes some 6000 cycles, 3.2 us: P is there after 900, P~'s first columns after 3000 and its last after 4800,
// b~ after 3000, and from there the tensor cores are busy with U, O2 and O1 until 5700; the outputs leave under the next
// chunk's P and mask, 3300 cycles. All of these share one shared memory, whose bandwidth takes some 2000 cycles for the
// products' operands, 800 for TMA's writes, 800 for b~ and Z and besides those the mask's powers and the stores' rows:
// more warps, more columns at once or loads further ahead in any of them slowed the others (483 to 491 us for what
// is 440 so). The rest is roles that wait for one another; the two have not been told apart. O1 begins with the
// columns that are there, those of the half with more zeros first. Where the state leaves the
// call and b~ has several terms, a chunk takes up to 9000 cycles. What carries the loops: code short enough for the
// instruction cache, one arrival per warp, work of one kind in each warp (80 registers at launch, 280 bytes spilled). 4 x 4096
// steps of 32 heads of 128 x 128: forward 111 us, 4.9 TB/s of q, k, v and y (127 with S_T), backward 317 us, 3.0 TB/s; 4 rows of up to 2048
// with 16 key heads and a carried state 77 us.
#include "gdn.h"
#include "gdn_layer.cuh"
#include "gdn_umma.cuh"

#include <type_traits>

namespace gdn {

namespace {

constexpr int kC = kLinattnChunk;
constexpr int kParts = 2, kPart = 128 / kParts;    // the state's columns by two groups of four warps
constexpr int kMaskGroup = 2;                      // blocks of 16 columns of P~ that are announced at once (4: 456 us for 451, 1: 497)
constexpr int kOutWarp = 8, kStateWarp = 12, kFetchWarp = kStateWarp + 4 * kParts, kThreads = (kFetchWarp + 4) * 32;
// registers of a thread: launched with kLaunchRegs, then dealt out again
constexpr int kLaunchRegs = 80, kMaskRegs = 64, kOutRegs = 64, kStateRegs = 120, kIssueRegs = 48;
static_assert(2 * kMaskRegs + kOutRegs + kParts * kStateRegs + kIssueRegs <= kThreads / 128 * kLaunchRegs, "register split exceeds the launch's registers");
constexpr int kTile = 64 * kC * 2;                 // 64 columns of a chunk: 128 rows of 128 bytes
constexpr int kOperand = 2 * kTile;
constexpr int kStage = 3 * kOperand;               // a, b, c
constexpr size_t kSmem = 1024 + 2 * kStage + kOperand + (32 + 136 + 16) * 4 + 24 * 8 + 16;
// tensor memory columns
constexpr int kColP = 0, kColO1 = 128, kColO2 = 256, kColU = 384;

struct SweepArgs {
    LinattnParams p;
    int blocks[3];                                 // column blocks of each sweep (of Db times of Dc)
    int state_only;                                // write the segments' end states from zero, nothing else
};

__device__ __forceinline__ uint64_t desc_k(uint32_t start) { return umma_sdesc(start, 16u, 1024u) | (uint64_t)2 << 61; }
__device__ __forceinline__ uint64_t desc_mn(uint32_t start) { return umma_sdesc(start, kTile, 1024u) | (uint64_t)2 << 61; }

// D (+)= A B with A (bf16 pairs, one 32-bit column per two of K) in tensor memory; executed by a whole warp
__device__ __forceinline__ void umma_bf16_tw(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, bool accumulate, uint32_t lead) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"((uint32_t)accumulate), "r"(lead)
        : "memory");
}

// The 16-byte piece `piece` (8 columns) of row r of an operand's tiles in the 128-byte swizzle
__device__ __forceinline__ uint4 *piece_at(unsigned char *operand, int r, int piece) {
    return reinterpret_cast<uint4 *>(operand + (piece >> 3) * kTile + r * 128 + (((piece & 7) ^ (r & 7)) << 4));
}

// One arrival for what a warp has done
__device__ __forceinline__ void warp_arrive(uint64_t *bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}
// mbar_wait by a whole warp, with one answer, and together from there (tensor memory is read by whole warps)
__device__ __forceinline__ bool all_wait(uint64_t *bar, uint32_t parity) {
    const bool there = __all_sync(kFullMask, mbar_wait(bar, parity));
    __syncwarp();
    return there;
}

// 32 bytes of a row, at once where they are aligned to that (every lane has a row of its own, and a store of 32
// rows takes a cycle for each)
__device__ __forceinline__ void store_piece2(void *p, float a, float b, float c, float d, float e, float f, float g, float h, bool wide) {
    if (wide) {
        asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(a), "f"(b), "f"(c), "f"(d), "f"(e), "f"(f), "f"(g), "f"(h)
                     : "memory");
    } else {
        *static_cast<float4 *>(p) = make_float4(a, b, c, d);
        *(static_cast<float4 *>(p) + 1) = make_float4(e, f, g, h);
    }
}

// b w for a pair of b and w = w0 + w1 + w2 as bf16 terms, in packed bf16 arithmetic (in float32 the conversions
// alone cost as much): t0 = b w0 rounded; the product of two bf16 has 16 bits, so its rest is a bf16 exactly; t1 =
// that rest + b w1 rounded, some 2^-9 of the product. Three terms: what t1 lost (a two-sum, and the rest of b w1,
// both exact) + b w2, some 2^-18, with an error of 2^-26 of the product.
using bf16x2 = __nv_bfloat162;
__device__ __forceinline__ uint32_t bits(const bf16x2 &x) { return *reinterpret_cast<const uint32_t *>(&x); }
// b w for a pair of b and w = w0 + w1, rounded once (but for some 2^-18)
__device__ __forceinline__ uint32_t weigh(uint32_t b, bf16x2 w0, bf16x2 w1) {
    const bf16x2 x = *reinterpret_cast<const bf16x2 *>(&b);
    return bits(__hfma2(x, w0, __hmul2_rn(x, w1)));
}
template <bool THREE>
__device__ __forceinline__ void split_product(uint32_t b, bf16x2 w0, bf16x2 w1, bf16x2 w2, uint32_t &t0, uint32_t &t1, uint32_t &t2) {
    const bf16x2 x = *reinterpret_cast<const bf16x2 *>(&b), a = __hmul2_rn(x, w0), rest = __hfma2(x, w0, __hneg2(a));
    t0 = bits(a);
    if (!THREE) {
        t1 = bits(__hfma2(x, w1, rest));
        return;
    }
    const bf16x2 u = __hmul2_rn(x, w1), u_rest = __hfma2(x, w1, __hneg2(u));
    const bf16x2 m = __hadd2_rn(rest, u), v = __hsub2_rn(m, rest);
    const bf16x2 lost = __hadd2_rn(__hsub2_rn(rest, __hsub2_rn(m, v)), __hsub2_rn(u, v));
    t1 = bits(m);
    t2 = bits(__hfma2(x, w2, __hadd2_rn(lost, u_rest)));
}

__device__ __forceinline__ void write_zeros(const LinattnSweep &w, size_t at, int n) {
    if (w.sums)
        for (int i = 0; i < n; i += 4) *reinterpret_cast<float4 *>(w.part + at + i) = make_float4(0.f, 0.f, 0.f, 0.f);
    else
        for (int i = 0; i < n; i += 8) *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(w.out) + at + i) = make_uint4(0u, 0u, 0u, 0u);
}

}  // namespace

// WHOLE: the states' rows are of whole pieces of eight.
template <bool WHOLE>
__global__ void __launch_bounds__(kThreads, 1) linattn_chunk_kernel(const __grid_constant__ LinattnMaps maps, const __grid_constant__ SweepArgs cp) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    unsigned char *zb = smem + 2 * kStage;                                   // the state as an operand [e][d]
    float *pw = reinterpret_cast<float *>(zb + kOperand) + 32;               // g^0 .. g^128, zeros for -32 .. -1
    float *pw_back = pw + 136;                                               // g^15 .. g^0
    uint64_t *full = reinterpret_cast<uint64_t *>(pw_back + 16), *empty = full + 2;
    uint64_t *p_full = full + 4, *o1_full = full + 6, *o2_full = full + 7, *o_empty = full + 8;
    uint64_t *u_full = full + 9, *p_seen = full + 10, *bt_full = full + 12, *z_full = bt_full + kParts;  // (the last two: one for each part)
    uint64_t *pt_full = z_full + kParts;                                     // (groups of a part's columns, then those of the other)
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(full + 24);
    const LinattnParams &p = cp.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // this CTA's sweep, column blocks and segment
    int x = blockIdx.x;
    const int segs = cp.state_only ? p.segs - 1 : p.segs;
    const int seg = x % segs;
    x /= segs;
    const int which = x < cp.blocks[0] ? 0 : x < cp.blocks[0] + cp.blocks[1] ? 1 : 2;
    const int unit = ((blockIdx.z * gridDim.y + blockIdx.y) * (gridDim.x / segs) + x) * (p.segs - 1);     // of its segments' states
    if (which > 0) x -= cp.blocks[0];
    if (which > 1) x -= cp.blocks[1];
    const LinattnSweep &w = p.sweep[which];
    const int nc = (w.Dc + 127) / 128, db0 = x / nc * 128, dc0 = x % nc * 128;
    const int Db = min(w.Db - db0, 128), Dc = min(w.Dc - dc0, 128);
    const int h = blockIdx.y, b = blockIdx.z, hk = h / (p.Hv / p.Hk);
    const size_t head = (size_t)b * p.Hv + h;
    const int n = row_length(p.lens, b, p.T), chunks = (n + kC - 1) / kC;
    const int first = seg * p.seg_chunks, last = min(first + p.seg_chunks, chunks);       // in the order of the sweep
    const bool rev = w.rev != 0, masked = p.lens != nullptr;
    auto chunk_of = [&](int i) { return rev ? chunks - 1 - i : i; };
    auto length_of = [&](int i) { return min(kC, n - chunk_of(i) * kC); };
    const int Dbp = (Db + 15) / 16 * 16, Dcp = (Dc + 15) / 16 * 16;                        // (zeros behind Db, Dc)
    const int work = cp.state_only ? (last < chunks ? last - first : 0) : last - first;   // (<= 0: none)

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, cp.state_only ? 1 : 2);
        }
        for (uint64_t *bar : {p_full, o1_full, o2_full, u_full}) mbar_init(bar, 1);
        for (int i = 0; i < 8 / kMaskGroup; ++i) mbar_init(pt_full + i, 4);  // (warps)
        mbar_init(o_empty, 4);
        for (int i = 0; i < 2 * kParts; ++i) mbar_init(bt_full + i, 4);
        mbar_init(p_seen, 1 + 4 * ((Dbp + kPart - 1) / kPart));
        fence_mbar_init();
    }
    if (warp == kFetchWarp) tmem_alloc(tmem_slot, 512);
    {
        const float g = p.g[h];
        for (int i = threadIdx.x; i <= kC; i += kThreads) pw[i] = powf(g, (float)i);
        if (threadIdx.x < 32) pw[(int)threadIdx.x - 32] = 0.f;
        if (threadIdx.x < 16) pw_back[threadIdx.x] = powf(g, (float)(15 - (int)threadIdx.x));
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // Terms of b~
    const float lg = log2f(p.g[h]);
    auto terms_of = [&](int i) {
        const int after = rev ? chunk_of(i) * kC : max(n - (chunk_of(i) + 1) * kC, 0);        // steps that follow it in the sweep
        const float weight = after == 0 ? 0.f : after * lg;                                  // (its log2)
        return w.last == nullptr ? 1 : weight >= -3.f ? 3 : weight >= -12.f ? 2 : 1;
    };
    // Whether P~ has two: with b~ of one, and where P is a part of the products of a pair of steps, which may cancel
    auto two_of = [&](int i) { return w.Db > 128 || terms_of(i) == 1; };
    const size_t out_step = (size_t)p.Hv * w.Dc;
    const size_t out0 = (size_t)(db0 / 128) * p.B * p.T * out_step + (size_t)b * p.T * out_step + (size_t)h * w.Dc + dc0;
    bool ok = true;

    if (warp < kOutWarp) {                         // ---- decay and mask P, columns 64 (warp / 4) and on
        regs_dec<kMaskRegs>();
        const int part = warp >> 2, i = threadIdx.x & 127;                  // this thread's step of the chunk
        const uint32_t mine = tmem + ((uint32_t)(warp & 3) << 21) + kColP + 64 * part;
        for (int k = 0; k < work && !cp.state_only; ++k) {
            const int L = length_of(first + k);
            const bool two = two_of(first + k);
            if (!(ok = all_wait(p_full, k & 1))) break;
            tc_fence_after();
#pragma unroll 1
            for (int cb = 0; cb < 4; ++cb) {       // 16 columns, from m0
                const int m0 = 64 * part + 16 * cb, near = (warp & 3) * 32;      // (rows near .. near + 31)
                float v[16];
                if (rev ? m0 + 15 >= near : m0 <= near + 31) {
                    tmem_ld16f(mine + 16 * cb, v);
                    tmem_wait_ld();
                    if (rev ? m0 >= near + 32 : m0 + 16 <= near) {          // g^|i-m| as a product of two powers
                        const float f = pw[rev ? m0 - i : i - m0 - 15];
                        const float4 *d4 = reinterpret_cast<const float4 *>(rev ? pw : pw_back);
#pragma unroll
                        for (int r = 0; r < 16; r += 4) {
                            const float4 d = d4[r / 4];
                            float2 x = __fmul2_rn(make_float2(v[r], v[r + 1]), __fmul2_rn(make_float2(d.x, d.y), make_float2(f, f)));
                            v[r] = x.x; v[r + 1] = x.y;
                            x = __fmul2_rn(make_float2(v[r + 2], v[r + 3]), __fmul2_rn(make_float2(d.z, d.w), make_float2(f, f)));
                            v[r + 2] = x.x; v[r + 3] = x.y;
                        }
                    } else {
                        const int e0 = rev ? m0 - i : i - m0;
#pragma unroll
                        for (int r = 0; r < 16; ++r) {
                            v[r] *= pw[rev ? e0 + r : e0 - r];      // (0 where negative)
                        }
                    }
                    if (L < kC)                    // (what lies behind the row may be anything)
#pragma unroll
                        for (int r = 0; r < 16; ++r) v[r] = m0 + r < L ? v[r] : 0.f;
                } else {
#pragma unroll
                    for (int r = 0; r < 16; ++r) v[r] = 0.f;
                }
                uint32_t hi[8];                    // its terms take its place: no warp waits for another
                if (two) {                         // (the first cut off, not rounded: the second holds the rest)
                    uint32_t lo[8];
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        const uint32_t e0 = __float_as_uint(v[2 * r]), e1 = __float_as_uint(v[2 * r + 1]);
                        hi[r] = __byte_perm(e0, e1, 0x7632);
                        const float2 x = __fadd2_rn(make_float2(v[2 * r], v[2 * r + 1]),
                                                    make_float2(-__uint_as_float(e0 & 0xffff0000u), -__uint_as_float(e1 & 0xffff0000u)));
                        lo[r] = pack2_bf16(x.x, x.y);
                    }
                    tmem_st8(mine + 16 * cb + 8, lo);
                } else {
#pragma unroll
                    for (int r = 0; r < 8; ++r) hi[r] = pack2_bf16(v[2 * r], v[2 * r + 1]);
                }
                tmem_st8(mine + 16 * cb, hi);
                if (cb % kMaskGroup == kMaskGroup - 1) {
                    tmem_wait_st();
                    tc_fence_before();
                    warp_arrive(pt_full + (4 * part + cb) / kMaskGroup, lane);
                }
            }
        }
    } else if (warp < kStateWarp) {                // ---- the outputs
        regs_dec<kOutRegs>();
        const bool wide = ((uintptr_t)(w.sums ? w.part : w.out) & 31) == 0 && w.Dc % 16 == 0;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
        const int i = threadIdx.x & 127;           // this thread's step of the chunk
        for (int k = 0; k < work && !cp.state_only; ++k) {
            const int L = length_of(first + k), t0 = chunk_of(first + k) * kC;
            const uint32_t ph = k & 1;
            if (!(ok = all_wait(o2_full, ph) && all_wait(o1_full, ph))) break;
            tc_fence_after();
            const float s = pw[rev ? max(L - 1 - i, 0) : i + 1];
            const size_t at = out0 + (size_t)(t0 + i) * out_step;
#pragma unroll 1
            for (int c = 0; c < Dc; c += 16) {
                float o1[16], o2[16];
                tmem_ld16f(lanes + kColO1 + c, o1);
                tmem_ld16f(lanes + kColO2 + c, o2);
                tmem_wait_ld();
#pragma unroll
                for (int r = 0; r < 16; r += 2) {
                    const float2 x = __ffma2_rn(make_float2(s, s), make_float2(o2[r], o2[r + 1]), make_float2(o1[r], o1[r + 1]));
                    o1[r] = x.x;
                    o1[r + 1] = x.y;
                }
                if (i < L) {
                    if (w.sums) {
                        float *out = w.part + at + c;
                        store_piece2(out, o1[0], o1[1], o1[2], o1[3], o1[4], o1[5], o1[6], o1[7], wide);
                        if (c + 8 < Dc) store_piece2(out + 8, o1[8], o1[9], o1[10], o1[11], o1[12], o1[13], o1[14], o1[15], wide);
                    } else {
                        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(w.out) + at + c;
                        float y[8];
#pragma unroll
                        for (int r = 0; r < 8; ++r) y[r] = __uint_as_float(pack2_bf16(o1[2 * r], o1[2 * r + 1]));
                        if (c + 8 < Dc) store_piece2(out, y[0], y[1], y[2], y[3], y[4], y[5], y[6], y[7], wide);
                        else *reinterpret_cast<float4 *>(out) = make_float4(y[0], y[1], y[2], y[3]);
                    }
                }
                __syncwarp();                      // (the loads above are the whole warp's)
            }
            tc_fence_before();
            warp_arrive(o_empty, lane);
        }
        // zeros behind the row: this segment's share of the steps
        if (!cp.state_only) {
            const int from = max(n, seg * p.seg_chunks * kC), to = seg == p.segs - 1 ? p.T : min(p.T, (seg + 1) * p.seg_chunks * kC);
            for (int t = from + i; t < to; t += 128) write_zeros(w, out0 + (size_t)t * out_step, Dc);
        }
    } else if (warp < kFetchWarp) {                // ---- the state: a thread holds a part of row e
        regs_inc<kStateRegs>();
        const int e = threadIdx.x & 127, part = (warp - kStateWarp) >> 2, d0 = kPart * part;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21) + kColU + d0;
        float Z[kPart];
        const bool row = e < Dc && (WHOLE || dc0 + e < w.Dc_of);
        const int work_here = d0 < Dbp ? work : 0;
        const float *init = cp.state_only ? nullptr : w.init;
#pragma unroll
        for (int d = 0; d < kPart; d += 4) {
            float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
            if (init != nullptr && row && d0 + d < Db) {
                if (WHOLE && !w.init_t) {
                    z = *reinterpret_cast<const float4 *>(init + (head * w.Dc + dc0 + e) * w.Db + db0 + d0 + d);
                } else if (WHOLE) {
                    const float *at = init + (head * w.Db + db0 + d0 + d) * w.Dc + dc0 + e;
                    z = make_float4(at[0], at[w.Dc], at[2 * w.Dc], at[3 * w.Dc]);
                } else {
                    float x[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int col = db0 + d0 + d + i;
                        x[i] = col >= w.Db_of ? 0.f : w.init_t ? init[(head * w.Db_of + col) * w.Dc_of + dc0 + e] : init[(head * w.Dc_of + dc0 + e) * w.Db_of + col];
                    }
                    z = make_float4(x[0], x[1], x[2], x[3]);
                }
            }
            Z[d] = z.x; Z[d + 1] = z.y; Z[d + 2] = z.z; Z[d + 3] = z.w;
        }
        if (!cp.state_only && work_here > 0 && seg > 0) {                    // through the earlier segments
            const float decay = powf(p.g[h], (float)(rev ? n - (chunks - first) * kC : first * kC));
            const float4 *E = reinterpret_cast<const float4 *>(p.seg_state) + (size_t)(unit + seg - 1) * (kC * 32) + part * (kC * kPart / 4);
#pragma unroll
            for (int d = 0; d < kPart / 4; ++d) {
                const float4 u = E[d * 128 + e];
                Z[4 * d] = fmaf(decay, Z[4 * d], u.x);
                Z[4 * d + 1] = fmaf(decay, Z[4 * d + 1], u.y);
                Z[4 * d + 2] = fmaf(decay, Z[4 * d + 2], u.z);
                Z[4 * d + 3] = fmaf(decay, Z[4 * d + 3], u.w);
            }
        }
        auto put_operand = [&]() {
#pragma unroll
            for (int c = 0; c < kPart / 8; ++c)
                *piece_at(zb, e, kPart / 8 * part + c) = make_uint4(pack2_bf16(Z[8 * c], Z[8 * c + 1]), pack2_bf16(Z[8 * c + 2], Z[8 * c + 3]),
                                                            pack2_bf16(Z[8 * c + 4], Z[8 * c + 5]), pack2_bf16(Z[8 * c + 6], Z[8 * c + 7]));
        };
        // Steps behind the row in the k-th chunk, where they are not beyond T (which reads as zeros): c may hold
        // anything there, and 0 x NaN is NaN.
        auto clear = [&](int k) {
            const int L = length_of(first + k);
            if (!masked || L == kC || part != 0) return true;
            if (!all_wait(full + (k & 1), k >> 1 & 1)) return false;
            if (e >= L)
                for (int c = 0; c < (Dc > 64 ? 16 : 8); ++c) *piece_at(smem + (k & 1) * kStage + 2 * kOperand, e, c) = make_uint4(0u, 0u, 0u, 0u);
            return true;
        };
        if (work_here > 0 && !cp.state_only) {
            put_operand();
            ok = clear(0);
            fence_proxy_async();
            warp_arrive(z_full + part, lane);
        }
        // b~ of the k-th chunk: this thread's step of it, weighted, as bf16 terms: the first takes b's place once P is there,
        // the others, formed meanwhile, those of a and the state once O2 is (three terms: the second half of the
        // pieces, whose terms the registers do not hold, behind that wait)
        auto write_terms = [&](int k, auto terms_) {
            constexpr int TERMS = decltype(terms_)::value;
            constexpr int N = kPart / 8, BATCH = 4, HELD = TERMS == 3 ? N / 2 : N;     // pieces, those read and those held at once
            const int L = length_of(first + k);
            if (!(cp.state_only ? all_wait(full + (k & 1), k >> 1 & 1) && clear(k) : all_wait(p_full, k & 1))) return false;
            if (lane == 0) mbar_arrive(p_seen);
            unsigned char *a = smem + (k & 1) * kStage, *bb = a + kOperand;
            const float wj = pw[e < L ? (rev ? e + 1 : L - 1 - e) : 0];
            const bf16x2 w0 = __float2bfloat162_rn(wj), w1 = __float2bfloat162_rn(wj - __low2float(w0)),
                         w2 = __float2bfloat162_rn(wj - __low2float(w0) - __low2float(w1));
            for (int h = 0; h < N; h += HELD) {
                const int first_piece = N * part + h;
                uint32_t t1[TERMS > 1 ? 4 * HELD : 1], t2[TERMS > 2 ? 4 * HELD : 1];
#pragma unroll
                for (int c0 = 0; c0 < HELD; c0 += BATCH) {
                    uint4 raw[BATCH];
#pragma unroll
                    for (int c = 0; c < BATCH; ++c) {
                        raw[c] = *piece_at(bb, e, first_piece + c0 + c);
                        if (e >= L) raw[c] = make_uint4(0u, 0u, 0u, 0u);
                    }
#pragma unroll
                    for (int c = 0; c < BATCH; ++c) {
                        const uint32_t in[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
                        uint32_t t0[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int at = 4 * (c0 + c) + q;
                            if constexpr (TERMS == 1) t0[q] = weigh(in[q], w0, w1);
                            else split_product<TERMS == 3>(in[q], w0, w1, w2, t0[q], t1[at], t2[TERMS == 3 ? at : 0]);
                        }
                        *piece_at(bb, e, first_piece + c0 + c) = make_uint4(t0[0], t0[1], t0[2], t0[3]);
                    }
                }
                if constexpr (TERMS > 1) {
                    if (h == 0 && !cp.state_only && !all_wait(o2_full, k & 1)) return false;
#pragma unroll
                    for (int c = 0; c < HELD; ++c) {
                        *piece_at(a, e, first_piece + c) = make_uint4(t1[4 * c], t1[4 * c + 1], t1[4 * c + 2], t1[4 * c + 3]);
                        if constexpr (TERMS > 2) *piece_at(zb, e, first_piece + c) = make_uint4(t2[4 * c], t2[4 * c + 1], t2[4 * c + 2], t2[4 * c + 3]);
                    }
                }
            }
            fence_proxy_async();
            return true;
        };
        // the state behind the k-th chunk
        auto add_u = [&](int k) {
            if (!all_wait(u_full, k & 1)) return false;
            tc_fence_after();
            const float gl = pw[length_of(first + k)];
            const float2 decay = make_float2(gl, gl);
#pragma unroll
            for (int c = 0; c < kPart; c += 32) {
                float u[32];
                tmem_ld32f(lanes + c, u);
                tmem_wait_ld();
#pragma unroll
                for (int r = 0; r < 32; r += 2) {
                    const float2 z = __ffma2_rn(decay, make_float2(Z[c + r], Z[c + r + 1]), make_float2(u[r], u[r + 1]));
                    Z[c + r] = z.x;
                    Z[c + r + 1] = z.y;
                }
            }
            tc_fence_before();
            return true;
        };
        for (int k = 0; k < work_here && ok; ++k) {
            const int terms = terms_of(first + k);
            // (without outputs one term is written under the last chunk's U; more take places that that may still read)
            const bool ahead = cp.state_only && terms == 1;
            if (ahead && !(ok = write_terms(k, std::integral_constant<int, 1>()))) break;
            if (k == 0 && ahead) warp_arrive(bt_full + part, lane);
            if (k > 0) {
                if (!(ok = add_u(k - 1))) break;
                if (!cp.state_only) {
                    // (the last state has been read: by U of several terms already)
                    if (terms_of(first + k - 1) == 1 && !(ok = all_wait(o2_full, (k - 1) & 1))) break;
                    put_operand();
                    ok = clear(k);
                    fence_proxy_async();
                }
                // (what was written ahead is announced here, when the last U has been issued: bt_full is never two phases
                // ahead of the warp that waits for it)
                if (ahead) warp_arrive(bt_full + part, lane);
                warp_arrive(z_full + part, lane);
            }
            if (ahead || !ok) continue;
            ok = terms == 1 ? write_terms(k, std::integral_constant<int, 1>()) :
                 terms == 2 ? write_terms(k, std::integral_constant<int, 2>()) : write_terms(k, std::integral_constant<int, 3>());
            warp_arrive(bt_full + part, lane);
        }
        if (ok && work_here > 0) ok = add_u(work - 1);
        if (cp.state_only) {
            float4 *E = reinterpret_cast<float4 *>(p.seg_state) + (size_t)(unit + seg) * (kC * 32) + part * (kC * kPart / 4);
            if (work > 0)
#pragma unroll
                for (int d = 0; d < kPart / 4; ++d) E[d * 128 + e] = make_float4(Z[4 * d], Z[4 * d + 1], Z[4 * d + 2], Z[4 * d + 3]);
        } else if (w.last != nullptr && row && seg == (chunks > 0 ? (chunks - 1) / p.seg_chunks : 0)) {
            const bool wide = ((uintptr_t)w.last & 31) == 0;
#pragma unroll
            for (int d = 0; d < kPart; d += 8) {
                if (d0 + d >= Db) break;
                float *out = w.last + (head * (WHOLE ? w.Dc : w.Dc_of) + dc0 + e) * (WHOLE ? w.Db : w.Db_of) + db0 + d0 + d;
                if (WHOLE) {
                    store_piece2(out, Z[d], Z[d + 1], Z[d + 2], Z[d + 3], Z[d + 4], Z[d + 5], Z[d + 6], Z[d + 7], wide);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (db0 + d0 + d + i < w.Db_of) out[i] = Z[d + i];
                }
            }
        }
    } else {
    regs_dec<kIssueRegs>();
    if (warp == kFetchWarp) {                      // ---- fetch a, b and c
        if (lane == 0) {
            const int nb = Db > 64 ? 2 : 1, nd = Dc > 64 ? 2 : 1;
            const unsigned bytes = ((cp.state_only ? 1 : 2) * nb + nd) * kTile;
            int k = 0;
            for (; k < work; ++k) {
                const int t0 = chunk_of(first + k) * kC, s = k & 1;
                if (k >= 2 && !(ok = mbar_wait(empty + s, (k >> 1 & 1) ^ 1))) break;
                unsigned char *st = smem + s * kStage;
                mbar_expect_tx(full + s, bytes);
                for (int i = 0; i < nb; ++i) {
                    if (!cp.state_only)
                        tma_load_4d(st + i * kTile, &maps.map[w.a_map], full + s, db0 + 64 * i, w.a_keys ? hk : h, t0, b);
                    tma_load_4d(st + kOperand + i * kTile, &maps.map[w.b_map], full + s, db0 + 64 * i, w.b_keys ? hk : h, t0, b);
                }
                for (int i = 0; i < nd; ++i)
                    tma_load_4d(st + 2 * kOperand + i * kTile, &maps.map[w.c_map], full + s, dc0 + 64 * i, w.c_keys ? hk : h, t0, b);
            }
            for (int i = max(k - 2, 0); i < k; ++i) mbar_wait(full + (i & 1), i >> 1 & 1);     // no copy outlives the CTA
        }
        __syncwarp();
    } else if (warp == kFetchWarp + 1) {           // ---- issue P and O1
        if (!cp.state_only) {
            const uint32_t lead = elect_one_sync();
            const uint32_t idesc_p = umma_idesc(1, 128, 128), idesc_o = umma_idesc_t(1, 128, Dcp, false, true);
            for (int k = 0; k < work; ++k) {
                const uint32_t ph = k & 1;
                const uint32_t a = smem_addr(smem) + (k & 1) * kStage, bb = a + kOperand, c = bb + kOperand;
                // (P takes the place of the last chunk's P~, and is issued when all have seen that the last one was there)
                if (!(ok = all_wait(full + (k & 1), k >> 1 & 1) && (k == 0 || (all_wait(o1_full, ph ^ 1) && all_wait(p_seen, ph ^ 1))))) break;
                tc_fence_after();
                for (int q = 0; 16 * q < Db; ++q) {
                    const uint32_t off = (q >> 2) * kTile + (q & 3) * 32;
                    umma_bf16_w(tmem + kColP, desc_k(a + off), desc_k(bb + off), idesc_p, q > 0, lead);
                }
                umma_commit_w(p_full, lead);
                ok = (k == 0 || all_wait(o_empty, ph ^ 1)) &&
                     (!(masked && length_of(first + k) < kC) || all_wait(o2_full, ph));           // (c is cleared by then)
                if (!ok) break;
                const bool two = two_of(first + k);
                const uint64_t cd = desc_mn(c);
                // The products of each group of columns as soon as it is there, those of the half with more zeros first
#pragma unroll 1
                for (int j = 0; j < 8 && ok; j += kMaskGroup) {
                    const int q0 = (j / kMaskGroup + (rev ? 0 : 1)) % 2 * 4 + j / (2 * kMaskGroup) * kMaskGroup;
                    if (!(ok = all_wait(pt_full + q0 / kMaskGroup, ph))) break;
                    tc_fence_after();
                    for (int term = two ? 1 : 0; term >= 0; --term)          // smallest first
#pragma unroll
                        for (int q = q0; q < q0 + kMaskGroup; ++q)
                            umma_bf16_tw(tmem + kColO1, tmem + kColP + 16 * q + 8 * term, cd + q * (2048 >> 4), idesc_o,
                                         j > 0 || q > q0 || (two && term == 0), lead);
                }
                if (!ok) break;
                umma_commit_w(o1_full, lead);
                umma_commit_w(empty + (k & 1), lead);
            }
        }
    } else if (warp == kFetchWarp + 2) {           // ---- issue O2 and U
        const uint32_t lead = elect_one_sync();
        const uint32_t idesc_o = umma_idesc(1, 128, Dcp), idesc_u = umma_idesc_t(1, 128, Dbp, true, true);
        const int parts = (Dbp + kPart - 1) / kPart;
        // (z_full: the state's operand is written, and the last U read)
        auto issue_u = [&](int k, int terms) {
            const uint32_t a = smem_addr(smem) + (k & 1) * kStage, bb = a + kOperand, c = bb + kOperand, z = smem_addr(zb);
            for (int part = 0; part < parts; ++part)
                if (!all_wait(bt_full + part, k & 1) || (cp.state_only && k > 0 && !all_wait(z_full + part, (k & 1) ^ 1))) return false;
            tc_fence_after();
            for (int term = terms - 1; term >= 0; --term) {                  // smallest first
                uint64_t cd = desc_mn(c), bd = desc_mn(term == 0 ? bb : term == 1 ? a : z);
#pragma unroll
                for (int q = 0; q < kC / 16; ++q, cd += 2048 >> 4, bd += 2048 >> 4)
                    umma_bf16_w(tmem + kColU, cd, bd, idesc_u, term < terms - 1 || q > 0, lead);
            }
            umma_commit_w(u_full, lead);
            return true;
        };
        for (int k = 0; k < work; ++k) {
            const uint32_t ph = k & 1;
            const uint32_t a = smem_addr(smem) + (k & 1) * kStage, z = smem_addr(zb);
            const int terms = terms_of(first + k);
            if (!(ok = all_wait(full + (k & 1), k >> 1 & 1))) break;
            if (!cp.state_only) {
                if (!(ok = all_wait(p_full, ph))) break;
                if (lane == 0) mbar_arrive(p_seen);
                for (int part = 0; part < parts && ok; ++part) ok = all_wait(z_full + part, ph);
                // the next state's product first, where it needs no place of a or Z
                if (ok && terms == 1) ok = issue_u(k, terms);
                if (!ok || !(ok = (k == 0 || all_wait(o_empty, ph ^ 1)))) break;
                tc_fence_after();
                for (int q = 0; 16 * q < Db; ++q) {
                    const uint32_t off = (q >> 2) * kTile + (q & 3) * 32;
                    umma_bf16_w(tmem + kColO2, desc_k(a + off), desc_k(z + off), idesc_o, q > 0, lead);
                }
                umma_commit_w(o2_full, lead);
            }
            if ((cp.state_only || terms > 1) && !(ok = issue_u(k, terms))) break;
            umma_commit_w(empty + (k & 1), lead);
        }
    }
    }
    if (!ok && lane == 0) report_status(p.status, kStatusTimeout);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kFetchWarp) tmem_dealloc(tmem, 512);
}

// What the segments up to each leave, from what each leaves: E_s += g^(steps of s) E_{s-1}. All segments here but the
// first hold whole chunks only.
__global__ void __launch_bounds__(256) linattn_join_kernel(const LinattnParams p) {
    const int b = blockIdx.z, h = blockIdx.y, blocks = gridDim.x / 16, x = blockIdx.x / 16;
    const int chunks = (row_length(p.lens, b, p.T) + kC - 1) / kC;
    const float decay = powf(p.g[h], (float)(p.seg_chunks * kC));
    float4 *E = reinterpret_cast<float4 *>(p.seg_state) + ((size_t)(b * gridDim.y + h) * blocks + x) * (p.segs - 1) * (kC * 32) +
                blockIdx.x % 16 * 256 + threadIdx.x;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = 0; s < p.segs - 1 && (s + 1) * p.seg_chunks < chunks; ++s, E += kC * 32) {
        const float4 u = *E;
        sum = make_float4(fmaf(decay, sum.x, u.x), fmaf(decay, sum.y, u.y), fmaf(decay, sum.z, u.z), fmaf(decay, sum.w, u.w));
        *E = sum;
    }
}

static int sweep_blocks(const LinattnSweep &w) { return ((w.Db + 127) / 128) * ((w.Dc + 127) / 128); }

// Segments of a row's chunks, where one CTA for each head and column block leaves SMs idle: as many as fill
// them once.
size_t linattn_segments(LinattnParams *p) {
    const int chunks = (p->T + kC - 1) / kC;
    long long ctas = 0;
    for (int i = 0; i < p->sweeps; ++i) ctas += sweep_blocks(p->sweep[i]);
    ctas *= (long long)p->B * p->Hv;
    long long segs = 152 / ctas;
    if (segs > chunks / 2) segs = chunks / 2;
    if (segs < 2) segs = 1;
    p->seg_chunks = (int)((chunks + segs - 1) / segs);
    p->segs = (chunks + p->seg_chunks - 1) / p->seg_chunks;
    return (size_t)ctas * (p->segs - 1);
}

cudaError_t launch_linattn_chunks(const LinattnParams &p, const LinattnMaps &maps, cudaStream_t s) {
    const bool whole = p.Dk % 8 == 0 && p.Dv % 8 == 0;
    cudaError_t e = whole ? allow_smem<linattn_chunk_kernel<true>>((int)kSmem) : allow_smem<linattn_chunk_kernel<false>>((int)kSmem);
    if (e != cudaSuccess) return e;
    auto *kernel = whole ? linattn_chunk_kernel<true> : linattn_chunk_kernel<false>;
    SweepArgs cp = {};
    cp.p = p;
    int blocks = 0;
    for (int i = 0; i < p.sweeps; ++i) blocks += cp.blocks[i] = sweep_blocks(p.sweep[i]);
    auto run = [&](const char *name, int segs) {
        timing_mark(name, 0, s);
        kernel<<<dim3(blocks * segs, p.Hv, p.B), kThreads, kSmem, s>>>(maps, cp);
        const cudaError_t err = cudaGetLastError();
        timing_mark(name, 1, s);
        return err;
    };
    if (p.segs > 1) {
        cp.state_only = 1;
        if ((e = run("linattn_states", p.segs - 1)) != cudaSuccess) return e;
        cp.state_only = 0;
    }
    if (p.segs > 2) {
        timing_mark("linattn_join", 0, s);
        linattn_join_kernel<<<dim3(blocks * 16, p.Hv, p.B), 256, 0, s>>>(p);
        e = cudaGetLastError();
        timing_mark("linattn_join", 1, s);
        if (e != cudaSuccess) return e;
    }
    if ((e = run("linattn_chunk", p.segs)) != cudaSuccess) return e;
    return p.sums > 0 ? launch_linattn_sums(p, 1, s) : cudaSuccess;
}

}  // namespace gdn

// The paged key-value cache (int8 codes with one fp32 scale per token and
// head, or bf16) and the attention of one new token over it.
//
//   l_t = scale * (q . k_t),  p_t = e^(l_t - m),  m = max_t l_t
//   y   = sum_t p_t v_t / sum_t p_t
//
// Bound by the cache's bytes: each key and value is read once, by whichever
// CTA holds its part of the context, for all the query heads that share it.
// Every warp streams tiles of TT tokens of its own through a ring in shared
// memory (cp.async, 16 bytes a lane, zeros in place of absent tokens), so that
// one to two tiles a warp, 100 to 200 KB an SM, are in flight whatever the
// arithmetic does.  The arithmetic rides on warp MMAs (fp32 or int32 sums):
//
//   lane = 4 g + c (g = 0..7, c = 0..3)
//   scores   S[query, token] = Q * K^T: lane takes 16 contiguous bytes of
//     token row 8j + g; which d a fragment slot means is free as long as Q's
//     hold the same d's, so the 16 bytes are the B operand as they are
//   outputs  O^T[d, query] = V^T (16 d x 16 tokens) * P^T (16 tokens x 8): the
//     scores' accumulators (query g, tokens 8j + 2c, + 1) have the B operand's
//     layout already; lane takes 16 contiguous bytes of d from each of its
//     tokens and pairs them across tokens with byte permutes
//
// int8 cache.  Scores are int8 MMAs on the codes themselves: the query's head
// is scaled by a power of two to integers and cut into planes of signed 8 bits.
// With up to 8 query heads a plane fills half of an MMA's 16 rows: two MMAs
// take four planes, 31 bits (exact but for elements 2^-22 below the head's
// largest, which round to 2^-30 of it).  With more heads a plane is an MMA of
// its own: three of them, 23 bits (2^-14, 2^-22; a fourth would cost 64
// sequences of up to 8191, 8 x 16 heads of 128, 165 -> 193 us).  The int32 sums
// are exact and join in
// fp32.  Keys' scales multiply the scores, values' scales the probabilities,
// which a running power of two per query brings to [0, 2^15) and which then are
// the sum of two fp16: good to 2^-22, and below 2^-17 of the loudest token's to
// 2^-39 of that (a single fp16 lost the quiet tokens wherever the loud ones'
// codes are 0; 64 sequences of up to 8191, 8 x 4 heads of 128: 116 us with two
// parts, 112 with one, 130 with two bf16, which have no such end but take two
// more instructions a pair of codes).  The values' codes become fp16 exactly
// (the byte, offset to unsigned, under the exponent of 1024, less 1152).  bf16
// cache: bf16 MMAs, with the probabilities as the sum of two bf16 (2^-16).
//
// Work split: chunks of 4 tiles (one per warp), ordered by (sequence, head),
// in equal contiguous shares over a fixed grid, whatever the lengths are (a
// share is ceil(chunks / grid): the largest of any even split, and who holds a
// chunk is one division).  A
// CTA's share is cut where a (sequence, head) ends; one that it holds whole is
// written out, of one it shares it leaves (m, sum p, sum p v) in fp32 for
// attn_join_kernel, which adds the parts in order.  Where a cluster's CTAs can
// have a (sequence, head) to themselves with a few chunks each, they do, and
// join through distributed shared memory: no search, workspace or second
// kernel (one sequence of 1000, 4 heads, bf16: 7.6 -> 6.9 us).
#pragma once

#include <cuda_fp16.h>
#include <float.h>

#include "common.cuh"

namespace w8a8 {

constexpr int kKernelIdKvAppend = 10;
constexpr int kKernelIdAttn = 11;

// ---------------------------------------------------------------- cache write
struct KvSide {
    const uint16_t* x;      // bf16 [T, Hkv, D]
    int64_t ldx;
    void* cache;            // [num_pages, Hkv, page, D]
    float* scale;           // [num_pages, Hkv, page] or null (bf16)
};
struct KvAppendArgs {
    KvSide k, v;
    const int64_t* slots;
    int64_t T, num_pages;
    int Hkv, page_shift;
};

// The key's row and the value's by the same lanes, two independent chains that
// hide each other's latency: bf16 32 bytes of each a lane (4096 tokens, 8 heads
// of 128: 5.0 us against 5.5 with 16), int8 16 (9.7 against 10.3, and 64 tokens
// 2.7 against 3.9: the divisions and codes are the latency there).  Bound by
// latency at decode sizes, by the bytes at prompt sizes.
template <int D, bool INT8>
struct AppendCfg {
    static constexpr int NV = INT8 ? 1 : 2;          // 16-byte vectors a lane and row
    static constexpr int L = D / (8 * NV);           // lanes a row
};
template <int D, bool INT8>
__global__ void __launch_bounds__(256) kv_append_kernel(KvAppendArgs a) {
    constexpr int NV = AppendCfg<D, INT8>::NV, L = AppendCfg<D, INT8>::L;
    const int64_t t = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
    const int l = threadIdx.x % L, h = blockIdx.y;
    uint4 x[2][NV] = {};
    int64_t slot = -1;
    asm volatile("griddepcontrol.wait;" ::: "memory");   // may overlap the kernel before it
    if (t < a.T) {
        slot = __ldca(a.slots + t);
        const uint4* ks = reinterpret_cast<const uint4*>(a.k.x + t * a.k.ldx + (int64_t)h * D) + l;
        const uint4* vs = reinterpret_cast<const uint4*>(a.v.x + t * a.v.ldx + (int64_t)h * D) + l;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            x[0][i] = __ldca(ks + i * L);
            x[1][i] = __ldca(vs + i * L);
        }
        if (slot >= 0 && (slot >> a.page_shift) >= a.num_pages) {
            record_error(W8A8_ERR_INVALID_ARG, (kKernelIdKvAppend << 16) | 1);
            slot = -1;
        }
    }
    const int64_t at = (((slot >> a.page_shift) * a.Hkv + h) << a.page_shift) + (slot & ((1 << a.page_shift) - 1));
    if constexpr (!INT8) {
        if (slot >= 0) {
            uint4* kd = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.k.cache) + at * D) + l;
            uint4* vd = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.v.cache) + at * D) + l;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                kd[i * L] = x[0][i];
                vd[i * L] = x[1][i];
            }
        }
    } else {
        // the row maxima as in the activation quant: |bf16| orders like its bits; the
        // fp32 maximum, which skips NaN, where one of those shows up
        uint32_t both = 0u;   // key's | value's << 16
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const uint4& v = x[s][0];
            const uint32_t m = max_u16x2(max_u16x2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                         max_u16x2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
            both |= max(m & 0xffffu, m >> 16) << (16 * s);
        }
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) both = max_u16x2(both, __shfl_xor_sync(0xffffffffu, both, o));
        float top[2] = {__uint_as_float(both << 16), __uint_as_float(both & 0xffff0000u)};
        if (__any_sync(0xffffffffu, (both & 0xffffu) > 0x7f80u || (both >> 16) > 0x7f80u)) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const uint32_t w[4] = {x[s][0].x, x[s][0].y, x[s][0].z, x[s][0].w};
                top[s] = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    top[s] = fmaxf(top[s], fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xffff0000u))));
#pragma unroll
                for (int o = L / 2; o > 0; o >>= 1) top[s] = fmaxf(top[s], __shfl_xor_sync(0xffffffffu, top[s], o));
            }
        }
        // scale and reciprocal of the key by the even lanes, of the value by the odd
        const QuantRow mine(l & 1 ? top[1] : top[0]);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const uint32_t w[4] = {x[s][0].x, x[s][0].y, x[s][0].z, x[s][0].w};
            const int from = (threadIdx.x & 30) + s;
            const QuantRow q(__shfl_sync(0xffffffffu, mine.s, from), __shfl_sync(0xffffffffu, mine.rcp, from));
            float f[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
            uint32_t c[2];
            quant_codes<2>(f, q, c);
            if (slot >= 0) {
                const KvSide& side = s ? a.v : a.k;
                *(reinterpret_cast<uint2*>(reinterpret_cast<int8_t*>(side.cache) + at * D) + l) = make_uint2(c[0], c[1]);
                if (l == 0) side.scale[at] = q.s;
            }
        }
    }
}

// ---------------------------------------------------------------- attention
constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = 32 * kAttnWarps;
constexpr int kAttnMaxB = 4096;

struct AttnArgs {
    const uint16_t* q;      // bf16 [B, Hq, D], sequence stride ldq
    int64_t ldq;
    const void* kc;
    const void* vc;
    const float* ks;
    const float* vs;
    const int32_t* table;
    int64_t ld_table;
    const int32_t* lengths;
    uint16_t* y;
    int B, Hq, Hkv, G, qtiles;
    int64_t num_pages;
    int64_t cap;            // max_pages * page_size
    int page_shift;
    float scale_log2;       // scale * log2(e)
    float* part_o;          // [grid][2][QT][D]
    float2* part_ml;        // [grid][2][QT]
    int grid;               // CTAs of the attention kernel
    int csize;              // CTAs of a cluster that has a unit to itself; 0: shares
};

// Tokens of a warp's tile: 4 KB of keys (8 KB for the bf16 rows of 512 bytes,
// since an MMA takes 16 tokens).
template <int D, bool INT8>
constexpr int attn_tt() { return INT8 ? (D == 256 ? 16 : 32) : (D == 64 ? 32 : 16); }

__device__ __forceinline__ int64_t attn_len(const AttnArgs& a, int b) {
    const int64_t n = __ldca(a.lengths + b);
    return n < 0 ? 0 : (n > a.cap ? a.cap : n);
}

// CTA's share [u0, u1) of the (sum over b of chunks(b)) * heads units, the
// sequence that holds u0 and the chunks before it.  All threads call it.
struct AttnPlace {
    int b;
    int64_t before, u0, u1;   // the CTA's units
};
template <int CH, int NT>
__device__ __forceinline__ AttnPlace attn_place(const AttnArgs& a, int cta, int64_t heads) {
    __shared__ int64_t wsum[NT / 32];
    __shared__ AttnPlace place;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int seqs = (a.B + NT - 1) / NT;   // a thread's
    const int b0 = min(tid * seqs, a.B), b1 = min(b0 + seqs, a.B);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += (attn_len(a, b) + CH - 1) / CH;
    int64_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int64_t total = 0, before = inc - mine;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += wsum[w];
        total += wsum[w];
    }
    total *= heads;
    const int64_t per = (total + a.grid - 1) / a.grid;
    const int64_t u0 = per * cta < total ? per * cta : total;
    if (u0 >= before * heads && u0 < (before + mine) * heads) {
        int b = b0;
        for (; b < b1 - 1; ++b) {
            const int64_t n = (attn_len(a, b) + CH - 1) / CH;
            if (u0 < (before + n) * heads) break;
            before += n;
        }
        place.b = b;
        place.before = before;
    }
    if (tid == 0) {
        place.u0 = u0;
        place.u1 = u0 + per < total ? u0 + per : total;
    }
    __syncthreads();
    return place;
}

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two bytes (offset to unsigned by ^ 0x80) at positions SEL picks -> two exact fp16 codes.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t code_pair(uint32_t biased) {
    const uint32_t h = __byte_perm(biased, 0x64646464u, SEL);
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&h), __half2half2(__ushort_as_half(0x6480)));   // 1152
    return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ float attn_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Exponent of the power of two that values of up to x are divided by: x comes to [2^14, 2^15).
__device__ __forceinline__ int attn_unit(float x) { return max((int)(__float_as_uint(x) >> 23) - 127 - 14, -126); }

// 16 bytes to shared memory, the first `bytes` of them from global memory, zeros behind.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}

// Sizes of one instance.  NQ: tiles of 8 query heads a pass.
template <int D, bool INT8, int NQ>
struct AttnCfg {
    static constexpr int TT = attn_tt<D, INT8>();
    static constexpr int CH = kAttnWarps * TT;
    static constexpr int QT = 8 * NQ;
    static constexpr int ROW = INT8 ? D : 2 * D;             // bytes of a cache row
    static constexpr int U = ROW / 16;                       // 16-byte units of a row
    static constexpr int kScales = INT8 ? TT * 4 : 0;
    static constexpr int kStage = 2 * (TT * ROW + kScales);  // keys, values, their scales
    // (int8 rows of 64: three stages, so that a fourth CTA fits an SM -- its short
    // tiles are bound by the latency of a warp's chain: 32 sequences of up to 16384,
    // 8 x 4 heads, 89 -> 81 us against four stages and three CTAs)
    static constexpr int kStages = kStage <= 4608 ? 3 : 2;
    static constexpr int kRing = kStages * kStage;           // a warp's
    // words of Q's fragments per lane and MMA k step: kPlanes of int8, or bf16
    static constexpr int kPlanes = NQ == 1 ? 4 : 3;
    static constexpr int kQWords = INT8 ? 2 * NQ * kPlanes : 2 * NQ;
    static constexpr int kQSteps = INT8 ? D / 32 : D / 16;
    static constexpr int kQ = kQSteps * 32 * kQWords * 4;
    static constexpr int kJoin = kAttnWarps * QT * (D + 4) * 4;   // over the ring, between segments
    static constexpr int kBytes = kQ + (kAttnWarps * kRing > kJoin ? kAttnWarps * kRing : kJoin);
    // CTAs an SM: what shared memory holds (some 2 KB more is static and reserved),
    // less where the registers would spill
    static constexpr int kFit = (227 * 1024) / (kBytes + 2048);
    static constexpr int kMost = NQ == 1 ? 4 : (D == 256 ? 2 : 3);
    static constexpr int kMinB = kFit < 1 ? 1 : (kFit < kMost ? kFit : kMost);
};

template <int D, bool INT8, int NQ>
__global__ void __launch_bounds__(kAttnThreads, (AttnCfg<D, INT8, NQ>::kMinB)) paged_attention_kernel(AttnArgs a) {
    using Cfg = AttnCfg<D, INT8, NQ>;
    constexpr int TT = Cfg::TT, CH = Cfg::CH, QT = Cfg::QT, ROW = Cfg::ROW, U = Cfg::U, ST = Cfg::kStages;
    constexpr int KL = ROW / 64;                      // 16-byte key loads per token and lane
    constexpr int NT8 = TT / 8;                       // score tiles of 8 tokens
    constexpr int VB = U == 4 ? 8 : 16;               // bytes per value load
    constexpr int VL = ROW / (8 * VB);                // value loads per token and lane
    constexpr int VW = VB / 4;                        // words per value load
    constexpr int OT = D / 16;                        // output tiles of 16 d
    constexpr int DPL = INT8 ? VB : VB / 2;           // d's per value load and lane
    constexpr int QW = Cfg::kQWords, PL = Cfg::kPlanes, kQBits = 8 * PL - 2;
    constexpr int QM = NQ == 1 ? PL / 2 : PL;         // MMAs of a step of int8 scores

    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float sm[kAttnWarps][QT], sl[kAttnWarps][QT];
    __shared__ float2 cml[QT];                        // the CTA's (m, sum p), in a cluster
    uint32_t* qs = reinterpret_cast<uint32_t*>(smem);         // Q's fragments: [step][word / 2][lane][2]
    float* so = reinterpret_cast<float*>(smem + Cfg::kQ);     // [warp][QT][D + 4], between segments

    // may overlap the kernel before it, whose results (and whose reads of y and of the
    // workspace) are complete only now (launched so, and with a plain stream order: one
    // sequence of 1000, 4 heads, bf16, 6.8 / 7.2 us)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // attn_join_kernel may launch; it waits for this grid before it reads the parts
    if (a.csize == 0) asm volatile("griddepcontrol.launch_dependents;");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const uint32_t ring = smem_u32(smem) + Cfg::kQ + warp * Cfg::kRing;
    const uint32_t qbase = smem_u32(smem) + lane * 8;
    const int64_t heads = (int64_t)a.Hkv * a.qtiles;
    int64_t u, u1, before;
    int b;
    if (a.csize == 0) {
        const AttnPlace place = attn_place<CH, kAttnThreads>(a, blockIdx.x, heads);
        u = place.u0;
        u1 = place.u1;
        b = place.b;
        before = place.before;
    } else {
        // an even part of one unit's chunks, numbered as if the sequence were the only one
        const int unit = blockIdx.x / a.csize, r = blockIdx.x - unit * a.csize;
        b = unit / (int)heads;
        before = 0;
        const int64_t n = (attn_len(a, b) + CH - 1) / CH, at = (unit - b * heads) * n;
        u = at + n * r / a.csize;
        u1 = at + n * (r + 1) / a.csize;
        if (u == u1) {   // nothing for this CTA
            for (int i = threadIdx.x; i < QT * (D / 4); i += kAttnThreads)
                *reinterpret_cast<float4*>(so + i / (D / 4) * (D + 4) + 4 * (i % (D / 4))) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (threadIdx.x < QT) cml[threadIdx.x] = make_float2(-INFINITY, 0.0f);
        }
    }
    const int pmask = (1 << a.page_shift) - 1;
    bool bad = false;
    // this lane's places in a stage, per copy instruction of 32 units (they repeat every kDst)
    constexpr int kDst = U == 8 ? 2 : (U >= 16 ? 8 * U / 32 : 1);
    uint32_t kdst[kDst], vdst[kDst];
#pragma unroll
    for (int x = 0; x < kDst; ++x) {
        const int r = (x * 32 + lane) / U, un = (x * 32 + lane) % U;
        kdst[x] = (r * U + (U == 4 ? un : un ^ ((r & 1) << 2))) * 16;
        vdst[x] = TT * ROW + (r * U + (U == 4 ? un : un ^ (((r >> 1) & 3) << 1))) * 16;
    }
    const uint8_t* kc_lane = reinterpret_cast<const uint8_t*>(a.kc) + 16 * lane;
    const uint8_t* vc_lane = reinterpret_cast<const uint8_t*>(a.vc) + 16 * lane;

    while (u < u1) {
        const int64_t len = attn_len(a, b);
        const int64_t nb = (len + CH - 1) / CH;
        if (u >= (before + nb) * heads) {
            before += nb;
            ++b;
            continue;
        }
        const int64_t rel = u - before * heads;
        const int hq = (int)(rel / nb);
        const int64_t ch0 = rel - hq * nb;
        const int64_t seg = nb - ch0 < u1 - u ? nb - ch0 : u1 - u;
        const int h = hq / a.qtiles, qt = hq - h * a.qtiles;
        const int nq = min(QT, a.G - qt * QT);        // query heads of this tile
        const int q0 = h * a.G + qt * QT;             // the first of them

        // ---- the warp's tiles: ch0 * 4 + warp, every fourth
        const int64_t tile_end = (ch0 + seg) * kAttnWarps;
        const int32_t* trow = a.table + (int64_t)b * a.ld_table;
        auto page_of = [&](int64_t tile) -> int {     // of the tile's token number `lane`; < 0: absent
            const int64_t t = tile * TT + lane;
            if (tile >= tile_end || lane >= TT || t >= len) return -1;
            const int pg = __ldca(trow + (t >> a.page_shift));
            if (pg < 0 || pg >= a.num_pages) {
                bad = true;
                return -1;
            }
            return pg;
        };
        // Copies a tile: eight tokens at a time lie in one page, their rows one
        // after the other.  In shared memory a key row's units are XORed with 4
        // on odd rows and a value row's with 2 * (row / 2 % 4), which keeps both
        // reads below (8 rows x 4 units; 4 even or odd rows x 2 units) free of
        // bank conflicts.  Each lane finds its token's row; the rest is one
        // 64-bit addition per eight tokens and constants.
        auto issue = [&](int pages, int64_t tile, int stage) {
            const uint32_t ks = ring + stage * Cfg::kStage;
            const int64_t t0 = tile * TT;
            const int64_t row = pages < 0 ? 0 : (((int64_t)pages * a.Hkv + h) << a.page_shift) + (((int)t0 + lane) & pmask);
            const uint64_t off = (uint64_t)row * ROW;
            const uint32_t off_lo = (uint32_t)off, off_hi = (uint32_t)(off >> 32);
            const bool full = __all_sync(0xffffffffu, pages >= 0 || lane >= TT);
#pragma unroll
            for (int j = 0; j < NT8; ++j) {
                const uint64_t from = ((uint64_t)__shfl_sync(0xffffffffu, off_hi, 8 * j) << 32) | __shfl_sync(0xffffffffu, off_lo, 8 * j);
                const uint8_t* ksrc = kc_lane + from;
                const uint8_t* vsrc = vc_lane + from;
                if (full) {
#pragma unroll
                    for (int x = 0; x < U / 4; ++x) {
                        cp_async16(ks + kdst[x % kDst] + (8 * j * U + 32 * (x - x % kDst)) * 16, ksrc + 512 * x);
                        cp_async16(ks + vdst[x % kDst] + (8 * j * U + 32 * (x - x % kDst)) * 16, vsrc + 512 * x);
                    }
                } else {
                    const int here = __shfl_sync(0xffffffffu, pages, 8 * j) < 0 ? 0 : (int)(len - t0 - 8 * j < 8 ? len - t0 - 8 * j : 8);
#pragma unroll
                    for (int x = 0; x < U / 4; ++x) {
                        const uint32_t n = (x * 32 + lane) / U < here ? 16u : 0u;
                        cp_async16(ks + kdst[x % kDst] + (8 * j * U + 32 * (x - x % kDst)) * 16, ksrc + 512 * x, n);
                        cp_async16(ks + vdst[x % kDst] + (8 * j * U + 32 * (x - x % kDst)) * 16, vsrc + 512 * x, n);
                    }
                }
            }
            if (INT8) {
                // lanes [0, 2 NT8): keys' scales, four tokens each; then values'
                const int tok = (lane * 4) % TT;
                const uint64_t from = ((uint64_t)__shfl_sync(0xffffffffu, (uint32_t)(row >> 32), tok) << 32) |
                                      __shfl_sync(0xffffffffu, (uint32_t)row, tok);
                const int64_t left = __shfl_sync(0xffffffffu, pages, tok) < 0 ? 0 : len - t0 - tok;
                if (lane < 4 * NT8)
                    cp_async16(ks + 2 * TT * ROW + lane * 16, (lane < 2 * NT8 ? a.ks : a.vs) + from,
                               left >= 4 ? 16u : 4u * (uint32_t)left);
            }
        };
        int64_t tile = ch0 * kAttnWarps + warp;
#pragma unroll
        for (int s = 0; s < ST; ++s) {
            issue(page_of(tile + s * kAttnWarps), tile + s * kAttnWarps, s);
            cp_async_commit();
        }
        int pages_next = page_of(tile + ST * kAttnWarps);

        // ---- the query's fragments, a share of the k steps per warp
        float qscale[NQ];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            qscale[n] = a.scale_log2;
            const bool has = 8 * n + g < nq;
            const uint16_t* qrow = a.q + (int64_t)b * a.ldq + (int64_t)(q0 + 8 * n + g) * D;
            if (INT8) {
                // 16 d's per key load and lane: d = 64 i + 16 c + e
                float amax = 0.0f;
                uint4 w[KL][2];
#pragma unroll
                for (int i = 0; i < KL; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        w[i][e] = make_uint4(0, 0, 0, 0);
                        if (has) w[i][e] = __ldca(reinterpret_cast<const uint4*>(qrow + 64 * i + 16 * c + 8 * e));
                        const uint32_t x[4] = {w[i][e].x, w[i][e].y, w[i][e].z, w[i][e].w};
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            amax = fmax_nan(amax, fmax_nan(fabsf(__uint_as_float(x[k] << 16)),
                                                           fabsf(__uint_as_float(x[k] & 0xffff0000u))));
                    }
                amax = fmax_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmax_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                // amax in [2^e, 2^(e+1)): integers below 2^kQBits; NaN and infinities pass through the scale
                const int e = max((int)(__float_as_uint(amax) >> 23) - 127, -90);
                const float up = __uint_as_float((uint32_t)(kQBits - 1 - e + 127) << 23);
                qscale[n] *= amax < INFINITY ? __uint_as_float((uint32_t)(e - (kQBits - 1) + 127) << 23) : __int_as_float(0x7fc00000);
#pragma unroll
                for (int i = 0; i < KL; ++i) {
                    if (i % kAttnWarps != warp) continue;
#pragma unroll
                    for (int st = 0; st < 2; ++st) {         // MMA step 2 i + st: d = 64 i + 16 c + 8 st + [0, 8)
                        const uint32_t x[4] = {w[i][st].x, w[i][st].y, w[i][st].z, w[i][st].w};
                        int p[PL][8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float f = __uint_as_float(k & 1 ? x[k / 2] & 0xffff0000u : x[k / 2] << 16);
                            int v = __float2int_rn(f * up);
#pragma unroll
                            for (int pl = PL - 1; pl > 0; --pl) {      // digits in [-128, 128)
                                p[pl][k] = (int)(int8_t)v;
                                v = (v - p[pl][k]) >> 8;
                            }
                            p[0][k] = v;
                        }
#pragma unroll
                        for (int pl = 0; pl < PL; ++pl)
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf) {
                                const uint32_t v = pack4_s8(p[pl][4 * hf], p[pl][4 * hf + 1], p[pl][4 * hf + 2], p[pl][4 * hf + 3]);
                                // NQ = 1: words (a0, a1, a2, a3) = planes 0, 1, 0, 1; then 2, 3, 2, 3.
                                // NQ = 2: plane by plane (a0, a1, a2, a3)
                                const int word = NQ == 1 ? 4 * (pl / 2) + 2 * hf + pl % 2 : 4 * pl + 2 * hf + n;
                                qs[(((2 * i + st) * (QW / 2) + word / 2) * 32 + lane) * 2 + (word & 1)] = v;
                            }
                    }
                }
            } else {
                // 8 d's per key load and lane: d = 32 i + 8 c + e; words (a0, a2), or (a0, a1, a2, a3) of two tiles
#pragma unroll
                for (int i = 0; i < KL; ++i) {
                    if (i % kAttnWarps != warp) continue;
                    uint4 w = make_uint4(0, 0, 0, 0);
                    if (has) w = __ldca(reinterpret_cast<const uint4*>(qrow + 32 * i + 8 * c));
                    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int word = (k & 1) * NQ + n;
                        qs[(((2 * i + k / 2) * (QW / 2) + word / 2) * 32 + lane) * 2 + (word & 1)] = x[k];
                    }
                }
            }
        }
        __syncthreads();

        float o[NQ][OT][4];
        float m[NQ], l[NQ];
        float big[NQ];            // int8: the largest p times value scale; o is in units of 2^attn_unit(big)
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            m[n] = -INFINITY;
            l[n] = 0.0f;
            big[n] = 0.0f;
#pragma unroll
            for (int i = 0; i < OT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[n][i][j] = 0.0f;
        }

        int stage = 0;
        for (; tile < tile_end; tile += kAttnWarps) {
            cp_async_wait<ST - 1>();
            __syncwarp();
            const uint32_t ks = ring + stage * Cfg::kStage, vs = ks + TT * ROW, cs = vs + TT * ROW;
            // ---- scores
            float s[NQ][NT8][2];
            if (INT8) {
                int acc[QM][NT8][4];   // of a pair of planes (NQ = 1) or a plane
#pragma unroll
                for (int x = 0; x < QM; ++x)
#pragma unroll
                    for (int j = 0; j < NT8; ++j)
#pragma unroll
                        for (int k = 0; k < 4; ++k) acc[x][j][k] = 0x4B400000;   // the bits of 1.5 * 2^23: sums come out as floats
#pragma unroll
                for (int i = 0; i < KL; ++i) {
                    uint4 kr[NT8];
#pragma unroll
                    for (int j = 0; j < NT8; ++j)
                        kr[j] = lds16(ks + ((8 * j + g) * U + (U == 4 ? c : (4 * i + c) ^ ((g & 1) << 2))) * 16);
#pragma unroll
                    for (int st = 0; st < 2; ++st) {
                        uint32_t q[QW];
#pragma unroll
                        for (int w = 0; w < QW / 2; ++w) {
                            const uint2 v = lds8(qbase + ((2 * i + st) * (QW / 2) + w) * 256);
                            q[2 * w] = v.x;
                            q[2 * w + 1] = v.y;
                        }
#pragma unroll
                        for (int j = 0; j < NT8; ++j) {
                            const uint32_t bk[2] = {st ? kr[j].z : kr[j].x, st ? kr[j].w : kr[j].y};
#pragma unroll
                            for (int x = 0; x < QM; ++x) {
                                const uint32_t aq[4] = {q[4 * x % QW], q[(4 * x + 1) % QW], q[(4 * x + 2) % QW], q[(4 * x + 3) % QW]};
                                mma_s8_16832(acc[x][j], aq, bk);
                            }
                        }
                    }
                }
                // planes join: |sums| <= 2^22, so sum + 1.5 * 2^23 is exact in fp32 and its bits were added up
                auto value = [](int bits) { return __fsub_rn(__int_as_float(bits), 12582912.0f); };
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int j = 0; j < NT8; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float sum = 0.0f;
#pragma unroll
                            for (int pl = PL - 1; pl >= 0; --pl) {
                                const float p = value(NQ == 1 ? acc[pl / 2][j][2 * (pl & 1) + e] : acc[pl % QM][j][2 * n + e]);
                                sum = pl == PL - 1 ? p : __fmaf_rn((float)(1u << (8 * (PL - 1 - pl))), p, sum);
                            }
                            s[n][j][e] = sum;
                        }
            } else {
                float acc[NT8][4];
#pragma unroll
                for (int j = 0; j < NT8; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[j][k] = 0.0f;
#pragma unroll
                for (int i = 0; i < KL; ++i) {
                    uint4 kr[NT8];
#pragma unroll
                    for (int j = 0; j < NT8; ++j) kr[j] = lds16(ks + ((8 * j + g) * U + ((4 * i + c) ^ ((g & 1) << 2))) * 16);
#pragma unroll
                    for (int st = 0; st < 2; ++st) {
                        uint32_t q[QW];
#pragma unroll
                        for (int w = 0; w < QW / 2; ++w) {
                            const uint2 v = lds8(qbase + ((2 * i + st) * (QW / 2) + w) * 256);
                            q[2 * w] = v.x;
                            q[2 * w + 1] = v.y;
                        }
#pragma unroll
                        for (int j = 0; j < NT8; ++j)
                            mma_bf16_16816(acc[j], q[0], NQ == 2 ? q[1] : 0u, NQ == 2 ? q[2 % QW] : q[1],
                                           NQ == 2 ? q[3 % QW] : 0u, st ? kr[j].z : kr[j].x, st ? kr[j].w : kr[j].y);
                    }
                }
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int j = 0; j < NT8; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) s[n][j][e] = acc[j][2 * n + e];
            }
            // ---- softmax of query rows g (and g + 8)
            const int64_t left = len - tile * TT;     // tokens from here on
            uint32_t there = 0xffffffffu;             // bit t: token t is there
            if (left < TT || __any_sync(0xffffffffu, lane < TT && bad)) {
                const int pg = page_of(tile);
                there = __ballot_sync(0xffffffffu, pg >= 0);
            }
            float2 ksc[NT8], vsc[NT8];
            if (INT8) {
#pragma unroll
                for (int j = 0; j < NT8; ++j) {
                    const uint2 kx = lds8(cs + (8 * j + 2 * c) * 4), vx = lds8(cs + TT * 4 + (8 * j + 2 * c) * 4);
                    ksc[j] = make_float2(__uint_as_float(kx.x), __uint_as_float(kx.y));
                    vsc[j] = make_float2(__uint_as_float(vx.x), __uint_as_float(vx.y));
                }
            }
            uint32_t pf[NQ][NT8], pl[NQ][NT8];        // pairs of fp16 or bf16: high and low parts
            float fac[NQ];
            bool rescale = false;
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                float x[NT8][2];
                float mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < NT8; ++j) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float v = s[n][j][e] * qscale[n];
                        if (INT8) v *= e ? ksc[j].y : ksc[j].x;
                        x[j][e] = v;
                    }
                }
                if (there != 0xffffffffu) {
#pragma unroll
                    for (int j = 0; j < NT8; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (!((there >> (8 * j + 2 * c + e)) & 1u)) x[j][e] = -INFINITY;
                }
#pragma unroll
                for (int j = 0; j < NT8; ++j) mx = fmaxf(mx, fmaxf(x[j][0], x[j][1]));
                // m = -inf: no token so far.  Tokens with scores of -inf alone: m is the lowest finite value, every
                // probability 0, and the output 0 / 0
                if (there) mx = fmaxf(mx, -FLT_MAX);
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float mn = fmaxf(m[n], mx);
                const float mu = mn == -INFINITY ? 0.0f : mn;
                const float corr = attn_ex2(m[n] - mu);
                m[n] = mn;
                float sum = 0.0f;
#pragma unroll
                for (int j = 0; j < NT8; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        x[j][e] = attn_ex2(x[j][e] - mu);
                        sum += x[j][e];
                    }
                l[n] = l[n] * corr + sum;
                if (INT8) {
                    // probabilities times the values' scales, brought to [0, 2^15) by a power of two
                    float um = 0.0f;
#pragma unroll
                    for (int j = 0; j < NT8; ++j) {
                        x[j][0] *= vsc[j].x;
                        x[j][1] *= vsc[j].y;
                        um = fmaxf(um, fmaxf(fabsf(x[j][0]), fabsf(x[j][1])));
                    }
                    um = fmaxf(um, __shfl_xor_sync(0xffffffffu, um, 1));
                    um = fmaxf(um, __shfl_xor_sync(0xffffffffu, um, 2));
                    // the unit follows the largest of all so far in the new reference, so fac stays below 2 (from
                    // the old unit's place instead, it fell by one with every rise of the maximum, however
                    // small, and o overflowed behind a hundred of them)
                    const float now = fmaxf(um, big[n] * corr);
                    const int eo = attn_unit(big[n]), en = attn_unit(now);
                    fac[n] = corr * __uint_as_float((uint32_t)min(max(eo - en + 127, 0), 254) << 23);
                    big[n] = now;
                    const float unit = __uint_as_float((uint32_t)(127 - en) << 23);
#pragma unroll
                    for (int j = 0; j < NT8; ++j) {
                        const float u0 = x[j][0] * unit, u1 = x[j][1] * unit;
                        const __half2 hv = __floats2half2_rn(u0, u1);
                        const float2 hf = __half22float2(hv);
                        const __half2 lv = __floats2half2_rn(u0 - hf.x, u1 - hf.y);
                        pf[n][j] = *reinterpret_cast<const uint32_t*>(&hv);
                        pl[n][j] = *reinterpret_cast<const uint32_t*>(&lv);
                    }
                } else {
                    fac[n] = corr;
#pragma unroll
                    for (int j = 0; j < NT8; ++j) {
                        const uint32_t hi = cvt_bf16x2(x[j][0], x[j][1]);
                        pf[n][j] = hi;
                        pl[n][j] = cvt_bf16x2(x[j][0] - __uint_as_float(hi << 16),
                                              x[j][1] - __uint_as_float(hi & 0xffff0000u));
                    }
                }
                rescale |= fac[n] != 1.0f;
            }
            if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    const float f0 = __shfl_sync(0xffffffffu, fac[n], 8 * c), f1 = __shfl_sync(0xffffffffu, fac[n], 8 * c + 4);
#pragma unroll
                    for (int i = 0; i < OT; ++i) {
                        o[n][i][0] *= f0;
                        o[n][i][1] *= f1;
                        o[n][i][2] *= f0;
                        o[n][i][3] *= f1;
                    }
                }
            }
            // ---- outputs
#pragma unroll
            for (int j = 0; j < NT8; j += 2) {
#pragma unroll
                for (int i = 0; i < VL; ++i) {
                    uint32_t vr[4][VW];               // tokens 8j + 2c, + 1, 8j + 8 + 2c, + 1
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const int r = 8 * (j + t / 2) + 2 * c + (t & 1);
                        if (VB == 16) {
                            const uint4 v = lds16(vs + (r * U + ((g + 8 * i) ^ (c << 1))) * 16);
                            vr[t][0] = v.x;
                            vr[t][1] = v.y;
                            vr[t][2 % VW] = v.z;
                            vr[t][3 % VW] = v.w;
                        } else {
                            const uint2 v = lds8(vs + r * ROW + 8 * g);
                            vr[t][0] = v.x;
                            vr[t][1] = v.y;
                        }
                    }
#pragma unroll
                    for (int w = 0; w < VW; ++w) {
                        if (INT8) {
                            // 4 d's: two output tiles
                            const uint32_t t0 = vr[0][w] ^ 0x80808080u, t1 = vr[1][w] ^ 0x80808080u;
                            const uint32_t t2 = vr[2][w] ^ 0x80808080u, t3 = vr[3][w] ^ 0x80808080u;
                            const uint32_t x0 = __byte_perm(t0, t1, 0x5140), x1 = __byte_perm(t0, t1, 0x7362);
                            const uint32_t y0 = __byte_perm(t2, t3, 0x5140), y1 = __byte_perm(t2, t3, 0x7362);
                            const uint32_t a0 = code_pair<0x4140>(x0), a1 = code_pair<0x4342>(x0);
                            const uint32_t a2 = code_pair<0x4140>(y0), a3 = code_pair<0x4342>(y0);
                            const uint32_t b0 = code_pair<0x4140>(x1), b1 = code_pair<0x4342>(x1);
                            const uint32_t b2 = code_pair<0x4140>(y1), b3 = code_pair<0x4342>(y1);
#pragma unroll
                            for (int n = 0; n < NQ; ++n) {
                                mma_f16_16816(o[n][(i * VW + w) * 2], a0, a1, a2, a3, pf[n][j], pf[n][j + 1]);
                                mma_f16_16816(o[n][(i * VW + w) * 2 + 1], b0, b1, b2, b3, pf[n][j], pf[n][j + 1]);
                                mma_f16_16816(o[n][(i * VW + w) * 2], a0, a1, a2, a3, pl[n][j], pl[n][j + 1]);
                                mma_f16_16816(o[n][(i * VW + w) * 2 + 1], b0, b1, b2, b3, pl[n][j], pl[n][j + 1]);
                            }
                        } else {
                            const uint32_t a0 = __byte_perm(vr[0][w], vr[1][w], 0x5410);
                            const uint32_t a1 = __byte_perm(vr[0][w], vr[1][w], 0x7632);
                            const uint32_t a2 = __byte_perm(vr[2][w], vr[3][w], 0x5410);
                            const uint32_t a3 = __byte_perm(vr[2][w], vr[3][w], 0x7632);
#pragma unroll
                            for (int n = 0; n < NQ; ++n) {
                                mma_bf16_16816(o[n][i * VW + w], a0, a1, a2, a3, pf[n][j], pf[n][j + 1]);
                                mma_bf16_16816(o[n][i * VW + w], a0, a1, a2, a3, pl[n][j], pl[n][j + 1]);
                            }
                        }
                    }
                }
            }
            __syncwarp();   // the stage has been read
            const int64_t next = tile + ST * kAttnWarps;
            issue(pages_next, next, stage);
            cp_async_commit();
            pages_next = page_of(next + kAttnWarps);
            stage = stage + 1 == ST ? 0 : stage + 1;
        }

        // ---- join of the four warps, over the rings (whose copies have all landed)
        cp_async_wait<0>();
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            l[n] += __shfl_xor_sync(0xffffffffu, l[n], 1);
            l[n] += __shfl_xor_sync(0xffffffffu, l[n], 2);
            if (c == 0) {
                sm[warp][8 * n + g] = m[n];
                sl[warp][8 * n + g] = l[n];
            }
            float un = 1.0f;
            if (INT8) un = __uint_as_float((uint32_t)(attn_unit(big[n]) + 127) << 23);
            const float u0f = __shfl_sync(0xffffffffu, un, 8 * c), u1f = __shfl_sync(0xffffffffu, un, 8 * c + 4);
            // tile i covers d = 8 DPL (i / (DPL / 2)) + DPL g + 2 (i % (DPL / 2)), + 1
            float* dst = so + (warp * QT + 8 * n + 2 * c) * (D + 4);
#pragma unroll
            for (int i = 0; i < OT; i += 2) {
                const int d = 8 * DPL * (i / (DPL / 2)) + DPL * g + 2 * (i % (DPL / 2));
                *reinterpret_cast<float4*>(dst + d) =
                    make_float4(o[n][i][0] * u0f, o[n][i][2] * u0f, o[n][i + 1][0] * u0f, o[n][i + 1][2] * u0f);
                *reinterpret_cast<float4*>(dst + D + 4 + d) =
                    make_float4(o[n][i][1] * u1f, o[n][i][3] * u1f, o[n][i + 1][1] * u1f, o[n][i + 1][3] * u1f);
            }
        }
        __syncthreads();
        const bool whole = seg == nb;
        const int slot = (ch0 == 0) ? 1 : 0;          // 0: it began in an earlier CTA
        const int64_t pbase = ((int64_t)blockIdx.x * 2 + slot) * QT;
        for (int i = threadIdx.x; i < nq * (D / 4); i += kAttnThreads) {
            const int qh = i / (D / 4), d = 4 * (i - qh * (D / 4));
            float mm = sm[0][qh];
#pragma unroll
            for (int w = 1; w < kAttnWarps; ++w) mm = fmaxf(mm, sm[w][qh]);
            const float mu = mm == -INFINITY ? 0.0f : mm;
            float ll = 0.0f;
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) {
                const float f = attn_ex2(sm[w][qh] - mu);
                const float4 v = *reinterpret_cast<const float4*>(so + (w * QT + qh) * (D + 4) + d);
                ll += sl[w][qh] * f;
                acc.x += v.x * f;
                acc.y += v.y * f;
                acc.z += v.z * f;
                acc.w += v.w * f;
            }
            if (a.csize != 0) {
                // over the first warp's values, which no other thread reads
                *reinterpret_cast<float4*>(so + qh * (D + 4) + d) = acc;
                if (d == 0) cml[qh] = make_float2(mm, ll);
            } else if (whole) {
                const float r = mm == -INFINITY ? 0.0f : 1.0f / ll;
                *reinterpret_cast<uint2*>(a.y + ((int64_t)b * a.Hq + q0 + qh) * D + d) =
                    make_uint2(cvt_bf16x2(acc.x * r, acc.y * r), cvt_bf16x2(acc.z * r, acc.w * r));
            } else {
                *reinterpret_cast<float4*>(a.part_o + (pbase + qh) * D + d) = acc;
                if (d == 0) a.part_ml[pbase + qh] = make_float2(mm, ll);
            }
        }
        __syncthreads();   // before the next segment's copies and query
        u += seg;
    }
    if (a.csize != 0) {
        // ---- join of the cluster: each CTA an even part of the outputs
        cluster_sync_all();
        const int unit = blockIdx.x / a.csize, r = blockIdx.x - unit * a.csize;
        const int hq = unit - b * (int)heads, h = hq / a.qtiles, qt = hq - h * a.qtiles;
        const int nq = min(QT, a.G - qt * QT), q0 = h * a.G + qt * QT;
        const uint32_t so_at = smem_u32(so), ml_at = smem_u32(cml);
        for (int i = r * kAttnThreads + threadIdx.x; i < nq * (D / 4); i += a.csize * kAttnThreads) {
            const int qh = i / (D / 4), d = 4 * (i - qh * (D / 4));
            float2 ml[8];
            float4 v[8];
            float mm = -INFINITY;
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                ml[p] = make_float2(-INFINITY, 0.0f);
                v[p] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (p < a.csize) {
                    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                                 : "=f"(ml[p].x), "=f"(ml[p].y)
                                 : "r"(mapa_shared(ml_at + qh * 8, p)));
                    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(v[p].x), "=f"(v[p].y), "=f"(v[p].z), "=f"(v[p].w)
                                 : "r"(mapa_shared(so_at + (qh * (D + 4) + d) * 4, p)));
                }
                mm = fmaxf(mm, ml[p].x);
            }
            const float mu = mm == -INFINITY ? 0.0f : mm;
            float ll = 0.0f;
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                const float f = attn_ex2(ml[p].x - mu);
                ll += ml[p].y * f;
                acc.x += v[p].x * f;
                acc.y += v[p].y * f;
                acc.z += v[p].z * f;
                acc.w += v[p].w * f;
            }
            const float inv = mm == -INFINITY ? 0.0f : 1.0f / ll;
            *reinterpret_cast<uint2*>(a.y + ((int64_t)b * a.Hq + q0 + qh) * D + d) =
                make_uint2(cvt_bf16x2(acc.x * inv, acc.y * inv), cvt_bf16x2(acc.z * inv, acc.w * inv));
        }
        cluster_sync_all();   // no CTA leaves while another reads its part
    }
    if (bad) record_error(W8A8_ERR_INVALID_ARG, (kKernelIdAttn << 16) | 1);
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < a.B; i += kAttnThreads)
            if (__ldca(a.lengths + i) > a.cap) record_error(W8A8_ERR_INVALID_ARG, (kKernelIdAttn << 16) | 2);
}

// Joins the parts of the (sequence, head) units that several CTAs shared, and
// writes the zeros of empty sequences.  Blocks (x, y): unit x, slice y of its
// outputs, four d's a thread; threads beyond the slice's take every NG-th part
// and meet in shared memory in a fixed order.  Latency is all that this kernel
// costs, so the loads of four parts are in flight at a time.
constexpr int kAttnJoinThreads = 256;
template <int D, int CH, int NQ>
__global__ void __launch_bounds__(kAttnJoinThreads) attn_join_kernel(AttnArgs a, int per_cta) {
    constexpr int QT = 8 * NQ, NT = kAttnJoinThreads;
    __shared__ int64_t red[2][NT / 32];
    __shared__ float4 racc[NT];
    __shared__ float2 rml[NT];
    const int64_t heads = (int64_t)a.Hkv * a.qtiles;
    const int b = (int)(blockIdx.x / heads), hq = (int)(blockIdx.x - b * heads);
    const int h = hq / a.qtiles, qt = hq - h * a.qtiles;
    const int nq = min(QT, a.G - qt * QT);
    const int q0 = h * a.G + qt * QT;
    // chunks before this sequence, and in all
    int64_t before = 0, total = 0;
    for (int i = threadIdx.x; i < a.B; i += NT) {
        const int64_t n = (attn_len(a, i) + CH - 1) / CH;
        total += n;
        if (i < b) before += n;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, o);
        total += __shfl_xor_sync(0xffffffffu, total, o);
    }
    if ((threadIdx.x & 31) == 0) {
        red[0][threadIdx.x >> 5] = before;
        red[1][threadIdx.x >> 5] = total;
    }
    __syncthreads();
    before = total = 0;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) {
        before += red[0][i];
        total += red[1][i];
    }
    total *= heads;
    const int64_t nb = (attn_len(a, b) + CH - 1) / CH;
    const int64_t us = before * heads + hq * nb, ue = us + nb;   // this unit's chunks
    const int64_t per = (total + a.grid - 1) / a.grid;
    const int i0 = nb ? (int)(us / per) : 0, i1 = nb ? (int)((ue - 1) / per) : -1;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (nb && i0 == i1) return;   // written by its CTA
    const int item = threadIdx.x % per_cta, grp = threadIdx.x / per_cta, ng = NT / per_cta;
    const int i = blockIdx.y * per_cta + item;
    const int qh = i / (D / 4), d = 4 * (i - qh * (D / 4));
    float mm = -INFINITY, ll = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto add = [&](const float2& ml, const float4& v) {
        const float mn = fmaxf(mm, ml.x);
        const float mu = mn == -INFINITY ? 0.0f : mn;
        const float f0 = attn_ex2(mm - mu), f = attn_ex2(ml.x - mu);
        mm = mn;
        ll = ll * f0 + ml.y * f;
        acc.x = acc.x * f0 + v.x * f;
        acc.y = acc.y * f0 + v.y * f;
        acc.z = acc.z * f0 + v.z * f;
        acc.w = acc.w * f0 + v.w * f;
    };
    if (qh < nq) {
        for (int k = i0 + grp; k <= i1; k += 4 * ng) {
            float2 ml[4];
            float4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int kk = k + j * ng;
                const int64_t p = ((int64_t)kk * 2 + (kk == i0 ? 1 : 0)) * QT + qh;
                ml[j] = make_float2(-INFINITY, 0.0f);
                v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (kk <= i1) {
                    ml[j] = __ldcg(&a.part_ml[p]);
                    v[j] = __ldcg(reinterpret_cast<const float4*>(a.part_o + p * D + d));
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) add(ml[j], v[j]);
        }
    }
    if (ng > 1) {
        racc[threadIdx.x] = acc;
        rml[threadIdx.x] = make_float2(mm, ll);
        __syncthreads();
        if (grp != 0) return;
        for (int j = 1; j < ng; ++j) add(rml[j * per_cta + item], racc[j * per_cta + item]);
    }
    if (qh >= nq) return;
    const float r = mm == -INFINITY ? 0.0f : 1.0f / ll;
    *reinterpret_cast<uint2*>(a.y + ((int64_t)b * a.Hq + q0 + qh) * D + d) =
        make_uint2(cvt_bf16x2(acc.x * r, acc.y * r), cvt_bf16x2(acc.z * r, acc.w * r));
}

}  // namespace w8a8

// The paged key-value cache (int8 codes with one fp32 scale per token and
// head, or bf16) and the attention of one new token over it.
//
//   l_t = scale * (q . k_t),  p_t = e^(l_t - m),  m = max_t l_t
//   y   = sum_t p_t v_t / sum_t p_t
//
// Bound by the cache's bytes: each key and value is read once, by whichever
// CTA holds its part of the context, for all the query heads that share it.
// The arithmetic rides on warp MMAs (m16n8k16, fp32 sums) whose fragments are
// the loaded registers themselves: no shared memory in the loop.
//
//   lane = 4 g + c (g = 0..7, c = 0..3); a tile of TT tokens per warp step
//   scores   S[query, token] = Q (16 x 16 over d) * K^T (16 d x 8 tokens):
//     lane loads 16 contiguous bytes of token row 8j + g; which d a fragment
//     slot means is free as long as Q's registers hold the same d's, so the
//     16 bytes feed the B operand as they are (four steps of int8, two of bf16)
//   outputs  O^T[d, query] = V^T (16 d x 16 tokens) * P^T (16 tokens x 8):
//     the scores' accumulators (query g, tokens 8j + 2c, + 1) are the B
//     operand's layout already; lane loads 16 contiguous bytes of d from each
//     of its tokens and pairs them across tokens with byte permutes
//
// int8 codes become fp16 exactly: the bytes, offset to unsigned, are placed
// under the exponent of 1024 (1024 + u), less 1152.  The query is scaled per
// head by a power of two to fp16 (8 significant bits fit 11: exact but for
// elements 2^-15 below the largest); the scales of keys multiply the scores,
// those of values the probabilities, which are then brought to [0, 2) by a
// running power of two per query before they round to fp16 (2^-12, an eighth
// of the output's own rounding).  With a bf16 cache the probabilities go in as
// the sum of two bf16 (2^-17).
//
// Work split: chunks of 4 tiles (one per warp), ordered by (sequence, head),
// in equal contiguous shares over a fixed grid, whatever the lengths are.  A
// CTA's share is cut where a (sequence, head) ends; one that it holds whole is
// written out, of one it shares it leaves (m, sum p, sum p v) in fp32 for
// attn_join_kernel, which adds the parts in order.
#pragma once

#include <cuda_fp16.h>

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

// D / 8 lanes per (token, head) row, 16 bytes each; the key's and the value's
// rows side by side along the grid.  Bound by latency at decode sizes, by the
// bytes at prompt sizes.
template <int D, bool INT8>
__global__ void __launch_bounds__(256) kv_append_kernel(KvAppendArgs a) {
    constexpr int L = D / 8;                 // lanes per row
    const KvSide s = blockIdx.y == 0 ? a.k : a.v;
    const int64_t row = ((int64_t)blockIdx.x * 256 + threadIdx.x) / L;
    const int l = threadIdx.x % L;
    const int64_t t = row / a.Hkv;
    const int h = (int)(row - t * a.Hkv);
    int64_t slot = -1;
    if (t < a.T) {
        slot = __ldg(a.slots + t);
        if (slot >= 0 && (slot >> a.page_shift) >= a.num_pages) {
            record_error(W8A8_ERR_INVALID_ARG, (kKernelIdKvAppend << 16) | 1);
            slot = -1;
        }
    }
    uint4 v = make_uint4(0, 0, 0, 0);
    if (slot >= 0) v = __ldg(reinterpret_cast<const uint4*>(s.x + t * s.ldx + (int64_t)h * D + 8 * l));
    const int64_t at = (((slot >> a.page_shift) * a.Hkv + h) << a.page_shift) + (slot & ((1 << a.page_shift) - 1));
    if (!INT8) {
        if (slot >= 0) *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(s.cache) + at * D + 8 * l) = v;
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float f[8], m = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        m = fmaxf(m, fmaxf(fabsf(f[2 * i]), fabsf(f[2 * i + 1])));
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const QuantRow q(m);
    uint32_t c[2];
    quant_codes<2>(f, q, c);
    if (slot >= 0) {
        *reinterpret_cast<uint2*>(reinterpret_cast<int8_t*>(s.cache) + at * D + 8 * l) = make_uint2(c[0], c[1]);
        if (l == 0) s.scale[at] = q.s;
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
};

// Tokens of a warp's tile: 4 KB of keys (8 KB for the bf16 rows of 512 bytes,
// since an MMA takes 16 tokens).
template <int D, bool INT8>
constexpr int attn_tt() { return INT8 ? (D == 256 ? 16 : 32) : (D == 64 ? 32 : 16); }

__device__ __forceinline__ int64_t attn_len(const AttnArgs& a, int b) {
    const int64_t n = __ldg(a.lengths + b);
    return n < 0 ? 0 : (n > a.cap ? a.cap : n);
}

// Sequence that holds unit u0 of (sum over b of chunks(b)) * heads units, the
// chunks before it, and the units in all.  All threads of the CTA call it.
struct AttnPlace {
    int b;
    int64_t before, total;
};
template <int CH, int NT>
__device__ __forceinline__ AttnPlace attn_place(const AttnArgs& a, int grid, int cta, int64_t heads) {
    __shared__ int64_t wsum[NT / 32];
    __shared__ AttnPlace place;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.B + NT - 1) / NT;
    const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
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
    const int64_t u0 = total * cta / grid;
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
    if (tid == 0) place.total = total;
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

// NQ: tiles of 8 query heads a pass (QT = 8 NQ of the heads that share a key-value head).
template <int D, bool INT8, int NQ, int MINB>
__global__ void __launch_bounds__(kAttnThreads, MINB) paged_attention_kernel(AttnArgs a) {
    constexpr int TT = attn_tt<D, INT8>();
    constexpr int CH = kAttnWarps * TT;
    constexpr int QT = 8 * NQ;
    constexpr int ROW = INT8 ? D : 2 * D;             // bytes of a cache row
    constexpr int KL = ROW / 64;                      // 16-byte key loads per token and lane
    constexpr int KS = INT8 ? 4 : 2;                  // k steps of 16 per load
    constexpr int NT8 = TT / 8;                       // score tiles of 8 tokens
    constexpr int VB = D * (INT8 ? 1 : 2) / 8 < 16 ? 8 : 16;   // bytes per value load (8 for int8 rows of 64)
    constexpr int VL = ROW / (8 * VB);                // value loads per token and lane
    constexpr int VW = VB / 4;                        // words per value load
    constexpr int OT = D / 16;                        // output tiles of 16 d
    constexpr int DPL = INT8 ? VB : VB / 2;           // d's per value load and lane

    __shared__ __align__(16) float so[kAttnWarps][QT][D + 4];
    __shared__ float sm[kAttnWarps][QT], sl[kAttnWarps][QT];

    // attn_join_kernel may launch; it waits for this grid before it reads the parts
    asm volatile("griddepcontrol.launch_dependents;");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int64_t heads = (int64_t)a.Hkv * a.qtiles;
    const AttnPlace place = attn_place<CH, kAttnThreads>(a, a.grid, blockIdx.x, heads);
    int64_t u = place.total * blockIdx.x / a.grid;
    const int64_t u1 = place.total * (blockIdx.x + 1) / a.grid;
    int b = place.b;
    int64_t before = place.before;
    const int pmask = (1 << a.page_shift) - 1;
    bool bad = false;

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

        // ---- the query's fragments
        uint32_t qf[KL * KS][NQ][2];
        float qscale[NQ];
        const int q0 = h * a.G + qt * QT;             // first query head
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            qscale[n] = a.scale_log2;
            const bool has = 8 * n + g < nq;
            const uint16_t* qrow = a.q + (int64_t)b * a.ldq + (int64_t)(q0 + 8 * n + g) * D;
            if (INT8) {
                // 16 d's per load and lane: d = 64 j + 16 c + e
                float amax = 0.0f;
#pragma unroll
                for (int j = 0; j < KL; ++j) {
                    uint4 w[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
                    if (has) {
                        w[0] = __ldg(reinterpret_cast<const uint4*>(qrow + 64 * j + 16 * c));
                        w[1] = __ldg(reinterpret_cast<const uint4*>(qrow + 64 * j + 16 * c + 8));
                    }
                    const uint32_t x[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        qf[j * KS + i / 2][n][i & 1] = x[i];
                        amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(x[i] << 16)),
                                                 fabsf(__uint_as_float(x[i] & 0xffff0000u))));
                    }
                }
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                // 2^e with amax * 2^-e in [1, 2)
                const int ex = min(max((int)(__float_as_uint(amax) >> 23), 1), 253);
                const float down = __uint_as_float((uint32_t)(254 - ex) << 23), up = __uint_as_float((uint32_t)ex << 23);
                qscale[n] *= up;
#pragma unroll
                for (int i = 0; i < KL * KS; ++i)
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        const uint32_t x = qf[i][n][w];
                        const __half2 hv = __floats2half2_rn(__uint_as_float(x << 16) * down,
                                                             __uint_as_float(x & 0xffff0000u) * down);
                        qf[i][n][w] = *reinterpret_cast<const uint32_t*>(&hv);
                    }
            } else {
#pragma unroll
                for (int j = 0; j < KL; ++j) {
                    uint4 w = make_uint4(0, 0, 0, 0);
                    if (has) w = __ldg(reinterpret_cast<const uint4*>(qrow + 32 * j + 8 * c));
                    qf[2 * j][n][0] = w.x;
                    qf[2 * j][n][1] = w.y;
                    qf[2 * j + 1][n][0] = w.z;
                    qf[2 * j + 1][n][1] = w.w;
                }
            }
        }

        float o[NQ][OT][4];
        float m[NQ], l[NQ];
        int oe[NQ];               // int8: o is in units of 2^oe (of sum p v)
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            m[n] = -INFINITY;
            l[n] = 0.0f;
            oe[n] = -127;
#pragma unroll
            for (int i = 0; i < OT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[n][i][j] = 0.0f;
        }

        // ---- the warp's tiles: ch0 * 4 + warp, every fourth
        const int64_t tile_end = (ch0 + seg) * kAttnWarps;
        const int32_t* trow = a.table + (int64_t)b * a.ld_table;
        auto page_of = [&](int64_t tile) -> int {     // of the tile's token number `lane`
            const int64_t t = tile * TT + lane;
            if (tile >= tile_end || lane >= TT || t >= len) return -1;
            const int pg = __ldg(trow + (t >> a.page_shift));
            if (pg < 0 || pg >= a.num_pages) {
                bad = true;
                return -1;
            }
            return pg;
        };
        // row of token x of a tile whose tokens' pages the lanes hold; < 0: absent
        auto row_of = [&](int pages, int64_t tile, int x) -> int64_t {
            const int pg = __shfl_sync(0xffffffffu, pages, x);
            const int off = (int)((tile * TT + x) & pmask);
            return pg < 0 ? -1 : ((((int64_t)pg * a.Hkv + h) << a.page_shift) + off);
        };
        uint4 kr[NT8][KL];
        uint32_t vr[NT8][2][VL][VW];                  // tokens 8j + 2c, 8j + 2c + 1
        float2 ksc[NT8], vsc[NT8];
        auto load_k = [&](int pages, int64_t tile) {
#pragma unroll
            for (int j = 0; j < NT8; ++j) {
                const int64_t row = row_of(pages, tile, 8 * j + g);
                const uint8_t* p = reinterpret_cast<const uint8_t*>(a.kc) + row * ROW + 16 * c;
#pragma unroll
                for (int i = 0; i < KL; ++i) kr[j][i] = row >= 0 ? ld_stream_16(p + 64 * i) : make_uint4(0, 0, 0, 0);
            }
        };
        auto load_v = [&](int pages, int64_t tile) {
#pragma unroll
            for (int j = 0; j < NT8; ++j) {
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const int64_t row = row_of(pages, tile, 8 * j + 2 * c + s);
                    const uint8_t* p = reinterpret_cast<const uint8_t*>(a.vc) + row * ROW + VB * g;
#pragma unroll
                    for (int i = 0; i < VL; ++i) {
                        if (VB == 16) {
                            const uint4 v = row >= 0 ? ld_stream_16(p + 128 * i) : make_uint4(0, 0, 0, 0);
                            vr[j][s][i][0] = v.x;
                            vr[j][s][i][1] = v.y;
                            vr[j][s][i][2 % VW] = v.z;
                            vr[j][s][i][3 % VW] = v.w;
                        } else {
                            const uint2 v = row >= 0 ? __ldg(reinterpret_cast<const uint2*>(p)) : make_uint2(0, 0);
                            vr[j][s][i][0] = v.x;
                            vr[j][s][i][1] = v.y;
                        }
                    }
                    if (INT8) {
                        const float sk = row >= 0 ? __ldg(a.ks + row) : 0.0f, sv = row >= 0 ? __ldg(a.vs + row) : 0.0f;
                        if (s == 0) {
                            ksc[j].x = sk;
                            vsc[j].x = sv;
                        } else {
                            ksc[j].y = sk;
                            vsc[j].y = sv;
                        }
                    }
                }
            }
        };

        int64_t tile = ch0 * kAttnWarps + warp;
        int pages = page_of(tile), pages_next = page_of(tile + kAttnWarps);
        load_k(pages, tile);
        load_v(pages, tile);
        for (; tile < tile_end; tile += kAttnWarps) {
            const uint32_t valid = __ballot_sync(0xffffffffu, pages >= 0);
            // ---- scores
            float s[NT8][4];
#pragma unroll
            for (int j = 0; j < NT8; ++j) {
#pragma unroll
                for (int i = 0; i < 4; ++i) s[j][i] = 0.0f;
#pragma unroll
                for (int i = 0; i < KL; ++i) {
                    const uint32_t w[4] = {kr[j][i].x, kr[j][i].y, kr[j][i].z, kr[j][i].w};
#pragma unroll
                    for (int st = 0; st < KS; ++st) {
                        const uint32_t(&qa)[NQ][2] = qf[i * KS + st];
                        const uint32_t a1 = NQ == 2 ? qa[NQ - 1][0] : 0u, a3 = NQ == 2 ? qa[NQ - 1][1] : 0u;
                        if (INT8) {
                            const uint32_t u8 = w[st] ^ 0x80808080u;
                            mma_f16_16816(s[j], qa[0][0], a1, qa[0][1], a3, code_pair<0x4140>(u8), code_pair<0x4342>(u8));
                        } else {
                            mma_bf16_16816(s[j], qa[0][0], a1, qa[0][1], a3, w[(2 * st) % 4], w[(2 * st + 1) % 4]);
                        }
                    }
                }
            }
            const int64_t next = tile + kAttnWarps;
            load_k(pages_next, next);   // in flight during the softmax and the outputs
            const int pages_after = page_of(next + kAttnWarps);
            // ---- softmax of query rows g (and g + 8)
            uint32_t pf[NQ][NT8], pl[NQ][NT8];        // fp16 pairs; bf16: high and low parts
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
                        float v = s[j][2 * n + e] * qscale[n];
                        if (INT8) v *= e ? ksc[j].y : ksc[j].x;
                        x[j][e] = (valid >> (8 * j + 2 * c + e)) & 1u ? v : -INFINITY;
                        mx = fmaxf(mx, x[j][e]);
                    }
                }
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
                    // probabilities times the values' scales, brought to [0, 2) by a power of two
                    float um = 0.0f;
#pragma unroll
                    for (int j = 0; j < NT8; ++j) {
                        x[j][0] *= vsc[j].x;
                        x[j][1] *= vsc[j].y;
                        um = fmaxf(um, fmaxf(x[j][0], x[j][1]));
                    }
                    um = fmaxf(um, __shfl_xor_sync(0xffffffffu, um, 1));
                    um = fmaxf(um, __shfl_xor_sync(0xffffffffu, um, 2));
                    // largest so far in the new reference: the old unit's 2 * 2^oe * corr bounds the old ones
                    const float old = __uint_as_float((uint32_t)min(max(oe[n] + 127, 0), 254) << 23) * corr;
                    const int en = min(max((int)(__float_as_uint(fmaxf(um, old)) >> 23) - 127, -126), 126);
                    fac[n] = corr * __uint_as_float((uint32_t)min(max(oe[n] - en + 127, 0), 254) << 23);
                    oe[n] = en;
                    const float unit = __uint_as_float((uint32_t)(127 - en) << 23);
#pragma unroll
                    for (int j = 0; j < NT8; ++j) {
                        const __half2 hv = __floats2half2_rn(x[j][0] * unit, x[j][1] * unit);
                        pf[n][j] = *reinterpret_cast<const uint32_t*>(&hv);
                    }
                } else {
                    fac[n] = corr;
#pragma unroll
                    for (int j = 0; j < NT8; ++j) {
                        const uint32_t hi = pack_bf16x2(x[j][0], x[j][1]);
                        pf[n][j] = hi;
                        pl[n][j] = pack_bf16x2(x[j][0] - __uint_as_float(hi << 16),
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
#pragma unroll
                    for (int w = 0; w < VW; ++w) {
                        if (INT8) {
                            // 4 d's: two output tiles
                            const uint32_t t0 = vr[j][0][i][w] ^ 0x80808080u, t1 = vr[j][1][i][w] ^ 0x80808080u;
                            const uint32_t t2 = vr[j + 1][0][i][w] ^ 0x80808080u, t3 = vr[j + 1][1][i][w] ^ 0x80808080u;
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
                            }
                        } else {
                            const uint32_t a0 = __byte_perm(vr[j][0][i][w], vr[j][1][i][w], 0x5410);
                            const uint32_t a1 = __byte_perm(vr[j][0][i][w], vr[j][1][i][w], 0x7632);
                            const uint32_t a2 = __byte_perm(vr[j + 1][0][i][w], vr[j + 1][1][i][w], 0x5410);
                            const uint32_t a3 = __byte_perm(vr[j + 1][0][i][w], vr[j + 1][1][i][w], 0x7632);
#pragma unroll
                            for (int n = 0; n < NQ; ++n) {
                                mma_bf16_16816(o[n][i * VW + w], a0, a1, a2, a3, pf[n][j], pf[n][j + 1]);
                                mma_bf16_16816(o[n][i * VW + w], a0, a1, a2, a3, pl[n][j], pl[n][j + 1]);
                            }
                        }
                    }
                }
            }
            load_v(pages_next, next);   // in flight during the next scores
            pages = pages_next;
            pages_next = pages_after;
        }

        // ---- join of the four warps
        __syncthreads();   // the previous segment's reads are done
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            l[n] += __shfl_xor_sync(0xffffffffu, l[n], 1);
            l[n] += __shfl_xor_sync(0xffffffffu, l[n], 2);
            if (c == 0) {
                sm[warp][8 * n + g] = m[n];
                sl[warp][8 * n + g] = l[n];
            }
            float un = 1.0f;
            if (INT8) un = __uint_as_float((uint32_t)(min(max(oe[n], -126), 126) + 127) << 23);
            const float u0f = __shfl_sync(0xffffffffu, un, 8 * c), u1f = __shfl_sync(0xffffffffu, un, 8 * c + 4);
            // tile i covers d = 8 DPL (i / (DPL / 2)) + DPL g + 2 (i % (DPL / 2)), + 1
#pragma unroll
            for (int i = 0; i < OT; i += 2) {
                const int d = 8 * DPL * (i / (DPL / 2)) + DPL * g + 2 * (i % (DPL / 2));
                *reinterpret_cast<float4*>(&so[warp][8 * n + 2 * c][d]) =
                    make_float4(o[n][i][0] * u0f, o[n][i][2] * u0f, o[n][i + 1][0] * u0f, o[n][i + 1][2] * u0f);
                *reinterpret_cast<float4*>(&so[warp][8 * n + 2 * c + 1][d]) =
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
                const float4 v = *reinterpret_cast<const float4*>(&so[w][qh][d]);
                ll += sl[w][qh] * f;
                acc.x += v.x * f;
                acc.y += v.y * f;
                acc.z += v.z * f;
                acc.w += v.w * f;
            }
            if (whole) {
                const float r = ll == 0.0f ? 0.0f : 1.0f / ll;
                *reinterpret_cast<uint2*>(a.y + ((int64_t)b * a.Hq + q0 + qh) * D + d) =
                    make_uint2(pack_bf16x2(acc.x * r, acc.y * r), pack_bf16x2(acc.z * r, acc.w * r));
            } else {
                *reinterpret_cast<float4*>(a.part_o + (pbase + qh) * D + d) = acc;
                if (d == 0) a.part_ml[pbase + qh] = make_float2(mm, ll);
            }
        }
        u += seg;
    }
    if (bad) record_error(W8A8_ERR_INVALID_ARG, (kKernelIdAttn << 16) | 1);
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < a.B; i += kAttnThreads)
            if (__ldg(a.lengths + i) > a.cap) record_error(W8A8_ERR_INVALID_ARG, (kKernelIdAttn << 16) | 2);
}

// Joins the parts of the (sequence, head) units that several CTAs shared, in
// CTA order, and writes the zeros of empty sequences.  One CTA per unit.
template <int D, int CH, int NQ>
__global__ void __launch_bounds__(128) attn_join_kernel(AttnArgs a) {
    constexpr int QT = 8 * NQ;
    __shared__ int64_t red[2][4];
    const int64_t heads = (int64_t)a.Hkv * a.qtiles;
    const int b = (int)(blockIdx.x / heads), hq = (int)(blockIdx.x - b * heads);
    const int h = hq / a.qtiles, qt = hq - h * a.qtiles;
    const int nq = min(QT, a.G - qt * QT);
    const int q0 = h * a.G + qt * QT;
    // chunks before this sequence, and in all
    int64_t before = 0, total = 0;
    for (int i = threadIdx.x; i < a.B; i += 128) {
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
    before = red[0][0] + red[0][1] + red[0][2] + red[0][3];
    total = (red[1][0] + red[1][1] + red[1][2] + red[1][3]) * heads;
    const int64_t nb = (attn_len(a, b) + CH - 1) / CH;
    const int64_t us = before * heads + hq * nb, ue = us + nb;   // this unit's chunks
    // CTA whose share [total i / grid, total (i + 1) / grid) holds chunk x
    auto owner = [&](int64_t x) -> int {
        int i = (int)(x * a.grid / total);
        while (i > 0 && total * i / a.grid > x) --i;
        while (i + 1 < a.grid && total * (i + 1) / a.grid <= x) ++i;
        return i;
    };
    const int i0 = nb ? owner(us) : 0, i1 = nb ? owner(ue - 1) : 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (nb && i0 == i1) return;   // written by its CTA
    for (int i = threadIdx.x; i < nq * (D / 4); i += 128) {
        const int qh = i / (D / 4), d = 4 * (i - qh * (D / 4));
        float mm = -INFINITY, ll = 0.0f;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (nb) {
            // a share of no chunks (fewer chunks than CTAs) leaves no part
            for (int k = i0; k <= i1; ++k)
                if (total * k / a.grid < total * (k + 1) / a.grid)
                    mm = fmaxf(mm, __ldcg(&a.part_ml[((int64_t)k * 2 + (k == i0 ? 1 : 0)) * QT + qh]).x);
            const float mu = mm == -INFINITY ? 0.0f : mm;
            for (int k = i0; k <= i1; ++k) {
                if (total * k / a.grid == total * (k + 1) / a.grid) continue;
                const int64_t p = ((int64_t)k * 2 + (k == i0 ? 1 : 0)) * QT + qh;
                const float2 ml = __ldcg(&a.part_ml[p]);
                const float f = attn_ex2(ml.x - mu);
                const float4 v = __ldcg(reinterpret_cast<const float4*>(a.part_o + p * D + d));
                ll += ml.y * f;
                acc.x += v.x * f;
                acc.y += v.y * f;
                acc.z += v.z * f;
                acc.w += v.w * f;
            }
        }
        const float r = ll == 0.0f ? 0.0f : 1.0f / ll;
        *reinterpret_cast<uint2*>(a.y + ((int64_t)b * a.Hq + q0 + qh) * D + d) =
            make_uint2(pack_bf16x2(acc.x * r, acc.y * r), pack_bf16x2(acc.z * r, acc.w * r));
    }
}

}  // namespace w8a8

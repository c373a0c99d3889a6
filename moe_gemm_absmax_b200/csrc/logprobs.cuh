// Log probabilities of given tokens, entropy and top alternatives from the
// head's logits (w8a8_token_logprobs).
//
//   m = max_i x_i,  s = sum_i e^(x_i - m),  u = sum_i (x_i - m) e^(x_i - m)
//   log p_i = (x_i - m) - log s,   entropy = log s - u / s
//
// One pass over the row: each thread keeps (m, s, u) of its own elements, and
// where its maximum rises by d it scales s by e^-d and u to (u - d s) e^-d;
// the parts then join the same way, threads, warps and the CTAs of a cluster
// (through distributed shared memory: one launch, no workspace).
//
// The alternatives come out of the same pass without a list per thread.  Any
// k disjoint groups of elements have k maxima, so the k-th largest of the
// groups' maxima bounds the row's k-th largest from below.  Here a group is
// four threads' elements (128 groups, which puts the bound at about the
// k-th to 1.15 k-th largest for k <= 32), and only the threads whose own
// maximum reaches the bound (about k of 512) have their elements read again,
// from L2, a warp at a time.  What reaches the bound is ranked by counting.
// Keys order by value, then lower index.
#pragma once

#include <cooperative_groups.h>
#include <float.h>

#include "common.cuh"

namespace w8a8 {

constexpr int kLpThreads = 512;
constexpr int kLpGroups = 128;
constexpr int kLpMaxTop = 32;
constexpr int kLpHits = kLpMaxTop * (kLpThreads / kLpGroups);   // threads that can reach the bound
constexpr int kLpCand = kLpHits * kLpMaxTop;
constexpr int kLpUnroll = 4;
constexpr float kLog2e = 1.4426950408889634f;

// Order-preserving bits of x (NaN as -inf, -0 as +0); every value's are > 0.
__device__ __forceinline__ uint32_t lp_ord(float x) {
    if (!(x == x)) x = -INFINITY;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float lp_unord(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ uint64_t lp_key(float x, uint32_t at) { return ((uint64_t)lp_ord(x) << 32) | (uint32_t)~at; }

__device__ __forceinline__ float lp_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Running (m, s, u).  m starts at the lowest finite value, so that a row of
// nothing but -inf has s = 0 and nothing is ever subtracted from -inf; the
// distance to a new maximum is cut at -1e4, where e^d is 0, so that no
// 0 * inf arises.  NaN and +inf reach s through e^(x - m).
struct LpStat {
    float m, s, u;
};
__device__ __forceinline__ void lp_join(LpStat& a, const LpStat& b) {
    const float m = fmaxf(a.m, b.m);
    const float da = fmaxf(a.m - m, -1.0e4f), db = fmaxf(b.m - m, -1.0e4f);
    const float ca = lp_ex2(da * kLog2e), cb = lp_ex2(db * kLog2e);
    a.u = (a.u + da * a.s) * ca + (b.u + db * b.s) * cb;
    a.s = a.s * ca + b.s * cb;
    a.m = m;
}

// A row as 16-byte windows: window w holds elements [w * E - lead, + E), the
// first and last of which may reach past the row (those read as -inf).
template <typename T>
struct LpRow {
    static constexpr int E = 16 / (int)sizeof(T);
    const T* p;     // row start
    int V, lead;    // elements; elements between the 16-byte boundary below p and p
    int W;          // windows
    __device__ __forceinline__ LpRow(const T* row, int v) : p(row), V(v) {
        lead = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
        W = (int)(((int64_t)V + lead + E - 1) / E);
    }
    __device__ __forceinline__ static float to_float(uint16_t h) { return bf16_bits_to_float(h); }
    __device__ __forceinline__ static float to_float(float f) { return f; }
    __device__ __forceinline__ bool whole(int w) const { return w * E >= lead && (int64_t)w * E - lead + E <= V; }
    __device__ __forceinline__ uint4 raw(int w) const {
        if (whole(w)) return ld_stream_16(p + ((int64_t)w * E - lead));
        uint32_t q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (sizeof(T) == 4) {
                const int64_t k = (int64_t)w * E - lead + i;
                q[i] = k >= 0 && k < V ? __float_as_uint(to_float(p[k])) : 0xff800000u;
            } else {
                q[i] = 0u;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int64_t k = (int64_t)w * E - lead + 2 * i + h;
                    const uint32_t b = k >= 0 && k < V ? __float_as_uint(to_float(p[k])) >> 16 : 0xff80u;
                    q[i] |= b << (16 * h);
                }
            }
        }
        return make_uint4(q[0], q[1], q[2], q[3]);
    }
    __device__ __forceinline__ static void unpack(const uint4& v, float (&x)[E]) {
        const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (sizeof(T) == 4) {
                x[i] = __uint_as_float(q[i]);
            } else {
                x[2 * i] = __uint_as_float(q[i] << 16);
                x[(2 * i + 1) % E] = __uint_as_float(q[i] & 0xffff0000u);
            }
        }
    }
};

struct LpArgs {
    const void* logits;
    int64_t ld;
    const int32_t* tokens;
    float* logprob;
    float* entropy;
    int32_t* top_ids;
    float* top_logprobs;
    int V, G, topk;
};

struct LpShared {
    uint64_t key[kLpThreads];      // each thread's maximum; then this CTA's best k in order
    uint64_t cand[kLpCand];
    uint64_t bound;
    int hits[kLpHits];
    int nhits, ncand;
    LpStat warp[kLpThreads / 32];
    LpStat cta;
};

// Ranks cand[0 .. n) by counting and leaves the first k in order in out (0 past the last).
__device__ __forceinline__ void lp_rank(const uint64_t* cand, int n, uint64_t* out, int k) {
    for (int i = threadIdx.x; i < k; i += kLpThreads)
        if (i >= n) out[i] = 0;
    for (int i = threadIdx.x; i < n; i += kLpThreads) {
        const uint64_t mine = cand[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += cand[j] > mine ? 1 : 0;
        if (rank < k) out[rank] = mine;
    }
}

// One cluster per row; CTA r takes its share of the row's windows.
template <typename T>
__global__ void __launch_bounds__(kLpThreads, 2) token_logprobs_kernel(LpArgs a) {
    using Row = LpRow<T>;
    constexpr int E = Row::E;
    __shared__ LpShared sh;
    namespace cgx = cooperative_groups;
    cgx::cluster_group cl = cgx::this_cluster();
    const int C = (int)cl.num_blocks(), r = (int)cl.block_rank();
    const int64_t row_i = blockIdx.x / C;
    const Row row(reinterpret_cast<const T*>(a.logits) + row_i * a.ld, a.V);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int w0 = (int)((int64_t)row.W * r / C), w1 = (int)((int64_t)row.W * (r + 1) / C);

    // ---- the pass
    LpStat st = {-FLT_MAX, 0.0f, 0.0f};
    float vmax = -INFINITY;
    int wbest = -1;              // first window that holds vmax
    for (int wb = w0 + tid; wb < w1; wb += kLpUnroll * kLpThreads) {
        uint4 q[kLpUnroll];
#pragma unroll
        for (int i = 0; i < kLpUnroll; ++i)
            if (wb + i * kLpThreads < w1) q[i] = row.raw(wb + i * kLpThreads);
#pragma unroll
        for (int i = 0; i < kLpUnroll; ++i) {
            const int w = wb + i * kLpThreads;
            if (w >= w1) break;
            float x[E];
            Row::unpack(q[i], x);
            float top = x[0];
#pragma unroll
            for (int j = 1; j < E; ++j) top = fmaxf(top, x[j]);
            if (top > vmax || wbest < 0) {
                if (!(top == top)) top = -INFINITY;   // nothing but NaN
                wbest = w;
                vmax = top;
                const float m = fmaxf(top, st.m);
                const float d = fmaxf(st.m - m, -1.0e4f), c = lp_ex2(d * kLog2e);
                st.u = (st.u + d * st.s) * c;
                st.s *= c;
                st.m = m;
            }
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const float t = x[j] - st.m;
                const float e = lp_ex2(t * kLog2e);
                st.s += e;
                st.u = fmaf(fmaxf(t, -1.0e4f), e, st.u);   // t = -inf: 0
            }
        }
    }
    // the given tokens' logits, in flight with the joins
    float xt = 0.0f;
    bool tok_ok = false;
    if (r == 0 && tid < a.G) {
        const int tok = a.tokens[row_i * a.G + tid];
        tok_ok = tok >= 0 && tok < a.V;
        if (tok_ok) xt = Row::to_float(row.p[tok]);
    }

    // ---- join of (m, s, u) over the CTA
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        LpStat b;
        b.m = __shfl_xor_sync(0xffffffffu, st.m, o);
        b.s = __shfl_xor_sync(0xffffffffu, st.s, o);
        b.u = __shfl_xor_sync(0xffffffffu, st.u, o);
        lp_join(st, b);
    }
    if (lane == 0) sh.warp[warp] = st;
    const uint64_t mykey = wbest >= 0 ? lp_key(vmax, (uint32_t)wbest) : 0;
    sh.key[tid] = mykey;
    if (tid == 0) {
        sh.bound = 0;
        sh.nhits = 0;
        sh.ncand = 0;
    }
    __syncthreads();
    if (warp == kLpThreads / 32 - 1) {   // the last warp: the first ones rank the groups meanwhile
        LpStat b = {-FLT_MAX, 0.0f, 0.0f};
        if (lane < kLpThreads / 32) b = sh.warp[lane];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            LpStat c;
            c.m = __shfl_xor_sync(0xffffffffu, b.m, o);
            c.s = __shfl_xor_sync(0xffffffffu, b.s, o);
            c.u = __shfl_xor_sync(0xffffffffu, b.u, o);
            lp_join(b, c);
        }
        if (lane == 0) sh.cta = b;
    }
    const int k = a.topk;
    if (k > 0) {
        // ---- bound: the k-th largest group maximum (0, everything, where fewer groups hold elements)
        if (tid < kLpGroups) {
            uint64_t g = mykey;
#pragma unroll
            for (int i = 1; i < kLpThreads / kLpGroups; ++i) {
                const uint64_t o = sh.key[tid + i * kLpGroups];
                g = o > g ? o : g;
            }
            sh.cand[tid] = g;
        }
        __syncthreads();
        if (tid < kLpGroups) {
            const uint64_t g = sh.cand[tid];
            int rank = 0;
#pragma unroll 8
            for (int j = 0; j < kLpGroups; ++j) rank += sh.cand[j] > g ? 1 : 0;
            if (rank == k - 1) sh.bound = g;   // keys of groups with elements are distinct
        }
        __syncthreads();
        const uint64_t bound = sh.bound;
        if (mykey != 0 && mykey >= bound) sh.hits[atomicAdd(&sh.nhits, 1)] = tid;
        __syncthreads();
        // ---- elements of those threads that reach the bound
        const int nhits = sh.nhits;
        for (int h = warp; h < nhits; h += kLpThreads / 32) {
            const int owner = sh.hits[h];
            int n = 0;   // this lane's
            for (int w = w0 + owner + lane * kLpThreads; w < w1; w += 32 * kLpThreads) {
                float x[E];
                Row::unpack(row.raw(w), x);
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    const int at = w * E - row.lead + j;
                    if (at >= 0 && at < a.V && lp_key(x[j], (uint32_t)w) >= bound) ++n;
                }
            }
            int total = n;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
            if (total <= kLpMaxTop) {
                if (n > 0) {
                    for (int w = w0 + owner + lane * kLpThreads; w < w1; w += 32 * kLpThreads) {
                        float x[E];
                        Row::unpack(row.raw(w), x);
#pragma unroll
                        for (int j = 0; j < E; ++j) {
                            const int at = w * E - row.lead + j;
                            if (at >= 0 && at < a.V && lp_key(x[j], (uint32_t)w) >= bound)
                                sh.cand[atomicAdd(&sh.ncand, 1)] = lp_key(x[j], (uint32_t)at);
                        }
                    }
                }
            } else {
                // many large values in one thread's elements: its k best, one at a time
                uint64_t last = ~0ull;
                for (int i = 0; i < k; ++i) {
                    uint64_t best = 0;
                    for (int w = w0 + owner + lane * kLpThreads; w < w1; w += 32 * kLpThreads) {
                        float x[E];
                        Row::unpack(row.raw(w), x);
#pragma unroll
                        for (int j = 0; j < E; ++j) {
                            const int at = w * E - row.lead + j;
                            const uint64_t key = lp_key(x[j], (uint32_t)at);
                            if (at >= 0 && at < a.V && key < last && key > best) best = key;
                        }
                    }
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) {
                        const uint64_t b = __shfl_xor_sync(0xffffffffu, best, o);
                        best = b > best ? b : best;
                    }
                    if (best == 0) break;
                    if (lane == 0) sh.cand[atomicAdd(&sh.ncand, 1)] = best;
                    last = best;
                }
            }
        }
        __syncthreads();
        lp_rank(sh.cand, sh.ncand, sh.key, k);
    }
    // ---- join over the cluster
    if (C > 1) {
        cl.sync();
        if (r == 0 && k > 0)
            for (int i = tid; i < C * k; i += kLpThreads) sh.cand[i] = cl.map_shared_rank(&sh, i / k)->key[i % k];
    }
    __syncthreads();
    if (r == 0) {
        LpStat all = sh.cta;
        for (int i = 1; i < C; ++i) lp_join(all, cl.map_shared_rank(&sh, i)->cta);
        if (C > 1 && k > 0) {
            lp_rank(sh.cand, C * k, sh.key, k);
            __syncthreads();
        }
        const float logs = logf(all.s);   // s = 0: every logit is -inf
        auto logp = [&](float x) { return all.s == 0.0f ? -INFINITY : (x - all.m) - logs; };
        if (tid == 0 && a.entropy) a.entropy[row_i] = all.s == 0.0f ? 0.0f : logs - all.u / all.s;
        if (tid < a.G) a.logprob[row_i * a.G + tid] = tok_ok ? logp(xt) : __int_as_float(0x7fc00000);
        for (int i = tid + kLpThreads; i < a.G; i += kLpThreads) {
            const int tok = a.tokens[row_i * a.G + i];
            a.logprob[row_i * a.G + i] =
                tok >= 0 && tok < a.V ? logp(Row::to_float(row.p[tok])) : __int_as_float(0x7fc00000);
        }
        if (tid < k) {
            const uint64_t key = sh.key[tid];
            a.top_ids[row_i * k + tid] = (int32_t)~(uint32_t)key;
            a.top_logprobs[row_i * k + tid] = logp(lp_unord((uint32_t)(key >> 32)));
        }
    }
    if (C > 1) cl.sync();   // the leader has read this CTA's shared memory
}

}  // namespace w8a8

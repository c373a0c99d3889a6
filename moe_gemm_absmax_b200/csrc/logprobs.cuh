// Log probabilities of given tokens, entropy and top alternatives from the
// head's logits (w8a8_token_logprobs).
//
//   m = max_i x_i,  s = sum_i e^(x_i - m),  u = sum_i (x_i - m) e^(x_i - m)
//   log p_i = (x_i - m) - log s,   entropy = log s - u / s
//
// One pass over the row: each thread keeps (m, s, u) of its own elements, and
// where its maximum rises by d it scales s by e^-d and u to (u - d s) e^-d;
// the parts then join the same way, threads, warps and the CTAs of a cluster
// (through distributed shared memory: one launch, no workspace).  Large
// batches are bound by HBM; next come the exponentials (16 a cycle and SM:
// 0.7 of the time that bf16 rows take to read), so the rest is kept to five
// instructions an element: two elements per fp32 instruction, maxima and the
// lower clamp on packed bf16, one test for a new maximum per 64 bytes.
//
// The alternatives come out of the same pass without a list per thread.  Any
// k disjoint groups of elements have k maxima, so the k-th largest of the
// groups' maxima bounds the row's k-th largest from below.  Here a group is
// four threads' elements (64 groups, which puts the bound at the k-th largest
// for small k, at about the 24th for k = 20 and the 44th for k = 32: in random
// order 64 (ln 64 - ln(64 - k)) elements reach k of the groups).  Of the threads
// whose own maximum reaches the bound only the parts of their share (16 to a
// thread) whose maximum does are read again, from L2, dealt out over the CTA.
// What reaches the bound is ranked by counting.  Keys order by value, then lower
// index.
#pragma once

#include <cooperative_groups.h>
#include <float.h>

#include "common.cuh"

namespace w8a8 {

constexpr int kLpThreads = 256;
constexpr int kLpGroups = 64;
constexpr int kLpMaxTop = 32;
constexpr int kLpHits = kLpMaxTop * (kLpThreads / kLpGroups);   // threads that can reach the bound
constexpr int kLpCand = kLpHits * kLpMaxTop + 16;              // and what the row's ends hold
constexpr int kLpSlots = 16;                                    // parts of a thread's share whose maxima are kept
constexpr int kLpUnroll = 4;                                     // windows a thread takes at a time: a batch
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

// (m, s, u) of some elements, u in units of log2 e: u = sum t e, t = (x - m) log2 e,
// e = 2^t.  Where there is no logit above -inf, s = 0 and m is the lowest
// finite value, so that nothing is ever subtracted from -inf; the distance
// to a new maximum is cut at -1e4, where e^d is 0, so that no 0 * inf
// arises (an element's own distance: take, below).  NaN and +inf reach s
// through e.
struct LpStat {
    float m, s, u;
};
__device__ __forceinline__ void lp_join(LpStat& a, const LpStat& b) {
    const float m = fmaxf(a.m, b.m);
    const float da = fmaxf((a.m - m) * kLog2e, -1.0e4f), db = fmaxf((b.m - m) * kLog2e, -1.0e4f);
    const float ca = lp_ex2(da), cb = lp_ex2(db);
    a.u = (a.u + da * a.s) * ca + (b.u + db * b.s) * cb;
    a.s = a.s * ca + b.s * cb;
    a.m = m;
}
// The same over a warp.
__device__ __forceinline__ void lp_join_warp(LpStat& a) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        LpStat b;
        b.m = __shfl_xor_sync(0xffffffffu, a.m, o);
        b.s = __shfl_xor_sync(0xffffffffu, a.s, o);
        b.u = __shfl_xor_sync(0xffffffffu, a.u, o);
        lp_join(a, b);
    }
}

// Logits below this count as it in the fast pass (their e is 0 unless the
// whole of a thread's share lies there, which is then taken again exactly):
// a finite floor keeps -inf out of the products.  A bf16 value.
constexpr uint32_t kLpFloorBits = 0xf1490000u;   // -9.95e29
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {   // NaN loses
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {   // NaN stays
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
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
    __device__ __forceinline__ const T* at(int w) const { return p + ((int64_t)w * E - lead); }
    // Any window, element by element where it reaches past the row.
    __device__ __noinline__ uint4 edge(int w) const {
        uint32_t q[4];
        for (int i = 0; i < 4; ++i) {
            q[i] = 0u;
            for (int h = 0; h < 4 / (int)sizeof(T); ++h) {
                const int64_t k = (int64_t)w * E - lead + i * (4 / (int)sizeof(T)) + h;
                const uint32_t b = k >= 0 && k < V ? __float_as_uint(to_float(p[k])) : 0xff800000u;
                q[i] |= sizeof(T) == 4 ? b : (b >> 16) << (16 * h);
            }
        }
        return make_uint4(q[0], q[1], q[2], q[3]);
    }
    // For a second look: through L1.
    __device__ __forceinline__ uint4 again(int w) const {
        return whole(w) ? __ldca(reinterpret_cast<const uint4*>(at(w))) : edge(w);
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
    __align__(16) uint64_t group[kLpGroups];
    union {
        float tops[kLpSlots][kLpThreads];   // until the slots to read again are known
        uint64_t cand[kLpCand];             // then
    };
    uint64_t bound;
    int hits[kLpHits * kLpSlots];  // slot << 16 | thread
    int nhits, ncand;
    LpStat warp[kLpThreads / 32];
    LpStat cta;
};

// The fast pass on a batch of windows: lifts its elements to the floor, returns
// their maximum and leaves each window's in tops.
template <typename T>
struct LpFast;
template <>
struct LpFast<uint16_t> {
    __device__ __forceinline__ static float clamp_top(uint4 (&q)[kLpUnroll], uint32_t (&tops)[kLpUnroll]) {
        const uint32_t fl = (kLpFloorBits >> 16) | kLpFloorBits;
        uint32_t top = fl;
#pragma unroll
        for (int i = 0; i < kLpUnroll; ++i) {
            q[i].x = max_nan_bf16x2(q[i].x, fl);
            q[i].y = max_nan_bf16x2(q[i].y, fl);
            q[i].z = max_nan_bf16x2(q[i].z, fl);
            q[i].w = max_nan_bf16x2(q[i].w, fl);
            tops[i] = max_bf16x2(max_bf16x2(q[i].x, q[i].y), max_bf16x2(q[i].z, q[i].w));
            top = max_bf16x2(top, tops[i]);
        }
        return fmaxf(__uint_as_float(top << 16), __uint_as_float(top & 0xffff0000u));
    }
    __device__ __forceinline__ static bool holds(uint32_t tops, float top) {
        return __uint_as_float(tops << 16) == top || __uint_as_float(tops & 0xffff0000u) == top;
    }
};
template <>
struct LpFast<float> {
    __device__ __forceinline__ static float clamp_top(uint4 (&q)[kLpUnroll], uint32_t (&tops)[kLpUnroll]) {
        const float fl = __uint_as_float(kLpFloorBits);
        float top = fl;
#pragma unroll
        for (int i = 0; i < kLpUnroll; ++i) {
            const float x = fmax_nan(__uint_as_float(q[i].x), fl), y = fmax_nan(__uint_as_float(q[i].y), fl);
            const float z = fmax_nan(__uint_as_float(q[i].z), fl), w = fmax_nan(__uint_as_float(q[i].w), fl);
            q[i] = make_uint4(__float_as_uint(x), __float_as_uint(y), __float_as_uint(z), __float_as_uint(w));
            const float t = fmaxf(fmaxf(x, y), fmaxf(z, w));
            tops[i] = __float_as_uint(t);
            top = fmaxf(top, t);
        }
        return top;
    }
    __device__ __forceinline__ static bool holds(uint32_t tops, float top) { return __uint_as_float(tops) == top; }
};

// A thread's share exactly, one element after the other: only shares with no
// logit above the floor come here.
template <typename T>
__device__ __noinline__ void lp_slow_share(const LpRow<T>& row, int first, int hi, int edge, LpStat& st, float& vmax,
                                           int& best) {
    st = {-FLT_MAX, 0.0f, 0.0f};
    vmax = -INFINITY;
    best = -1;
    auto window = [&](int w) {
        float x[LpRow<T>::E];
        LpRow<T>::unpack(row.again(w), x);
        for (int j = 0; j < LpRow<T>::E; ++j) {
            if (x[j] > vmax || best < 0) {
                vmax = fmaxf(x[j], -INFINITY);   // NaN: -inf
                best = w;
            }
            LpStat one = {fmaxf(x[j], -FLT_MAX), 1.0f, 0.0f};
            if (!(fabsf(x[j]) < INFINITY)) one.s = x[j] == -INFINITY ? 0.0f : x[j] - x[j];   // NaN and +inf: NaN
            lp_join(st, one);
        }
    };
    // in the order of indexes: the first of equal values counts
    if (edge >= 0 && edge < first) window(edge);
    for (int w = first; w < hi; w += kLpThreads) window(w);
    if (edge >= first) window(edge);
}

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
__global__ void __launch_bounds__(kLpThreads, 4) token_logprobs_kernel(LpArgs a) {
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

    asm volatile("griddepcontrol.wait;" ::: "memory");   // may overlap the kernel before it
    // the given tokens' logits, in flight with the pass
    float xt = 0.0f;
    bool tok_ok = false;
    if (r == 0 && tid < a.G) {
        const int tok = a.tokens[row_i * a.G + tid];
        tok_ok = tok >= 0 && tok < a.V;
        if (tok_ok) xt = Row::to_float(row.p[tok]);
    }

    // ---- the pass: whole windows in batches, the row's first and last window by themselves
    float m = __uint_as_float(kLpFloorBits);
    uint64_t s2 = 0ull, u2 = 0ull;   // sums of the even and the odd elements
    int best = -1;                   // first window that holds m
    auto take = [&](uint4 (&q)[kLpUnroll], int wb) -> float {
        uint32_t tops[kLpUnroll];
        const float top = LpFast<T>::clamp_top(q, tops);
        if (top > m) {
            const float d = fmaxf((m - top) * kLog2e, -1.0e4f), c = lp_ex2(d);
            const uint64_t d2 = f2_pack(d, d), c2 = f2_pack(c, c);
            u2 = f2_mul(f2_fma(d2, s2, u2), c2);
            s2 = f2_mul(s2, c2);
            m = top;
#pragma unroll
            for (int i = kLpUnroll - 1; i >= 0; --i)
                if (LpFast<T>::holds(tops[i], top)) best = wb + i * kLpThreads;
        }
        // a distance below a maximum of more than FLT_MAX / log2 e could pass fp32's range
        // as t, and t e = -inf * 0 would be NaN: past 1e38 two values are equal or 1e31
        // apart, so e is 1 or 0 and t e is 0 whatever the factor
        const float lg = m > 1.0e38f ? 1.0f : kLog2e;
        const uint64_t nm = f2_pack(-m, -m), l2 = f2_pack(lg, lg);
#pragma unroll
        for (int i = 0; i < kLpUnroll; ++i) {
            float x[E];
            Row::unpack(q[i], x);
#pragma unroll
            for (int j = 0; j < E; j += 2) {
                const uint64_t t = f2_mul(f2_add(f2_pack(x[j], x[j + 1]), nm), l2);
                float t0, t1;
                f2_unpack(t, t0, t1);
                const uint64_t e = f2_pack(lp_ex2(t0), lp_ex2(t1));
                s2 = f2_add(s2, e);
                u2 = f2_fma(t, e, u2);
            }
        }
        return top;
    };
    // whole windows [lo, hi): thread t takes lo + t, lo + t + 256, ...; up to two others
    // at the row's ends, which threads 0 and 1 take element by element
    const int lo = w0 == 0 && w1 > 0 && !row.whole(0) ? 1 : w0;
    const int hi = w1 == row.W && w1 > lo && !row.whole(w1 - 1) ? w1 - 1 : w1;
    const int edge = tid == 0 ? (lo > w0 ? w0 : -1) : (tid == 1 && hi < w1 ? hi : -1);
    // batches of a thread, 1 << part of them to a slot
    constexpr int kStep = kLpUnroll * kLpThreads;
    const int batches = max(hi - lo + kStep - 1, 0) / kStep;
    int part = 0;
    while (((batches - 1) >> part) >= kLpSlots) ++part;
    const int first = lo + tid;
    const uint32_t none = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;       // -inf
    // in the order of indexes, as the first of equal values counts: the row's
    // first window before the whole ones, its last behind them
    auto take_edge = [&]() {
        uint4 q[kLpUnroll];
#pragma unroll
        for (int i = 0; i < kLpUnroll; ++i) q[i] = make_uint4(none, none, none, none);
        q[0] = row.edge(edge);
        take(q, edge);
    };
    if (edge >= 0 && edge < first) take_edge();
    {
        // the next batch's loads are in flight while one is taken
        const int mine = hi > first ? (hi - first + kLpThreads - 1) / kLpThreads : 0;   // windows
        const int full = mine / kLpUnroll;
        const T* at = row.at(first);
        auto load = [&](uint4 (&q)[kLpUnroll]) {
#pragma unroll
            for (int i = 0; i < kLpUnroll; ++i) q[i] = ld_stream_16_coherent(at + i * kLpThreads * E);
            at += kStep * E;
        };
        int batch = 0;
        float slot_top = 0.0f;
        auto note = [&](float top) {
            slot_top = (batch & ((1 << part) - 1)) ? fmaxf(slot_top, top) : top;
            sh.tops[batch >> part][tid] = slot_top;
            ++batch;
        };
        uint4 qa[kLpUnroll], qb[kLpUnroll];
        if (full > 0) load(qa);
        while (batch < full) {
            if (batch + 1 < full) load(qb);
            note(take(qa, first + batch * kStep));
            if (batch >= full) break;
            if (batch + 1 < full) load(qa);
            note(take(qb, first + batch * kStep));
        }
        const int left = mine - full * kLpUnroll;
        if (left > 0) {
#pragma unroll
            for (int i = 0; i < kLpUnroll; ++i) {
                qa[i] = make_uint4(none, none, none, none);
                if (i < left) qa[i] = ld_stream_16_coherent(at + i * kLpThreads * E);
            }
            note(take(qa, first + batch * kStep));
        }
    }
    if (edge >= first) take_edge();
    LpStat st = {m, 0.0f, 0.0f};
    {
        float a0, a1;
        f2_unpack(s2, a0, a1);
        st.s = a0 + a1;
        f2_unpack(u2, a0, a1);
        st.u = a0 + a1;
    }
    const bool slow = best < 0;
    if (slow) lp_slow_share(row, first, hi, edge, st, m, best);

    // ---- join of (m, s, u) over the CTA
    lp_join_warp(st);
    if (lane == 0) sh.warp[warp] = st;
    const uint64_t mykey = best >= 0 ? lp_key(m, (uint32_t)best) : 0;
    sh.key[tid] = mykey;
    if (tid == 0) {
        sh.bound = 0;
        sh.nhits = 0;
        sh.ncand = 0;
    }
    __syncthreads();
    if (warp == kLpThreads / 32 - 1) {
        LpStat b = {-FLT_MAX, 0.0f, 0.0f};
        if (lane < kLpThreads / 32) b = sh.warp[lane];
        lp_join_warp(b);
        if (lane == 0) sh.cta = b;
    }
    const int k = a.topk;
    if (k > 0) {
        // ---- bound: the k-th largest group maximum (0, everything, where fewer groups hold elements).
        // Four threads rank a group, each against a quarter of the groups.
        constexpr int kPer = kLpThreads / kLpGroups;
        static_assert(kPer == 4, "four threads a group");
        if (tid < kLpGroups) {
            uint64_t top = mykey;
#pragma unroll
            for (int i = 1; i < kPer; ++i) top = max(top, sh.key[tid + i * kLpGroups]);
            sh.group[tid] = top;
        }
        __syncthreads();
        {
            const uint64_t mine = sh.group[tid / kPer];
            const ulonglong2* part = reinterpret_cast<const ulonglong2*>(sh.group + (tid % kPer) * (kLpGroups / kPer));
            int rank = 0;
#pragma unroll
            for (int j = 0; j < kLpGroups / kPer / 2; ++j) {
                const ulonglong2 v = part[j];
                rank += (v.x > mine ? 1 : 0) + (v.y > mine ? 1 : 0);
            }
            rank += __shfl_xor_sync(0xffffffffu, rank, 1);
            rank += __shfl_xor_sync(0xffffffffu, rank, 2);
            if (rank == k - 1) sh.bound = mine;   // keys of groups with elements are distinct
        }
        __syncthreads();
        const uint64_t bound = sh.bound;
        const float low = lp_unord((uint32_t)(bound >> 32));      // NaN where everything counts
        if (mykey != 0 && mykey >= bound) {
            const int n = (batches + (1 << part) - 1) >> part;
            for (int i = 0; i < n; ++i)
                if (slow || !(sh.tops[i][tid] < low)) sh.hits[atomicAdd(&sh.nhits, 1)] = tid | i << 16;
        }
        __syncthreads();
        // ---- elements of those slots that reach the bound, by value and window:
        // the windows are dealt out over the whole CTA
        const int nhits = sh.nhits;
        const int log_nw = part + 2;                              // windows of a slot
        static_assert(kLpUnroll == 4, "two bits");
        auto window = [&](int hit, int j) {                       // its j-th; past the share: >= hi
            return lo + (hit & 0xffff) + (((hit >> 16) << log_nw) + j) * kLpThreads;
        };
        auto each = [&](const uint4& q, int w, auto f) {   // elements of window w that reach the bound: key
            float x[E];
            Row::unpack(q, x);
            bool any = false;
#pragma unroll
            for (int j = 0; j < E; ++j) any |= !(x[j] < low);   // NaN passes: it may rank among -inf
            if (!any) return;
#pragma unroll
            for (int j = 0; j < E; ++j) {
                if (x[j] < low) continue;
                const int at = w * E - row.lead + j;
                if (at >= 0 && at < a.V && lp_key(x[j], (uint32_t)w) >= bound) f(lp_key(x[j], (uint32_t)at));
            }
        };
        auto push = [&](uint64_t key) {
            const int at = atomicAdd(&sh.ncand, 1);
            if (at < kLpCand) sh.cand[at] = key;
        };
        for (int i = tid; i < nhits << log_nw; i += kLpThreads) {
            const int w = window(sh.hits[i >> log_nw], i & ((1 << log_nw) - 1));
            if (w < hi) each(row.again(w), w, push);
        }
        if (edge >= 0) each(row.edge(edge), edge, push);
        __syncthreads();
        if (sh.ncand > kLpCand) {
            // thousands of large values in a few threads' elements: each thread's k best, one at a time, a warp a thread
            __syncthreads();
            if (tid == 0) sh.ncand = 0;
            __syncthreads();
            for (int h = warp; h < kLpThreads; h += kLpThreads / 32) {
                if (lo + h >= hi) break;
                uint64_t last = ~0ull;
                for (int i = 0; i < k; ++i) {
                    uint64_t top = 0;
                    for (int w = lo + h + lane * kLpThreads; w < hi; w += 32 * kLpThreads)
                        each(row.again(w), w, [&](uint64_t key) {
                            if (key < last && key > top) top = key;
                        });
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                    if (top == 0) break;
                    if (lane == 0) push(top);
                    last = top;
                }
            }
            if (edge >= 0) each(row.edge(edge), edge, push);
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
        if (tid == 0 && a.entropy) a.entropy[row_i] = all.s == 0.0f ? 0.0f : logs - 0.6931471805599453f * (all.u / all.s);
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

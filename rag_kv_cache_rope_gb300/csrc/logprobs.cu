// Log probabilities of given tokens, entropy and top alternatives from logits (token_logprobs in
// blend.h): bound by reading the logits once.
//
// A row belongs to a cluster of 1..16 CTAs, each with a stretch of the vocabulary (few rows: many CTAs a
// row, so that every SM reads; many rows: one CTA each).  Threads stream 16-byte vectors and keep, against
// a reference R that is raised only when a term would pass 4, Z = sum 2^(x c - R) and
// S = sum 2^(x c - R) (x c - R), c = scale log2(e); then log p = ln 2 (x c - R - log2 Z) and the entropy is
// ln 2 (log2 Z - S / Z).  R is whatever rounded number it is: every term uses the same one, in one
// multiply-add, so its rounding cancels.
//
// Ranking without sorting and without a second pass: a thread also keeps the largest logit it saw.  The
// k-th largest of the maxima of 64 groups of threads is a lower bound T of the k-th largest logit, which
// at most a few dozen logits of the stretch reach, and those lie with the few threads whose maximum reaches T: only
// these threads' vectors are read again (from L2).  The candidates, 64-bit keys of value and index, are
// ranked by counting.  Ties at T in numbers (a masked row), masks by value and NaN at the end of the ranking are taken
// in order of their index.  Each CTA of a cluster ranks its own stretch; the first joins sums and lists through
// distributed shared memory in the CTAs' order, so nothing depends on timing and no workspace is needed.
//
// 2047 x 32000 fp32, one alternative: 54 us, 4.9 TB/s; 2047 x 32003 bf16 35 us, 3.7 TB/s (without ranking 30 us): with
// two bytes a logit, issue slots (62 %), the two exponentials of a pair and the barriers at a row's ends bound it.  512 x
// 128256 bf16, 20 alternatives: 39 us.  Few rows are a chain of latencies: 1 x 152064 with 20 alternatives 8.2 us (without
// 4.2), of which a cluster of 16 saves 10; 64 x 128256 fp32 13.4 us for 30.5 without clusters.
#include <cooperative_groups.h>

#include "tokens.cuh"

namespace cg = cooperative_groups;

namespace blend {
namespace {

// Threads of a CTA, NT: 256, or 128 for many short rows. CTAs per SM: a row's start and end wait for memory and for
// one another. LP_U: vectors of a thread on their way together.
template <int NT> constexpr int LP_CTAS = NT == 256 ? 5 : 8;
template <int NT> constexpr int LP_U = NT == 256 ? 4 : 6;
constexpr int LP_SHORT = 32, LP_FEW = 8;  // vectors of a thread and alternatives of a row, at most, with 128 threads
constexpr int LP_GROUPS = 64;   // groups of threads whose maxima bound the k-th logit: twice the largest k
constexpr int LP_CAND = 1024;   // candidates of one stretch
constexpr int LP_MAX_CLUSTER = 16;
constexpr float LP_RAISE = 2.f;
// References beyond this are not used: x c - R, a rounding of R by then, could be anything. A thread that saw nothing
// above -LP_HUGE counts nothing; what it left out is 2^-LP_CLEAR of the row's sum at most where R is LP_CLEAR above.
constexpr float LP_HUGE = 16777216.f, LP_CLEAR = 256.f;
constexpr float LN2 = 0.693147180559945309f;
constexpr float FAR = -200.f;    // 2^FAR is 0 in fp32, and 0 times FAR is a number
// Logits count as this at least in the sums: with a scale of up to 2^20 they are numbers then, and 2^t of them 0 with one
// of 2^-64 or more (LP_LOW c is -8e10 at most, R above -2^24).
constexpr float LP_LOW = -1e30f;

using key_t = unsigned long long;

// Ranking key: value (order-preserving bits, -0 as +0, NaN 0), then lower index first.
__device__ __forceinline__ uint32_t value_bits(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return x != x ? 0u : (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ key_t rank_key(float x, int idx) { return ((key_t)value_bits(x) << 32) | (uint32_t)~idx; }
__device__ __forceinline__ float key_value(key_t k) {
    const uint32_t o = (uint32_t)(k >> 32);
    if (o == 0) return __int_as_float(0x7fc00000);
    return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ int key_index(key_t k) { return (int)~(uint32_t)k; }

__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A row as aligned 16-byte vectors: vector j holds elements j VE - off .. + VE - 1 (off of the first are
// before the row).  Vectors that reach over an end of the row are read element by element; what is not in
// the row comes back as -infinity.
template <typename T> struct Row {
    static constexpr int VE = 16 / sizeof(T);
    const T* p;  // the row's first element
    int off, vocab, n_vec;
    __device__ Row(const T* row, int v) {
        p = row;
        vocab = v;
        off = (int)(((uintptr_t)row & 15) / sizeof(T));
        n_vec = (int)(((long long)off + v + VE - 1) / VE);
    }
    __device__ __forceinline__ void load(int j, float (&x)[VE]) const {
        const int e0 = j * VE - off;
        if (e0 >= 0 && e0 + VE <= vocab) {
            const Vec<T> v = ld16(p + e0);
#pragma unroll
            for (int i = 0; i < VE; ++i) x[i] = v.get(i);
        } else {
#pragma unroll
            for (int i = 0; i < VE; ++i) x[i] = e0 + i >= 0 && e0 + i < vocab ? to_f<T>(p[e0 + i]) : -INFINITY;
        }
    }
    // The same as it lies in memory.
    __device__ __forceinline__ uint4 raw(int j) const {
        Vec<T> v;
        float x[VE];
        load(j, x);
#pragma unroll
        for (int i = 0; i < VE; ++i) v.set(i, x[i]);
        return v.raw;
    }
    // A vector that is neither the first nor the last.
    __device__ __forceinline__ uint4 inner(int j) const { return reinterpret_cast<const uint4*>(p - off)[j]; }
    __device__ __forceinline__ bool holds(int j, int i) const {  // element i of vector j is in the row
        const int e = j * VE - off + i;
        return e >= 0 && e < vocab;
    }
    __device__ __forceinline__ int index(int j, int i) const { return j * VE - off + i; }
};

struct Sums {
    float r, z, s;  // reference, sum of 2^(t), sum of 2^(t) t with t = x c - r
};
__device__ __forceinline__ float max_keep_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// A vector's logits, LP_LOW at least, in pairs, and the largest of them (NaN stays NaN and is not the largest).
__device__ __forceinline__ float pairs_of(const uint4& raw, float2 (&x)[4], bf16) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    const __nv_bfloat162 low = __float2bfloat162_rn(LP_LOW);
    __nv_bfloat162 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i] = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), low);
        const uint32_t u = *reinterpret_cast<const uint32_t*>(&h[i]);
        x[i] = make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
}
__device__ __forceinline__ float pairs_of(const uint4& raw, float2 (&x)[2], float) {
    x[0] = make_float2(max_keep_nan(__uint_as_float(raw.x), LP_LOW), max_keep_nan(__uint_as_float(raw.y), LP_LOW));
    x[1] = make_float2(max_keep_nan(__uint_as_float(raw.z), LP_LOW), max_keep_nan(__uint_as_float(raw.w), LP_LOW));
    return fmaxf(fmaxf(x[0].x, x[0].y), fmaxf(x[1].x, x[1].y));
}
template <int NT> struct Shared {
    key_t cand[LP_CAND];
    key_t list[BLEND_MAX_TOP];       // this stretch's ranking
    key_t all[LP_MAX_CLUSTER][BLEND_MAX_TOP];
    key_t merged[BLEND_MAX_TOP];
    Sums sums[NT / 32];
    Sums total;
    float group_max[LP_GROUPS];
    int active[NT];
    int n_active, n_cand, overflow, warp_tot[NT / 32];
    float bound;
};

// Appends elements of the stretch's vectors [v0, v1) that `take` accepts to sh.cand, in ascending index, from
// sh.n_cand on until it holds `until`.  All threads; barriers inside.
template <int NT, typename T, typename Take>
__device__ void take_in_order(const Row<T>& row, int v0, int v1, int until, Shared<NT>& sh, Take take) {
    constexpr int VE = Row<T>::VE;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int j0 = v0; j0 < v1; j0 += NT) {
        const int have = sh.n_cand;
        if (have >= until) break;
        const int j = j0 + tid;
        float x[VE];
        unsigned m = 0;
        if (j < v1) {
            row.load(j, x);
#pragma unroll
            for (int i = 0; i < VE; ++i)
                if (row.holds(j, i) && take(x[i])) m |= 1u << i;
        }
        int incl = __popc(m);
        const int mine = incl;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) sh.warp_tot[warp] = incl;
        __syncthreads();
        int at = have + incl - mine, total = have;
        for (int w = 0; w < (NT / 32); ++w) {
            if (w < warp) at += sh.warp_tot[w];
            total += sh.warp_tot[w];
        }
#pragma unroll
        for (int i = 0; i < VE; ++i)
            if ((m >> i & 1) && at < until) sh.cand[at++] = rank_key(x[i], row.index(j, i));
        __syncthreads();
        if (tid == 0) sh.n_cand = min(total, until);
        __syncthreads();
    }
}

// The stretch's `top` highest keys, descending, into sh.list (0 behind the last).  All threads.
template <int NT, typename T>
__device__ void rank_stretch(const Row<T>& row, int v0, int v1, int top, float my_max, Shared<NT>& sh) {
    constexpr int VE = Row<T>::VE;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int PER_GROUP = NT / LP_GROUPS;
    float g = my_max;
#pragma unroll
    for (int o = 1; o < PER_GROUP; o <<= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
    if (tid % PER_GROUP == 0) sh.group_max[tid / PER_GROUP] = g;
    if (tid < BLEND_MAX_TOP) sh.list[tid] = 0;
    if (tid == 0) sh.n_active = sh.n_cand = sh.overflow = 0;
    __syncthreads();
    {
        // (PER_GROUP threads compare a group's maximum with a part of the others)
        const int mine = tid / PER_GROUP, part = tid % PER_GROUP;
        const float m = sh.group_max[mine];
        int above = 0;
#pragma unroll
        for (int i = part; i < LP_GROUPS; i += PER_GROUP) {
            const float y = sh.group_max[i];
            above += y > m || (y == m && i < mine);
        }
#pragma unroll
        for (int o = 1; o < PER_GROUP; o <<= 1) above += __shfl_xor_sync(0xffffffffu, above, o);
        if (part == 0 && above == top - 1) sh.bound = m;
    }
    __syncthreads();
    const float bound = sh.bound > LP_LOW ? sh.bound : -INFINITY;
    // threads that hold a candidate
    if (my_max >= bound) sh.active[atomicAdd(&sh.n_active, 1)] = tid;
    __syncthreads();
    // Where most threads reach the bound, it is one value of many logits (a mask: fewer than `top` groups hold an allowed
    // token). Then only what is above it, or above the masks, is collected, and the rest in order of its index: 2047 x 32003
    // bf16, three tokens allowed, 5 alternatives 37 us under masks of -1e9 and 76 under -infinity; 189 with all of the masked
    // as candidates.
    const bool masked = sh.n_active > NT / 2;
    float least = bound;
    if (masked) {
        least = nextafterf(fmaxf(bound, LP_LOW), INFINITY);
        __syncthreads();
        if (tid == 0) sh.n_active = 0;
        __syncthreads();
        if (my_max >= least) sh.active[atomicAdd(&sh.n_active, 1)] = tid;
        __syncthreads();
    }
    const int n_active = sh.n_active;
    const int w0 = max(v0, 1), w1 = min(v1, row.n_vec - 1);
    const int each = (max(w1 - w0, 0) + NT - 1) / NT;  // inner vectors of a thread
    // (the row's first and last vectors besides)
    for (int i = tid; i < n_active * each + 2; i += NT) {
        const int k = i - 2;
        int j = i == 0 ? 0 : row.n_vec - 1;
        bool mine = i == 0 ? v0 == 0 : v1 == row.n_vec && row.n_vec > 1;
        if (k >= 0) {
            j = w0 + sh.active[k / each] + k % each * NT;
            mine = j < w1;
        }
        if (mine) {
            float x[VE];
            row.load(j, x);
#pragma unroll
            for (int e = 0; e < VE; ++e)
                if (x[e] >= least && row.holds(j, e)) {
                    const int at = atomicAdd(&sh.n_cand, 1);
                    if (at < LP_CAND) sh.cand[at] = rank_key(x[e], row.index(j, e));
                    else sh.overflow = 1;
                }
        }
    }
    __syncthreads();
    if (sh.overflow) {
        // Many equal logits at the bound (or few threads holding nearly all of the largest): those above it,
        // and of the equal ones the first `top`.
        __syncthreads();
        if (tid == 0) sh.n_cand = 0;
        __syncthreads();
        take_in_order(row, v0, v1, LP_CAND - BLEND_MAX_TOP, sh, [&](float x) { return x > bound; });
        if (sh.n_cand >= LP_CAND - BLEND_MAX_TOP) {
            // Still too many: the ranking one by one, each the highest key below the last.
            key_t last = ~0ull;
            for (int r = 0; r < top; ++r) {
                key_t best = 0;
                for (int j = v0 + tid; j < v1; j += NT) {
                    float x[VE];
                    row.load(j, x);
#pragma unroll
                    for (int i = 0; i < VE; ++i) {
                        const key_t k = rank_key(x[i], row.index(j, i));
                        if (row.holds(j, i) && k < last && k > best) best = k;
                    }
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const key_t y = __shfl_xor_sync(0xffffffffu, best, o);
                    best = y > best ? y : best;
                }
                __syncthreads();
                if (lane == 0) sh.cand[warp] = best;
                __syncthreads();
                for (int w = 0; w < (NT / 32); ++w) best = sh.cand[w] > best ? sh.cand[w] : best;
                if (tid == 0) sh.list[r] = best;
                last = best;
            }
            __syncthreads();
            return;
        }
        const int until = sh.n_cand + BLEND_MAX_TOP;
        __syncthreads();
        take_in_order(row, v0, v1, until, sh, [&](float x) { return x == bound; });
    }
    if (masked && !sh.overflow && sh.n_cand < top) {
        __syncthreads();
        if (bound > LP_LOW) take_in_order(row, v0, v1, top, sh, [&](float x) { return x == bound; });
        // masks: one value after the other, one or two as a rule
        uint32_t level = value_bits(LP_LOW) + 1u;
        while (bound <= LP_LOW && sh.n_cand < top) {
            uint32_t next = 0;
            for (int j = v0 + tid; j < v1; j += NT) {
                float x[VE];
                row.load(j, x);
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    const uint32_t o = value_bits(x[i]);
                    if (row.holds(j, i) && o < level && o > next) next = o;
                }
            }
            next = __reduce_max_sync(0xffffffffu, next);
            if (lane == 0) sh.warp_tot[warp] = (int)next;
            __syncthreads();
            for (int w = 0; w < NT / 32; ++w) next = max(next, (uint32_t)sh.warp_tot[w]);
            __syncthreads();
            if (next == 0) break;
            level = next;
            take_in_order(row, v0, v1, top, sh, [&](float x) { return value_bits(x) == level; });
        }
    }
    // fewer numbers than asked for: NaN in order
    if (sh.n_cand < top) {
        __syncthreads();
        take_in_order(row, v0, v1, top, sh, [](float x) { return x != x; });
    }
    const int n = sh.n_cand;
    for (int c = tid; c < n; c += NT) {
        const key_t k = sh.cand[c];
        int above = 0;
        for (int i = 0; i < n; ++i) above += sh.cand[i] > k;
        if (above < top) sh.list[above] = k;
    }
    __syncthreads();
}

// The sums of `lanes` neighbouring lanes (a power of two) under their largest reference, for all of them.
__device__ __forceinline__ Sums lanes_join(Sums t, int lanes) {
    float r = t.r;
    for (int o = 1; o < lanes; o <<= 1) r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, o));
    if (r > -INFINITY) {
        const float d = t.r - r, f = ex2f(d);
        t.s = f * (t.s + t.z * fmaxf(d, FAR));
        t.z *= f;
    }
    for (int o = 1; o < lanes; o <<= 1) {
        t.z += __shfl_xor_sync(0xffffffffu, t.z, o);
        t.s += __shfl_xor_sync(0xffffffffu, t.s, o);
    }
    t.r = r;
    return t;
}
// The threads' sums joined, the same way every time, for every thread.  Two barriers.
template <int NT> __device__ __forceinline__ Sums block_join(Sums t, Shared<NT>& sh) {
    t = lanes_join(t, 32);
    __syncthreads();
    if (threadIdx.x % 32 == 0) sh.sums[threadIdx.x / 32] = t;
    __syncthreads();
    return lanes_join(sh.sums[threadIdx.x % (NT / 32)], (NT / 32));
}
template <int NT> __device__ __forceinline__ float block_max(float m, Shared<NT>& sh) {
    return block_join({m, 0.f, 0.f}, sh).r;
}

template <int NT, typename T, bool TOP>
__global__ void __launch_bounds__(NT, LP_CTAS<NT>) k_logprobs(const Logprobs a, int cluster, float c) {
    constexpr int VE = Row<T>::VE, U = LP_U<NT>;
    __shared__ Shared<NT> sh;
    const int tid = threadIdx.x;
    const int rank = cluster > 1 ? (int)cg::this_cluster().block_rank() : 0;
    const long long r = blockIdx.x / cluster;
    const T* logits = (const T*)a.logits + r * a.ld;
    const Row<T> row(logits, a.vocab);
    const int v0 = (int)((long long)row.n_vec * rank / cluster), v1 = (int)((long long)row.n_vec * (rank + 1) / cluster);

    // (asked for now, used at the end)
    int my_id = -1;
    float my_x = 0.f;
    if (rank == 0 && tid < a.n_ids) {
        my_id = __ldg(a.ids + r * a.n_ids + tid);
        if (my_id >= 0 && my_id < a.vocab) my_x = to_f<T>(logits[my_id]);
    }
    float ref = -INFINITY, top_x = -INFINITY;
    float2 z2 = make_float2(0.f, 0.f), s2 = z2;
    const float2 c2 = make_float2(c, c);
    auto step = [&](const uint4& raw) {
        float2 x[VE / 2];
        const float m = pairs_of(raw, x, T());
        if (TOP) top_x = fmaxf(top_x, m);
        const float t_max = m * c;
        if (t_max > fmaxf(ref + LP_RAISE, -LP_HUGE)) {
            if (ref > -INFINITY) {
                const float d = ref - t_max, f = ex2f(d), df = fmaxf(d, FAR);
                s2 = make_float2(f * (s2.x + z2.x * df), f * (s2.y + z2.y * df));
                z2 = make_float2(f * z2.x, f * z2.y);
            }
            ref = t_max;
        }
        const float neg = ref == -INFINITY ? 0.f : -ref;
        const float2 neg2 = make_float2(neg, neg);
#pragma unroll
        for (int i = 0; i < VE / 2; ++i) {
            const float2 t = __ffma2_rn(x[i], c2, neg2), e = make_float2(ex2f(t.x), ex2f(t.y));
            z2 = __fadd2_rn(z2, e);
            s2 = __ffma2_rn(e, t, s2);
        }
    };
    // the row's first and last vectors may reach over its ends: thread 0's
    const int w0 = max(v0, 1), w1 = min(v1, row.n_vec - 1);
    if (tid == 0 && v0 == 0 && v1 > 0) step(row.raw(0));
    if (tid == 0 && v1 == row.n_vec && v0 < v1 && row.n_vec > 1) step(row.raw(row.n_vec - 1));
    int j = w0 + tid;
    for (; j + (U - 1) * NT < w1; j += U * NT) {
        uint4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = row.inner(j + u * NT);
#pragma unroll
        for (int u = 0; u < U; ++u) step(x[u]);
    }
    {
        uint4 x[U - 1];
#pragma unroll
        for (int u = 0; u < U - 1; ++u)
            if (j + u * NT < w1) x[u] = row.inner(j + u * NT);
#pragma unroll
        for (int u = 0; u < U - 1; ++u)
            if (j + u * NT < w1) step(x[u]);
    }
    float z = z2.x + z2.y, s = s2.x + s2.y;
    Sums t = block_join({ref, z, s}, sh);
    if (TOP) rank_stretch(row, v0, v1, a.top, top_x, sh);
    if (tid == 0) sh.total = t;
    const key_t* list = sh.list;
    if (cluster > 1) {
        cg::cluster_group cl = cg::this_cluster();
        cl.sync();
        // sums and lists of all to the first
        const int keys = cluster * a.top;
        if (rank == 0) {
            if (tid < 32) {
                t = tid < cluster ? cl.map_shared_rank(&sh, tid)->total : Sums{-INFINITY, 0.f, 0.f};
                t = lanes_join(t, 32);
                if (tid == 0) sh.total = t;
            }
            if (TOP)
                for (int i = tid; i < keys; i += NT)
                    sh.all[i / a.top][i % a.top] = cl.map_shared_rank(&sh, i / a.top)->list[i % a.top];
        }
        cl.sync();
        if (rank != 0) return;
        if (TOP) {
            // The m-th largest of the lists' p-th keys, m p >= top: that many keys at least reach it, and few more.
            const int p = (a.top + cluster - 1) / cluster, m = (a.top + p - 1) / p;
            if (tid == 0) sh.n_cand = 0;
            if (tid < cluster) {
                const key_t k = sh.all[tid][p - 1];
                int above = 0;
                for (int q = 0; q < cluster; ++q) above += sh.all[q][p - 1] > k || (sh.all[q][p - 1] == k && q < tid);
                if (above == m - 1) sh.merged[0] = k;
            }
            __syncthreads();
            const key_t least = sh.merged[0];
            for (int i = tid; i < keys; i += NT) {
                const key_t k = sh.all[i / a.top][i % a.top];
                if (k >= least && k != 0) sh.cand[atomicAdd(&sh.n_cand, 1)] = k;
            }
            __syncthreads();
            const int n = sh.n_cand;
            for (int c = tid; c < n; c += NT) {
                const key_t k = sh.cand[c];
                int above = 0;
                for (int i = 0; i < n; ++i) above += sh.cand[i] > k;
                if (above < a.top) sh.merged[above] = k;
            }
            __syncthreads();
        }
        list = sh.merged;
    } else
        __syncthreads();
    t = sh.total;
    // Nothing counted (R is -infinity): nothing is allowed, or every logit is far below 0 (masks of the type's
    // lowest value in a row that allows nothing else).  Such a row, one whose largest logit is so near -LP_HUGE that
    // some threads may have counted and others not, and one of huge logits, once more, against its maximum.
    float low = 0.f;
    bool none = false;
    if (!(t.r >= -LP_HUGE + LP_CLEAR && t.r <= LP_HUGE)) {
        float m = -INFINITY;
        for (int j = tid; j < row.n_vec; j += NT) {
            float x[VE];
            row.load(j, x);
#pragma unroll
            for (int i = 0; i < VE; ++i) m = fmaxf(m, x[i]);
        }
        low = block_max(m, sh);
        if (low == -INFINITY)
            none = t.z == 0.f;  // (else there is a NaN)
        else {
            z = s = 0.f;
            for (int j = tid; j < row.n_vec; j += NT) {
                float x[VE];
                row.load(j, x);
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    const float d = (x[i] - low) * c, e = ex2f(d);
                    z += e;
                    s = fmaf(e, fmaxf(d, FAR), s);
                }
            }
            t = block_join({0.f, z, s}, sh);
        }
    }
    const float lz = log2f(t.z);
    // log p = ln 2 (x c - R - log2 Z); where that difference is too low for fp32, the rest does not count (in halves:
    // two numbers may be further apart than the largest number, and their scaled distance be one). Roundings do not make
    // a probability larger than 1, nor an entropy smaller than 0.
    auto logp_of = [&](float x) {
        if (none) return x != x ? x : -INFINITY;
        const float d = fmaf(x - low, c, -t.r);
        const float lp = d == -INFINITY && x > d && lz == lz ? (0.5f * x - 0.5f * low) * a.scale * 2.f : LN2 * (d - lz);
        return lp > 0.f ? 0.f : lp;  // (NaN stays)
    };
    if (tid == 0 && a.entropy) {
        const float e = none ? 0.f : LN2 * (lz - t.s / t.z);
        a.entropy[r] = e < 0.f ? 0.f : e;
    }
    for (int i = tid; i < a.n_ids; i += NT) {
        const int id = i == tid ? my_id : __ldg(a.ids + r * a.n_ids + i);
        float lp = 0.f;
        if (id >= a.vocab) {
            set_error(a.err, BLEND_EDEVICE);
            lp = __int_as_float(0x7fc00000);
        } else if (id >= 0)
            lp = logp_of(i == tid ? my_x : to_f<T>(logits[id]));
        a.logp[r * a.n_ids + i] = lp;
    }
    if (TOP && tid < a.top) {
        const key_t k = list[tid];
        a.top_id[r * a.top + tid] = key_index(k);
        if (a.top_logp) a.top_logp[r * a.top + tid] = logp_of(key_value(k));
    }
}

template <int NT, typename T, bool TOP> int launch(const Logprobs& a, cudaStream_t s) {
    // A row's CTAs: as many as keep 152 SMs busy, each with 2048 logits at least.
    int cluster = 1;
    while (cluster < LP_MAX_CLUSTER && (long long)a.rows * cluster * 2 <= 152 * LP_CTAS<256> && a.vocab / (cluster * 2) >= 2048) cluster *= 2;
    auto* kern = k_logprobs<NT, T, TOP>;
    if (cluster > 8 && cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return BLEND_ECUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.rows * (long long)cluster));
    cfg.blockDim = dim3(NT);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    const float c = (float)((double)a.scale * 1.4426950408889634);
    if (cudaLaunchKernelEx(&cfg, kern, a, cluster, c) != cudaSuccess) return BLEND_ECUDA;
    note_launch();
    return BLEND_OK;
}

// Half the threads a row, and more rows at once, where rows are many, short and ranked for few: a CTA of 256 then
// waits for itself (barriers, the last vectors) more than for memory. bf16 logits, 256 against 128 threads: 4096 x 4000,
// top 5 35.0 and 26.1 us; 2047 x 32003, top 1 38.2 and 35.1, top 20 42.7 and 45.4 (a thread's vectors that are looked at
// again are twice as many); 2047 x 65000, top 5 59.6 and 62.6; 1250 x 32000, top 5 25.9 and 30.2 (less than two rounds of 256).
template <typename T, bool TOP> int launch_threads(const Logprobs& a, cudaStream_t s) {
    const bool many = a.rows >= 2 * 152 * LP_CTAS<256>, is_short = a.vocab <= LP_SHORT * 128 * Row<T>::VE;
    return many && is_short && a.top <= LP_FEW ? launch<128, T, TOP>(a, s) : launch<256, T, TOP>(a, s);
}

}  // namespace

int launch_logprobs(int dtype, const Logprobs& a, cudaStream_t s) {
    if (dtype == BLEND_BF16) return a.top ? launch_threads<bf16, true>(a, s) : launch_threads<bf16, false>(a, s);
    return a.top ? launch_threads<float, true>(a, s) : launch_threads<float, false>(a, s);
}

}  // namespace blend

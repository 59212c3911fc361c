// Attention of single tokens and few rows over a paged cache (paged_attention in blend.h), bf16
// models: bound by reading the pages, so every SM has to stream all the time whatever the number
// of sequences and their lengths.
//
// Work: an item is one sequence and kv head (its rows x group <= 8 NT pairs share every key); its
// keys are steps of 16, which lie in one page.  All items' steps form one line, and CTA b takes
// steps b Q .. b Q + Q - 1 of it (Q = total / CTAs, found on the device from the lengths, so a
// captured call follows them).  An item cut by such a border leaves partial sums in the workspace
// (at most two slots per CTA), and the CTA that arrives last at the item joins its parts in
// order: the result does not depend on the order of arrival.
//
// Within a CTA every warp works alone on every W-th step of the segment: it copies steps into a
// ring of its own in shared memory with cp.async, STAGES - 1 ahead, and keeps its own running
// maximum, sum and output in registers; warps join once per segment.  No barrier, no producer.
//   S^T = K Q^T   mma.m16n8k16: 16 keys x 8 pairs, so a group of 4 to 8 heads wastes no more than
//                 half of the tile (with pairs as the 16-row side it would be 8 of 16 or more)
//   O^T += V^T P^T  P^T comes from S^T by one 8x8 transpose per 8 keys (movmatrix), all in registers
// P goes into its product as two bf16 parts (2^-16 of it is lost) for up to 16 pairs, where reading the pages
// hides the second product: 163 us for the 64 sequences below either way, 159 and 158 for 16 sequences with three
// rows.  With 32 pairs the products bound the kernel (265 instead of 225 us for eight rows), and over 4-bit
// pages its issue slots do (15 % more for the 32 sequences below, 22 % for three rows of 16): there P is
// rounded to bf16 once, as in the prefill's attention.
// The running maximum used for P is raised only when it grows by more than 2^8 (as in the
// prefill's kernel); sums use the same reference, so O / l is exact.
// 4-bit pages: codes go from shared memory to operands in registers: a mask and one multiply-add give a
// pair's (n - 8) / 64 exactly (see code_pair; an offset left in the sums would cancel against results that
// are far smaller than it).  Keys: their products with the bf16 queries are exact, a key's scales multiply
// its partial scores of each 32 dims in fp32, and the 64 goes into the scores' factor.  (A mask alone makes
// fp16 operands (n + 8) 2^-24 for queries turned into fp16: 113 instead of 119 us for the 32 sequences below
// with two CTAs per SM, but a score was off by up to 2^-21 of the row's largest element times the keys' scales,
// which is much where the codes at the large elements are 0.)
// Values: the value's scale multiplies P in fp32 before its one rounding to bf16; the 64 goes into the last
// division.
// Measured (GB300, 6.8 TB/s copy rate), host call included: 64 sequences of 3.3-8.2 K tokens, window
// 4096, Mistral-7B heads 163 us, 6.5 TB/s of pages; one sequence of 128 K tokens, 14B heads, 93 us, 5.7 TB/s
// (10 us of it are finding the shares and joining 304 parts).  4-bit pages, 32 sequences of 10-16 K
// tokens: 112 us, 4.4 TB/s: bound by instruction issue and its dependencies, not by HBM.
// Tokens that no row sees are filled with zeros instead of loaded (values, scales), so what they
// hold does not matter.
#include <climits>

#include "paged.cuh"

namespace blend {
namespace {

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float pow2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The G bf16 scales of a row as fp32.
template <int G> __device__ __forceinline__ void scales(const uint8_t* p, float (&f)[G]) {
    uint32_t w[G / 2];
    if constexpr (G == 4) {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        w[0] = x.x;
        w[1] = x.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
#pragma unroll
    for (int i = 0; i < G / 2; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// Token (0..15) of a step that takes row i of the 4-bit S^T tile: the order under which the lanes'
// shared-memory reads of both K and V fall on distinct banks.
__device__ __forceinline__ int token4(int i) {
    const int c = (i & 7) >> 1;
    return (i & 8) + ((i & 1) ? 4 + (c ^ 1) : c);
}

template <bool I4, int D> struct StepCfg {
    static constexpr int ROW = I4 ? D / 2 : 2 * D;            // bytes of a K or V row
    static constexpr int KV = PAGED_STEP * ROW;               // one of K, V
    static constexpr int SCALE = I4 ? D / 16 : 0;             // bytes of a row's scales
    static constexpr int BYTES = 2 * KV + 2 * PAGED_STEP * SCALE;  // K, V, K scales, V scales
};
// U: steps of a stage (and of a pass through the softmax)
template <bool I4, int D, int NT, int W, int STAGES, int U> struct SplitCfg {
    static constexpr int PER_SM = I4 && NT == 1 ? 3 : 2;  // CTAs of an SM (see launch_nt)
    static constexpr int CTAS = 152 * PER_SM;
    static_assert(CTAS <= PAGED_MAX_CTAS, "workspace");
    static constexpr int RING = W * STAGES * U * StepCfg<I4, D>::BYTES;
    static constexpr int OPAD = D + 4;  // distinct banks for the four pairs of a quad
    static constexpr int JOIN = W * 8 * NT * OPAD * 4;
    static constexpr int PARTS = CTAS * 8 * NT * 4 + W * 4 * 32 * 16;  // weights of an item's parts, sums of a round
    static constexpr int MOST = RING > JOIN ? RING : JOIN;
    static constexpr int SMEM = MOST > PARTS ? MOST : PARTS;
};

template <bool I4, int D, int NT, int W, int STAGES, int U>
__global__ void __launch_bounds__(W * 32, (SplitCfg<I4, D, NT, W, STAGES, U>::PER_SM))
    k_paged_split(const __grid_constant__ PagedAttn a) {
    using S = StepCfg<I4, D>;
    using Cfg = SplitCfg<I4, D, NT, W, STAGES, U>;
    constexpr int R = 8 * NT, T = W * 32, KT = D / 16, G = D / 32, OPAD = Cfg::OPAD;
    constexpr bool P2 = !I4 && NT <= 2;  // P in two parts
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int pre[BLEND_MAX_SEQS + 1];
    __shared__ int scan[W], items[W];
    __shared__ int s_row[R], s_off[R];  // a pair's row, and its offset in the output from the item's first
    __shared__ float sm[W][R], sl[W][R], sM[R], sL[R];
    __shared__ int last_sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r = lane >> 2, c = lane & 3;
    const float sc = I4 ? a.scale_log2 * CODE_UNIT : a.scale_log2;  // score to exponent of 2
    const int hkv = a.pg.hkv, n_seq = a.pg.n_seq;

    if (tid < R) {
        s_row[tid] = tid / a.group;
        s_off[tid] = (tid / a.group * a.hq + tid % a.group) * D;
    }
    // ---- the line of steps: pre[s] = steps of all items of sequences before s
    {
        const int per = (n_seq + T - 1) / T;
        int mine = 0, active = 0;
        for (int i = 0; i < per; ++i) {
            const int s = tid * per + i;
            if (s >= n_seq) break;
            const SeqInfo si = seq_info(a, s);
            const int np = si.n_q * a.group;
            int n = 0;
            if (np > 0 && np <= R)
                // a sequence without a visible key keeps one (empty) step: its rows get their zeros
                n = max(1, key_range<PAGED_STEP>(si.len - si.n_q, si.len - 1, a.window, a.n_sink).total());
            pre[s + 1] = n * hkv;
            mine += n * hkv;
            active += n > 0;
        }
        active = __reduce_add_sync(0xffffffffu, active);
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) scan[warp] = incl;
        if (lane == 0) items[warp] = active;
        __syncthreads();
        int at = incl - mine;
        for (int w = 0; w < warp; ++w) at += scan[w];
        for (int i = 0; i < per; ++i) {
            const int s = tid * per + i;
            if (s >= n_seq) break;
            at += pre[s + 1];
            pre[s + 1] = at;
        }
        if (tid == 0) pre[0] = 0;
        __syncthreads();
    }
    const int total = pre[n_seq];
    int n_item = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) n_item += items[w];
    if (n_item == 0) return;
    n_item *= hkv;
    // An equal share of the line, but at least a pass per warp.  Leaving parts of an item and joining
    // them takes about as long as five more steps of every warp, so items of fewer than six steps per
    // warp are never cut for a small total, nor those of fewer than four at a border (GB300, bf16, 8 items, in a
    // captured graph: 22 steps 7.5 us whole, 8.4 in six parts; 32 steps 8.1 either way; 44 steps 8.3 in 11
    // parts).  Eight warps on every SM, one CTA each, measured 7.0, 7.6 and 8.6 us there, but 9.1 instead of
    // 8.8 for 63 steps and 15.6 instead of 13.8 for 1000.
    constexpr int SHORT = 6 * W;
    const int per_item = Shares::parts(total, n_item);
    const int quota = max(Shares::parts(total, (int)gridDim.x), per_item < SHORT ? per_item : U * W);
    const Shares sh(total, quota, min(2 * W, quota));
    const int share = blockIdx.x;
    if (share >= sh.n) return;
    int x = sh.start(share);
    int seq;
    {
        int lo = 0, hi = n_seq - 1;  // last sequence with pre[seq] <= x (empty ones before it share the value)
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (pre[mid] <= x) lo = mid;
            else hi = mid - 1;
        }
        seq = lo;
    }
    const uint32_t ring = smem_u32(smem) + warp * STAGES * U * S::BYTES;
    uint8_t* ring_p = smem + warp * STAGES * U * S::BYTES;

    // where this lane's 16-byte chunks of a step come from and go to; the chunks of a row are permuted
    // in shared memory so that the rows of one read fall on distinct banks (bf16: chunk ^ row % 8)
    constexpr int CH = S::ROW / 16;
    auto ring_at = [&](uint32_t first, int u) {  // the lane's chunk 32 u further on: 32 / CH rows down
        return (I4 ? first : first ^ (uint32_t)(((32 / CH * u) & 7) << 4)) + u * 512;
    };
    const int t_lane = lane / CH, ch_lane = lane % CH;
    const uint32_t k_at = t_lane * S::ROW + (I4 ? ch_lane : ch_lane ^ (t_lane & 7)) * 16;
    const uint32_t v_at = S::KV + t_lane * S::ROW +
                          (!I4 ? ch_lane ^ (t_lane & 7) : D == 128 ? ch_lane ^ (((t_lane >> 1) & 1) << 1) : ch_lane) * 16;
    const char* k_lane = a.pg.k + lane * 16;
    const char* v_lane = a.pg.v + lane * 16;
    const char* s_lane = (lane < 16 ? a.pg.ks : a.pg.vs) + (lane & 15) * S::SCALE;

    // what holds for all heads of a sequence
    SeqInfo si{0, 0, 0};
    KeyRange kr{0, 0, 0};
    int known = -1, steps = 0, npair = 0, p0 = 0, p1 = 0, clean0 = 0, n_clean = 0;

    while (x < total) {
        while (pre[seq + 1] <= x) ++seq;  // skips sequences without steps
        if (seq != known) steps = (pre[seq + 1] - pre[seq]) / hkv;
        const int head = (x - pre[seq]) / steps;
        const int item0 = pre[seq] + head * steps;
        x = item0 + steps;  // the next item
        if (sh.first(item0, x) > share) break;
        if (sh.last(item0, x) < share) {
            known = -1;
            continue;
        }
        const int s0 = sh.begin(share, item0, x), s1 = sh.end(share, item0, x);
        if (seq != known) {
            known = seq;
            si = seq_info(a, seq);
            npair = si.n_q * a.group;
            p0 = si.len - si.n_q;
            p1 = si.len - 1;
            kr = key_range<PAGED_STEP>(p0, p1, a.window, a.n_sink);
            // steps of the window's range that every row sees whole: no masks, no token to leave out
            clean0 = kr.n_a + max(0, (max(p1 - a.window, -1) + PAGED_STEP) / PAGED_STEP - kr.first_b);
            n_clean = (p0 + 1) / PAGED_STEP - kr.first_b + kr.n_a - clean0;
        }
        const int n_real = min(s1, kr.total());  // the empty step of a sequence without keys is none
        auto clean = [&](int i) { return n_clean > 0 && (unsigned)(i - clean0) < (unsigned)n_clean; };

        // ---- loads of step i into a place of the ring
        auto load = [&](int i, uint32_t dst, int entry) {
            const int j0 = kr.block(i) * PAGED_STEP;
            const long long row = page_row(a.pg, checked_page(a.pg, entry, a.err), head, j0 & ((1 << a.pg.shift) - 1));
            const char* ksrc = k_lane + row * S::ROW;
            const char* vsrc = v_lane + row * S::ROW;
            constexpr int N = S::KV / 512;
            if (clean(i)) {
#pragma unroll
                for (int u = 0; u < N; ++u) {
                    cp_async<16>(dst + ring_at(k_at, u), ksrc + u * 512);
                    cp_async<16>(dst + ring_at(v_at, u), vsrc + u * 512);
                }
                if constexpr (I4) cp_async<S::SCALE>(dst + 2 * S::KV + lane * S::SCALE, s_lane + row * S::SCALE);
            } else {
#pragma unroll
                for (int u = 0; u < N; ++u) {
                    const bool ok = seen_by_any(j0 + (lane + 32 * u) / CH, p0, p1, a.window, a.n_sink);
                    cp_async<16>(dst + ring_at(k_at, u), ksrc + u * 512, ok);
                    cp_async<16>(dst + ring_at(v_at, u), vsrc + u * 512, ok);
                }
                if constexpr (I4)
                    cp_async<S::SCALE>(dst + 2 * S::KV + lane * S::SCALE, s_lane + row * S::SCALE,
                                       seen_by_any(j0 + (lane & 15), p0, p1, a.window, a.n_sink));
            }
        };
        auto entry_at = [&](int i) { return page_entry(a.pg, seq, kr.block(i) * PAGED_STEP); };

        // ---- queries, asked for before the keys
        uint32_t qf[NT][KT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int p = nt * 8 + r;
            const bool ok = p < npair;
            const bf16* qr = reinterpret_cast<const bf16*>(a.q) + (si.row0 + (ok ? s_row[p] : 0)) * a.ld_q + head * a.group * D +
                             (ok ? s_off[p] - s_row[p] * a.hq * D : 0);
            if constexpr (!I4) {
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    qf[nt][kt][0] = ok ? *reinterpret_cast<const uint32_t*>(qr + 16 * kt + 2 * c) : 0u;
                    qf[nt][kt][1] = ok ? *reinterpret_cast<const uint32_t*>(qr + 16 * kt + 2 * c + 8) : 0u;
                }
            } else {
#pragma unroll
                for (int g = 0; g < G; ++g) {  // dims 32 g + 8 c .. +7
                    const uint4 w = ok ? *reinterpret_cast<const uint4*>(qr + 32 * g + 8 * c) : make_uint4(0, 0, 0, 0);
                    qf[nt][2 * g][0] = w.x;
                    qf[nt][2 * g][1] = w.y;
                    qf[nt][2 * g + 1][0] = w.z;
                    qf[nt][2 * g + 1][1] = w.w;
                }
            }
        }
        // ---- first steps on their way; the warp takes U neighbouring steps of every U W
        int li = s0 + U * warp;  // next step to load
        int entry[U];
        auto next_entries = [&]() {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (li + u < n_real) entry[u] = entry_at(li + u);
        };
        auto load_next = [&](int st) {
            if (li < n_real) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (li + u < n_real) load(li + u, ring + (st * U + u) * S::BYTES, entry[u]);
                li += U * W;
                next_entries();
            }
            cp_commit();
        };
        next_entries();
#pragma unroll
        for (int st = 0; st < STAGES - 1; ++st) load_next(st);
        // ---- the pairs' positions
        int rp[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int pc = nt * 8 + 2 * c + e;
                rp[nt][e] = pc < npair ? p0 + s_row[pc] : -1;
            }
        float m[NT][2], ref[NT][2], l[NT][2], o[KT][NT][4];  // ref: m, or 0 while no key was seen
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -INFINITY;
            ref[nt][0] = ref[nt][1] = l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[t][nt][e] = 0.f;
        }

        int stage = 0;
        for (int i = s0 + U * warp; i < n_real; i += U * W) {
            cp_wait<STAGES - 2>();
            __syncwarp();
            load_next(stage == 0 ? STAGES - 1 : stage - 1);
            float s[U][NT][4];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t kb = ring + (stage * U + u) * S::BYTES;
                if constexpr (!I4) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) s[u][nt][0] = s[u][nt][1] = s[u][nt][2] = s[u][nt][3] = 0.f;
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt) {
                        uint32_t k[4];
                        const int t = lane & 15, ch = 2 * kt + (lane >> 4);
                        ldsm4(k, kb + t * S::ROW + ((ch ^ (t & 7)) << 4));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma(s[u][nt], k, qf[nt][kt][0], qf[nt][kt][1]);
                    }
                } else {
                    const uint8_t* kp = ring_p + (stage * U + u) * S::BYTES;
                    const int t0 = token4(r), t1 = t0 + 8;
                    uint32_t w0[G], w1[G];
                    float f0[G], f1[G];
                    const uint8_t* sp = kp + 2 * S::KV;
                    if constexpr (D == 128) {
                        const uint4 u0 = *reinterpret_cast<const uint4*>(kp + t0 * S::ROW + c * 16);
                        const uint4 u1 = *reinterpret_cast<const uint4*>(kp + t1 * S::ROW + c * 16);
                        w0[0] = u0.x; w0[1] = u0.y; w0[2] = u0.z; w0[3] = u0.w;
                        w1[0] = u1.x; w1[1] = u1.y; w1[2] = u1.z; w1[3] = u1.w;
                    } else {
                        const uint2 u0 = *reinterpret_cast<const uint2*>(kp + t0 * S::ROW + c * 8);
                        const uint2 u1 = *reinterpret_cast<const uint2*>(kp + t1 * S::ROW + c * 8);
                        w0[0] = u0.x; w0[1] = u0.y;
                        w1[0] = u1.x; w1[1] = u1.y;
                    }
                    scales<G>(sp + t0 * S::SCALE, f0);
                    scales<G>(sp + t1 * S::SCALE, f1);
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        const uint32_t v0 = w0[g] >> 8, v1 = w1[g] >> 8;
                        const uint32_t ka[4] = {code_pair<false>(w0[g]), code_pair<false>(w1[g]), code_pair<true>(w0[g]), code_pair<true>(w1[g])};
                        const uint32_t kc[4] = {code_pair<false>(v0), code_pair<false>(v1), code_pair<true>(v0), code_pair<true>(v1)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float d[4] = {0.f, 0.f, 0.f, 0.f};
                            mma(d, ka, qf[nt][2 * g][0], qf[nt][2 * g][1]);
                            mma(d, kc, qf[nt][2 * g + 1][0], qf[nt][2 * g + 1][1]);
                            s[u][nt][0] = g ? fmaf(d[0], f0[g], s[u][nt][0]) : d[0] * f0[g];
                            s[u][nt][1] = g ? fmaf(d[1], f0[g], s[u][nt][1]) : d[1] * f0[g];
                            s[u][nt][2] = g ? fmaf(d[2], f1[g], s[u][nt][2]) : d[2] * f1[g];
                            s[u][nt][3] = g ? fmaf(d[3], f1[g], s[u][nt][3]) : d[3] * f1[g];
                        }
                    }
                }
                // ---- mask (steps at an edge, and a pass's missing last step)
                if (!clean(i + u) || i + u >= n_real) {
                    const int j0 = kr.block(i + u) * PAGED_STEP;
                    const int ja = i + u < n_real ? j0 + (I4 ? token4(r) : r) : INT_MAX - 8, jb = ja + 8;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            if (!sees(ja, rp[nt][e], a.window, a.n_sink)) s[u][nt][e] = -INFINITY;
                            if (!sees(jb, rp[nt][e], a.window, a.n_sink)) s[u][nt][2 + e] = -INFINITY;
                        }
                }
            }
            // ---- running maximum: looked at across lanes only when some score has outgrown it by 2^8
            bool need = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float v = fmaxf(s[0][nt][e], s[0][nt][2 + e]);
#pragma unroll
                    for (int u = 1; u < U; ++u) v = fmaxf(v, fmaxf(s[u][nt][e], s[u][nt][2 + e]));
                    need = need || v * sc > m[nt][e] + 8.f;
                }
            if (__any_sync(0xffffffffu, need)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float v = fmaxf(s[0][nt][e], s[0][nt][2 + e]);
#pragma unroll
                        for (int u = 1; u < U; ++u) v = fmaxf(v, fmaxf(s[u][nt][e], s[u][nt][2 + e]));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                        const float mx = v * sc;
                        if (!(mx > m[nt][e] + 8.f)) continue;
                        const float corr = pow2(m[nt][e] - mx);
                        m[nt][e] = ref[nt][e] = mx;
                        l[nt][e] *= corr;
#pragma unroll
                        for (int t = 0; t < KT; ++t) {
                            o[t][nt][e] *= corr;
                            o[t][nt][2 + e] *= corr;
                        }
                    }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t vb = ring + (stage * U + u) * S::BYTES + S::KV;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        s[u][nt][e] = pow2(fmaf(s[u][nt][e], sc, -ref[nt][e]));
                        s[u][nt][2 + e] = pow2(fmaf(s[u][nt][2 + e], sc, -ref[nt][e]));
                        l[nt][e] += s[u][nt][e] + s[u][nt][2 + e];
                    }
                if constexpr (!I4) {
                    uint32_t pb[NT][2], pl[NT][2];  // P, and what its rounding leaves
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float x = s[u][nt][2 * e], y = s[u][nt][2 * e + 1];
                            const uint32_t hi = pack2(x, y);
                            pb[nt][e] = transpose8(hi);
                            if constexpr (P2) pl[nt][e] = transpose8(pack2(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u)));
                        }
#pragma unroll
                    for (int t = 0; t < KT; ++t) {
                        uint32_t v[4];
                        const int tok = ((lane >> 4) << 3) + (lane & 7), ch = 2 * t + ((lane >> 3) & 1);
                        ldsm4t(v, vb + tok * S::ROW + ((ch ^ (tok & 7)) << 4));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma(o[t][nt], v, pb[nt][0], pb[nt][1]);
                            if constexpr (P2) mma(o[t][nt], v, pl[nt][0], pl[nt][1]);
                        }
                    }
                } else if (u == 0 || i + u < n_real) {  // (a missing step's place in the ring holds no values)
                    const uint8_t* vp = ring_p + (stage * U + u) * S::BYTES + S::KV;
                    const uint8_t* sp = vp + S::KV + PAGED_STEP * S::SCALE;
                    float f0[G], f1[G];  // scales of the keys whose P this lane holds
                    scales<G>(sp + token4(r) * S::SCALE, f0);
                    scales<G>(sp + (token4(r) + 8) * S::SCALE, f1);
                    // tokens of columns 2c, 2c + 1, 2c + 8, 2c + 9 of V^T
                    const int tk[4] = {c, 4 + (c ^ 1), 8 + c, 12 + (c ^ 1)};
                    uint32_t v[4][G / 2];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if constexpr (D == 128) {
                            const uint2 w = *reinterpret_cast<const uint2*>(
                                vp + tk[q] * S::ROW + (((r >> 1) ^ (((tk[q] >> 1) & 1) << 1)) << 4) + ((r & 1) << 3));
                            v[q][0] = w.x; v[q][1] = w.y;
                        } else {
                            v[q][0] = *reinterpret_cast<const uint32_t*>(vp + tk[q] * S::ROW + (r << 2));
                        }
                    }
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        const uint32_t sel = (g & 1) ? 0x7632 : 0x5410;  // the 16-bit half of group g
                        const uint32_t x01 = __byte_perm(v[0][g >> 1], v[1][g >> 1], sel);
                        const uint32_t x23 = __byte_perm(v[2][g >> 1], v[3][g >> 1], sel);
                        const uint32_t y01 = x01 >> 8, y23 = x23 >> 8;
                        const uint32_t va[4] = {code_pair<false>(x01), code_pair<true>(x01), code_pair<false>(x23), code_pair<true>(x23)};
                        const uint32_t vc[4] = {code_pair<false>(y01), code_pair<true>(y01), code_pair<false>(y23), code_pair<true>(y23)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint32_t b0 = transpose8(pack2(s[u][nt][0] * f0[g], s[u][nt][1] * f0[g]));
                            const uint32_t b1 = transpose8(pack2(s[u][nt][2] * f1[g], s[u][nt][3] * f1[g]));
                            mma(o[2 * g][nt], va, b0, b1);
                            mma(o[2 * g + 1][nt], vc, b0, b1);
                        }
                    }
                }
            }
            stage = stage == STAGES - 1 ? 0 : stage + 1;
        }

        // ---- join the warps
        cp_wait<0>();
        __syncthreads();  // every warp is done with its ring
        float* so = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float v = l[nt][e];
                v += __shfl_xor_sync(0xffffffffu, v, 4);
                v += __shfl_xor_sync(0xffffffffu, v, 8);
                v += __shfl_xor_sync(0xffffffffu, v, 16);
                const int pc = nt * 8 + 2 * c + e;
                if (r == 0) {
                    sm[warp][pc] = isnan(v) ? v : m[nt][e];  // a NaN must not lose its weight below
                    sl[warp][pc] = v;
                }
                float* d = so + (warp * R + pc) * OPAD;
#pragma unroll
                for (int t = 0; t < KT; ++t) {
                    const int d0 = I4 ? 32 * (t >> 1) + 4 * r + 2 * (t & 1) : 16 * t + r, d1 = I4 ? d0 + 1 : d0 + 8;
                    d[d0] = o[t][nt][e];
                    d[d1] = o[t][nt][2 + e];
                }
            }
        __syncthreads();
        if (tid < R) {
            float mx = -INFINITY, sum = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) mx = max_nan(mx, sm[w][tid]);
            const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float f = pow2(sm[w][tid] - ref);
                sum += sl[w][tid] * f;
                sm[w][tid] = f;
            }
            sM[tid] = mx;
            sL[tid] = I4 ? sum * (1.f / CODE_UNIT) : sum;  // (the outputs lack the unit of their codes)
        }
        __syncthreads();
        const bool whole_item = s0 == 0 && s1 == steps;
        float* slot = a.part + (size_t)(2 * blockIdx.x + (s0 == 0 ? 1 : 0)) * paged_slot_floats(D);
        bf16* out = reinterpret_cast<bf16*>(a.out) + ((long long)si.row0 * a.hq + head * a.group) * D;
        for (int i = tid; i < npair * (D / 2); i += T) {
            const int p = i / (D / 2), e = 2 * (i % (D / 2));
            float y0 = 0.f, y1 = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float f = sm[w][p];
                const float2 v = *reinterpret_cast<const float2*>(so + (w * R + p) * OPAD + e);
                y0 = fmaf(v.x, f, y0);
                y1 = fmaf(v.y, f, y1);
            }
            if (whole_item) {
                const float inv = sL[p] == 0.f ? 0.f : 1.f / sL[p];
                *reinterpret_cast<uint32_t*>(out + s_off[p] + e) = pack2(y0 * inv, y1 * inv);
            } else {
                *reinterpret_cast<float2*>(slot + p * D + e) = make_float2(y0, y1);
            }
        }
        if (!whole_item) {
            const int first = sh.first(item0, item0 + steps), n_part = sh.last(item0, item0 + steps) - first + 1;
            if (tid < npair) {
                slot[PAGED_MAX_TILE * D + tid] = sM[tid];
                slot[PAGED_MAX_TILE * (D + 1) + tid] = sL[tid];
            }
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const int before = atomicAdd(a.count + first, 1);
                last_sh = before == n_part - 1;
                if (last_sh) a.count[first] = 0;  // ready for the next launch
            }
            __syncthreads();
            if (last_sh) {
                __threadfence();
                // Part k is CTA first + k's: its slot 1 when the item starts there, else slot 0.  First the
                // parts' weights, a warp per pair; then threads share the parts of every four outputs.
                const size_t sf = paged_slot_floats(D);
                const float* base = a.part + (size_t)2 * first * sf;
                auto part = [&](int k) { return base + (size_t)(2 * k + (k == 0 ? 1 : 0)) * sf; };
                float* wt = reinterpret_cast<float*>(smem);  // [part][R], of the ring
                for (int p = warp; p < npair; p += W) {
                    float mx = -INFINITY;
                    for (int k = lane; k < n_part; k += 32) {
                        const float v = __ldcg(part(k) + PAGED_MAX_TILE * D + p);
                        wt[k * R + p] = v;
                        mx = max_nan(mx, v);
                    }
#pragma unroll
                    for (int x2 = 16; x2; x2 >>= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, x2));
                    const float ref = mx == -INFINITY ? 0.f : mx;
                    float sum = 0.f;
                    for (int k = lane; k < n_part; k += 32) {
                        const float f = pow2(wt[k * R + p] - ref);
                        wt[k * R + p] = f;
                        sum += f * __ldcg(part(k) + PAGED_MAX_TILE * (D + 1) + p);
                    }
#pragma unroll
                    for (int x2 = 16; x2; x2 >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x2);
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;
                    for (int k = lane; k < n_part; k += 32) wt[k * R + p] *= inv;
                }
                __syncthreads();
                // each warp adds every W-th part of 128 x 4 outputs (four of a lane: 16 loads on their way), then
                // the warps' sums are added in order
                constexpr int V4 = D / 4, Q = 4;
                const int n_out = npair * V4;
                float4* acc = reinterpret_cast<float4*>(wt + ((n_part * R + 3) & ~3));  // [W][Q][32] of one round
                for (int q0 = 0; q0 < n_out; q0 += 32 * Q) {
                    float4 y[Q];
#pragma unroll
                    for (int j = 0; j < Q; ++j) y[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                    for (int k = warp; k < n_part; k += W) {
                        const float4* src = reinterpret_cast<const float4*>(part(k));  // pair p's output e4 is p V4 + e4
#pragma unroll
                        for (int j = 0; j < Q; ++j) {
                            const int q = q0 + 32 * j + lane;
                            if (q < n_out) {
                                const float4 v = __ldcg(src + q);
                                const float f = wt[k * R + q / V4];
                                y[j].x = fmaf(v.x, f, y[j].x);
                                y[j].y = fmaf(v.y, f, y[j].y);
                                y[j].z = fmaf(v.z, f, y[j].z);
                                y[j].w = fmaf(v.w, f, y[j].w);
                            }
                        }
                    }
#pragma unroll
                    for (int j = 0; j < Q; ++j) acc[(warp * Q + j) * 32 + lane] = y[j];
                    __syncthreads();
                    for (int i = tid; i < 32 * Q && q0 + i < n_out; i += T) {
                        float4 t = acc[i];
#pragma unroll
                        for (int x2 = 1; x2 < W; ++x2) {
                            const float4 v = acc[x2 * 32 * Q + i];
                            t.x += v.x;
                            t.y += v.y;
                            t.z += v.z;
                            t.w += v.w;
                        }
                        const int p = (q0 + i) / V4, e4 = (q0 + i) % V4;
                        *reinterpret_cast<uint2*>(out + s_off[p] + 4 * e4) = make_uint2(pack2(t.x, t.y), pack2(t.z, t.w));
                    }
                    __syncthreads();
                }
            }
        }
        __syncthreads();  // the ring is loaded again for the next segment
    }
}

template <bool I4, int D, int NT, int W, int STAGES, int U> void launch_one(const PagedAttn& a, cudaStream_t s) {
    using Cfg = SplitCfg<I4, D, NT, W, STAGES, U>;
    auto kern = k_paged_split<I4, D, NT, W, STAGES, U>;
    static const bool ready = [&] {
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM);
        return true;
    }();
    (void)ready;
    kern<<<Cfg::CTAS, W * 32, Cfg::SMEM, s>>>(a);
    note_launch(1);
}
template <bool I4, int D> void launch_nt(const PagedAttn& a, cudaStream_t s) {
    const int pairs = a.max_q * a.group;
    // Four warps, two CTAs per SM.  4-bit pages of up to 8 pairs: two steps a pass and three CTAs, at 165 registers (32
    // sequences of up to 16 K tokens, 128 short ones, one of 8 K: 111.7, 33.7 and 14.0 us; two CTAs 119, 37.4 and 13.2;
    // those with eight warps each 116, 36.5 and 14.5, or with one step a pass in a ring of four 128, 35.9 and 13.1).
    if (pairs <= 8) {
        if constexpr (I4) launch_one<I4, D, 1, 4, 3, 2>(a, s);
        else launch_one<I4, D, 1, 4, 3, 1>(a, s);
    } else if (pairs <= 16) launch_one<I4, D, 2, 4, I4 ? 5 : 3, 1>(a, s);
    else launch_one<I4, D, 4, 4, I4 ? 5 : 3, 1>(a, s);
}

}  // namespace

void launch_paged_attn_split(bool i4, const PagedAttn& a, int d, cudaStream_t s) {
    if (i4) {
        if (d == 64) launch_nt<true, 64>(a, s);
        else launch_nt<true, 128>(a, s);
    } else {
        if (d == 64) launch_nt<false, 64>(a, s);
        else launch_nt<false, 128>(a, s);
    }
}

}  // namespace blend

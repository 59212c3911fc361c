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
// The running maximum used for P is raised only when it grows by more than 2^8 (as in the
// prefill's kernel); sums use the same reference, so O / l is exact.
// 4-bit pages: codes go from shared memory to operands in registers, (w >> 4 i) & 0x000F000F being
// a pair of operand elements in the order that the rows are packed in; n + 128 is the bf16 0x4300
// | n, so one subtraction gives n - 8 exactly.  A key's scales multiply its partial scores of
// each 32 dims in fp32, a value's scale multiplies P (rounded to bf16 once more: a value n s would
// be rounded there as well).
// Measured (GB300, 6.8 TB/s copy rate): 64 sequences of 3.3-8.2 K tokens, window 4096, Mistral-7B
// heads 172 us, 6.2 TB/s of pages.
// Tokens that no row sees are filled with zeros instead of loaded (values, scales), so what they
// hold does not matter.
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
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
// Codes at bits 4 i and 16 + 4 i of w as two bf16 values n - 8.
__device__ __forceinline__ uint32_t codes2(uint32_t w, int i) {
    uint32_t x = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;  // 128 + n
    const uint32_t off = 0x43084308u;                            // 136
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&off));
    return *reinterpret_cast<const uint32_t*>(&r);
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
template <bool I4, int D, int NT, int W, int STAGES> struct SplitCfg {
    static constexpr int RING = W * STAGES * StepCfg<I4, D>::BYTES;
    static constexpr int OPAD = D + 4;  // distinct banks for the four pairs of a quad
    static constexpr int JOIN = W * 8 * NT * OPAD * 4;
    static constexpr int PARTS = PAGED_MAX_CTAS * 4;  // weights of an item's parts, one pair at a time
    static constexpr int SMEM = (RING > JOIN ? RING : JOIN) > PARTS ? (RING > JOIN ? RING : JOIN) : PARTS;
};

template <bool I4, int D, int NT, int W, int STAGES>
__global__ void __launch_bounds__(W * 32, 2)
    k_paged_split(const __grid_constant__ PagedAttn a) {
    using S = StepCfg<I4, D>;
    using Cfg = SplitCfg<I4, D, NT, W, STAGES>;
    constexpr int R = 8 * NT, T = W * 32, KT = D / 16, G = D / 32, OPAD = Cfg::OPAD;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int pre[BLEND_MAX_SEQS + 1];
    __shared__ int scan[W];
    __shared__ float sm[W][R], sl[W][R], sM[R], sL[R];
    __shared__ int last_sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r = lane >> 2, c = lane & 3;
    const int hkv = a.pg.hkv, n_seq = a.pg.n_seq;

    // ---- the line of steps: pre[s] = steps of all items of sequences before s
    {
        const int per = (n_seq + T - 1) / T;
        int mine = 0;
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
        }
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) scan[warp] = incl;
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
    const int quota = max(W, (total + (int)gridDim.x - 1) / (int)gridDim.x);
    long long x64 = (long long)blockIdx.x * quota;
    if (x64 >= total) return;
    int x = (int)x64;
    const int x_end = (int)min((long long)total, x64 + quota);
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
    const uint32_t ring = smem_u32(smem) + warp * STAGES * S::BYTES;
    uint8_t* ring_p = smem + warp * STAGES * S::BYTES;

    while (x < x_end) {
        while (pre[seq + 1] <= x) ++seq;  // skips sequences without steps
        const SeqInfo si = seq_info(a, seq);
        const int steps = (pre[seq + 1] - pre[seq]) / hkv;
        const int head = (x - pre[seq]) / steps;
        const int item0 = pre[seq] + head * steps;
        const int s0 = x - item0, s1 = min(steps, s0 + (x_end - x));
        const int npair = si.n_q * a.group;
        const int p0 = si.len - si.n_q, p1 = si.len - 1;
        const KeyRange kr = key_range<PAGED_STEP>(p0, p1, a.window, a.n_sink);
        const int n_real = min(s1, kr.total());  // the empty step of a sequence without keys is none

        // ---- loads of step i into a stage
        auto load = [&](int i, int stage, int page) {
            const int j0 = kr.block(i) * PAGED_STEP;
            const long long row = page_row(a.pg, page, head, j0 & ((1 << a.pg.shift) - 1));
            const int j1 = j0 + PAGED_STEP - 1;
            const bool whole = j1 <= p1 && (j1 < a.n_sink || j0 > p0 - a.window);  // some row sees each of them
            const uint32_t dst = ring + stage * S::BYTES;
            const char* ksrc = a.pg.k + row * S::ROW;
            const char* vsrc = a.pg.v + row * S::ROW;
            constexpr int CH = S::ROW / 16, N = S::KV / 512;
#pragma unroll
            for (int u = 0; u < N; ++u) {
                const int q = lane + 32 * u, t = q / CH, ch = q % CH;
                const bool ok = whole || seen_by_any(j0 + t, p0, p1, a.window, a.n_sink);
                int kch, vch;  // chunk order in shared memory: rows of one read on distinct banks
                if constexpr (!I4) kch = vch = ch ^ (t & 7);
                else {
                    kch = ch;
                    vch = D == 128 ? ch ^ (((t >> 1) & 1) << 1) : ch;
                }
                cp_async<16>(dst + t * S::ROW + kch * 16, ksrc + q * 16, ok);
                cp_async<16>(dst + S::KV + t * S::ROW + vch * 16, vsrc + q * 16, ok);
            }
            if constexpr (I4) {
                const int t = lane & 15;
                const char* src = (lane < 16 ? a.pg.ks : a.pg.vs) + (row + t) * S::SCALE;
                cp_async<S::SCALE>(dst + 2 * S::KV + lane * S::SCALE, src,
                                   whole || seen_by_any(j0 + t, p0, p1, a.window, a.n_sink));
            }
        };
        auto page_at = [&](int i) { return page_of(a.pg, seq, kr.block(i) * PAGED_STEP, a.err); };

        // ---- first steps on their way
        int li = s0 + warp;  // next step to load
        int page = li < n_real ? page_at(li) : 0;
#pragma unroll
        for (int st = 0; st < STAGES - 1; ++st) {
            if (li < n_real) {
                load(li, st, page);
                li += W;
                if (li < n_real) page = page_at(li);
            }
            cp_commit();
        }
        // ---- queries (B operand) and the pairs' positions
        uint32_t qf[NT][KT][2];
        int rp[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int p = nt * 8 + r;
            const bool ok = p < npair;
            const bf16* qr = reinterpret_cast<const bf16*>(a.q) + (long long)(si.row0 + (ok ? p / a.group : 0)) * a.ld_q +
                             (head * a.group + (ok ? p % a.group : 0)) * D;
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                // 4-bit: the dims of a lane are 8 in a row of each 32
                const int e0 = I4 ? 32 * (kt >> 1) + 8 * c + 4 * (kt & 1) : 16 * kt + 2 * c, e1 = I4 ? e0 + 2 : e0 + 8;
                qf[nt][kt][0] = ok ? *reinterpret_cast<const uint32_t*>(qr + e0) : 0u;
                qf[nt][kt][1] = ok ? *reinterpret_cast<const uint32_t*>(qr + e1) : 0u;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int pc = nt * 8 + 2 * c + e;
                rp[nt][e] = pc < npair ? p0 + pc / a.group : -1;
            }
        }
        float m[NT][2], l[NT][2], o[KT][NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[t][nt][e] = 0.f;
        }

        int stage = 0;
        for (int i = s0 + warp; i < n_real; i += W) {
            cp_wait<STAGES - 2>();
            __syncwarp();
            {
                const int ns = stage == 0 ? STAGES - 1 : stage - 1;
                if (li < n_real) {
                    load(li, ns, page);
                    li += W;
                    if (li < n_real) page = page_at(li);
                }
                cp_commit();
            }
            const uint32_t kb = ring + stage * S::BYTES, vb = kb + S::KV;
            float s[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
            if constexpr (!I4) {
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    uint32_t k[4];
                    const int t = lane & 15, ch = 2 * kt + (lane >> 4);
                    ldsm4(k, kb + t * S::ROW + ((ch ^ (t & 7)) << 4));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma(s[nt], k, qf[nt][kt][0], qf[nt][kt][1]);
                }
            } else {
                const uint8_t* kp = ring_p + stage * S::BYTES;
                const int t0 = token4(r), t1 = t0 + 8;
                uint32_t w0[G], w1[G];
                float f0[G], f1[G];
                const uint8_t* sp = kp + 2 * S::KV;
                if constexpr (D == 128) {
                    const uint4 u0 = *reinterpret_cast<const uint4*>(kp + t0 * S::ROW + c * 16);
                    const uint4 u1 = *reinterpret_cast<const uint4*>(kp + t1 * S::ROW + c * 16);
                    w0[0] = u0.x; w0[1] = u0.y; w0[2] = u0.z; w0[3] = u0.w;
                    w1[0] = u1.x; w1[1] = u1.y; w1[2] = u1.z; w1[3] = u1.w;
                    const uint2 a0 = *reinterpret_cast<const uint2*>(sp + t0 * 8), a1 = *reinterpret_cast<const uint2*>(sp + t1 * 8);
                    f0[0] = __uint_as_float(a0.x << 16); f0[1] = __uint_as_float(a0.x & 0xffff0000u);
                    f0[2] = __uint_as_float(a0.y << 16); f0[3] = __uint_as_float(a0.y & 0xffff0000u);
                    f1[0] = __uint_as_float(a1.x << 16); f1[1] = __uint_as_float(a1.x & 0xffff0000u);
                    f1[2] = __uint_as_float(a1.y << 16); f1[3] = __uint_as_float(a1.y & 0xffff0000u);
                } else {
                    const uint2 u0 = *reinterpret_cast<const uint2*>(kp + t0 * S::ROW + c * 8);
                    const uint2 u1 = *reinterpret_cast<const uint2*>(kp + t1 * S::ROW + c * 8);
                    w0[0] = u0.x; w0[1] = u0.y;
                    w1[0] = u1.x; w1[1] = u1.y;
                    const uint32_t a0 = *reinterpret_cast<const uint32_t*>(sp + t0 * 4), a1 = *reinterpret_cast<const uint32_t*>(sp + t1 * 4);
                    f0[0] = __uint_as_float(a0 << 16); f0[1] = __uint_as_float(a0 & 0xffff0000u);
                    f1[0] = __uint_as_float(a1 << 16); f1[1] = __uint_as_float(a1 & 0xffff0000u);
                }
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const uint32_t ka[4] = {codes2(w0[g], 0), codes2(w1[g], 0), codes2(w0[g], 1), codes2(w1[g], 1)};
                    const uint32_t kc[4] = {codes2(w0[g], 2), codes2(w1[g], 2), codes2(w0[g], 3), codes2(w1[g], 3)};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float d[4] = {0.f, 0.f, 0.f, 0.f};
                        mma(d, ka, qf[nt][2 * g][0], qf[nt][2 * g][1]);
                        mma(d, kc, qf[nt][2 * g + 1][0], qf[nt][2 * g + 1][1]);
                        s[nt][0] = fmaf(d[0], f0[g], s[nt][0]);
                        s[nt][1] = fmaf(d[1], f0[g], s[nt][1]);
                        s[nt][2] = fmaf(d[2], f1[g], s[nt][2]);
                        s[nt][3] = fmaf(d[3], f1[g], s[nt][3]);
                    }
                }
            }
            // ---- mask (steps at an edge), running maximum, P
            const int j0 = kr.block(i) * PAGED_STEP;
            const int ja = j0 + (I4 ? token4(r) : r), jb = ja + 8;
            if (!all_see(j0, j0 + PAGED_STEP - 1, p0, p1, a.window, a.n_sink)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (!sees(ja, rp[nt][e], a.window, a.n_sink)) s[nt][e] = -INFINITY;
                        if (!sees(jb, rp[nt][e], a.window, a.n_sink)) s[nt][2 + e] = -INFINITY;
                    }
            }
            bool need = false;
            float mx[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float v = fmaxf(s[nt][e], s[nt][2 + e]);
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                    mx[nt][e] = v * a.scale_log2;
                    need = need || mx[nt][e] > m[nt][e] + 8.f;
                }
            if (__any_sync(0xffffffffu, need)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (!(mx[nt][e] > m[nt][e] + 8.f)) continue;
                        const float corr = pow2(m[nt][e] - mx[nt][e]);
                        m[nt][e] = mx[nt][e];
                        l[nt][e] *= corr;
#pragma unroll
                        for (int t = 0; t < KT; ++t) {
                            o[t][nt][e] *= corr;
                            o[t][nt][2 + e] *= corr;
                        }
                    }
            }
            uint32_t pb[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float pv[4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float ref = m[nt][e] == -INFINITY ? 0.f : m[nt][e];
                    pv[e] = pow2(fmaf(s[nt][e], a.scale_log2, -ref));
                    pv[2 + e] = pow2(fmaf(s[nt][2 + e], a.scale_log2, -ref));
                    l[nt][e] += pv[e] + pv[2 + e];
                }
                pb[nt][0] = transpose8(pack2(pv[0], pv[1]));
                pb[nt][1] = transpose8(pack2(pv[2], pv[3]));
            }
            if constexpr (!I4) {
#pragma unroll
                for (int t = 0; t < KT; ++t) {
                    uint32_t v[4];
                    const int tok = ((lane >> 4) << 3) + (lane & 7), ch = 2 * t + ((lane >> 3) & 1);
                    ldsm4t(v, vb + tok * S::ROW + ((ch ^ (tok & 7)) << 4));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma(o[t][nt], v, pb[nt][0], pb[nt][1]);
                }
            } else {
                const uint8_t* vp = ring_p + stage * S::BYTES + S::KV;
                const uint8_t* sp = vp + S::KV + PAGED_STEP * S::SCALE;
                // tokens of columns 2c, 2c + 1, 2c + 8, 2c + 9 of V^T
                const int tk[4] = {c, 4 + (c ^ 1), 8 + c, 12 + (c ^ 1)};
                uint32_t v[4][G / 2], f[4][G / 2];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if constexpr (D == 128) {
                        const uint2 w = *reinterpret_cast<const uint2*>(
                            vp + tk[u] * S::ROW + (((r >> 1) ^ (((tk[u] >> 1) & 1) << 1)) << 4) + ((r & 1) << 3));
                        const uint2 g = *reinterpret_cast<const uint2*>(sp + tk[u] * 8);
                        v[u][0] = w.x; v[u][1] = w.y;
                        f[u][0] = g.x; f[u][1] = g.y;
                    } else {
                        v[u][0] = *reinterpret_cast<const uint32_t*>(vp + tk[u] * S::ROW + (r << 2));
                        f[u][0] = *reinterpret_cast<const uint32_t*>(sp + tk[u] * 4);
                    }
                }
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const uint32_t sel = (g & 1) ? 0x7632 : 0x5410;  // the 16-bit half of group g
                    const uint32_t x01 = __byte_perm(v[0][g >> 1], v[1][g >> 1], sel);
                    const uint32_t x23 = __byte_perm(v[2][g >> 1], v[3][g >> 1], sel);
                    const uint32_t f01 = __byte_perm(f[0][g >> 1], f[1][g >> 1], sel);
                    const uint32_t f23 = __byte_perm(f[2][g >> 1], f[3][g >> 1], sel);
                    const uint32_t va[4] = {codes2(x01, 0), codes2(x01, 1), codes2(x23, 0), codes2(x23, 1)};
                    const uint32_t vc[4] = {codes2(x01, 2), codes2(x01, 3), codes2(x23, 2), codes2(x23, 3)};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint32_t b0 = mul2(pb[nt][0], f01), b1 = mul2(pb[nt][1], f23);
                        mma(o[2 * g][nt], va, b0, b1);
                        mma(o[2 * g + 1][nt], vc, b0, b1);
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
            sL[tid] = sum;
        }
        __syncthreads();
        const bool whole_item = s0 == 0 && s1 == steps;
        const int first = item0 / quota, n_part = (item0 + steps - 1) / quota - first + 1;
        float* slot = a.part + (size_t)(2 * blockIdx.x + (s0 == 0 ? 1 : 0)) * paged_slot_floats(D);
        bf16* out = reinterpret_cast<bf16*>(a.out);
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
                const long long row = si.row0 + p / a.group;
                *reinterpret_cast<uint32_t*>(out + (row * a.hq + head * a.group + p % a.group) * D + e) = pack2(y0 * inv, y1 * inv);
            } else {
                *reinterpret_cast<float2*>(slot + p * D + e) = make_float2(y0, y1);
            }
        }
        if (!whole_item) {
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
                // part k is CTA first + k's: its slot 1 when the item starts there, else slot 0
                const size_t sf = paged_slot_floats(D);
                const float* base = a.part + (size_t)2 * first * sf;
                auto part = [&](int k) { return base + (size_t)(2 * k + (k == 0 ? 1 : 0)) * sf; };
                float* wt = so;  // weights of the parts of one pair
                for (int p = 0; p < npair; ++p) {
                    float mx = -INFINITY;
                    for (int k = 0; k < n_part; ++k) mx = max_nan(mx, __ldcg(part(k) + PAGED_MAX_TILE * D + p));
                    const float ref = mx == -INFINITY ? 0.f : mx;
                    for (int k = tid; k < n_part; k += T) wt[k] = pow2(__ldcg(part(k) + PAGED_MAX_TILE * D + p) - ref);
                    __syncthreads();
                    float sum = 0.f;
                    for (int k = 0; k < n_part; ++k) sum += wt[k] * __ldcg(part(k) + PAGED_MAX_TILE * (D + 1) + p);
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;
                    for (int e = 2 * tid; e < D; e += 2 * T) {
                        float y0 = 0.f, y1 = 0.f;
#pragma unroll 4
                        for (int k = 0; k < n_part; ++k) {
                            const float2 v = __ldcg(reinterpret_cast<const float2*>(part(k) + p * D + e));
                            y0 = fmaf(v.x, wt[k], y0);
                            y1 = fmaf(v.y, wt[k], y1);
                        }
                        const long long row = si.row0 + p / a.group;
                        *reinterpret_cast<uint32_t*>(out + (row * a.hq + head * a.group + p % a.group) * D + e) =
                            pack2(y0 * inv, y1 * inv);
                    }
                    __syncthreads();
                }
            }
        }
        __syncthreads();  // the ring is loaded again for the next segment
        x += s1 - s0;
    }
}

template <bool I4, int D, int NT, int W, int STAGES> void launch_one(const PagedAttn& a, cudaStream_t s) {
    using Cfg = SplitCfg<I4, D, NT, W, STAGES>;
    auto kern = k_paged_split<I4, D, NT, W, STAGES>;
    static const bool ready = [&] {
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM);
        return true;
    }();
    (void)ready;
    kern<<<304, W * 32, Cfg::SMEM, s>>>(a);  // two CTAs on each of 152 SMs
    note_launch(1);
}
template <bool I4, int D> void launch_nt(const PagedAttn& a, cudaStream_t s) {
    const int pairs = a.max_q * a.group;
    constexpr int W1 = I4 ? 8 : 4, ST = I4 ? 5 : 3;
    if (pairs <= 8) launch_one<I4, D, 1, W1, ST>(a, s);
    else if (pairs <= 16) launch_one<I4, D, 2, 4, ST>(a, s);
    else launch_one<I4, D, 4, 4, ST>(a, s);
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

// Attention of prompt pieces over a paged cache (paged_attention in blend.h), bf16 models: tcgen05
// on CTA pairs, after the prefill's k_attn_pair.
//
// A tile is the 128 / group rows (times the group) of one kv head that fill TMEM's 128 lanes; an
// item is two neighbouring tiles of one sequence and kv head, one per CTA of a cluster of two, which
// share every 128-key block.  Per block each CTA stages 64 of the keys (for S) and half of V's
// columns (for P.V); the leading CTA issues M256 products for both.  TMEM holds three S buffers,
// each block's P over its own S, and O: see k_attn_pair for why.
//
// Work: all items' blocks form one line (as in the split kernel) and every cluster takes an equal
// stretch of it, so a few long rows fill the GPU as well as many pieces do and ragged lengths
// leave no tail.  A tile cut by a border leaves its unnormalised O, maximum and sum per row in the
// workspace; each warp owns 32 rows, and the warp that arrives last at them joins the parts in
// order.  Blocks outside every row's window are not visited.
//
// Pages: model pages come by TMA, one box per page and column half (a page of 16 tokens is eight
// boxes a block), 4-bit pages as they are by bulk copies, and four more warps per CTA turn the codes
// into bf16 n s in the swizzled layout the products read.  V rows of tokens that no
// row of the item sees are zeroed (they may hold anything, and 0 x NaN is NaN): by those warps,
// or, in the few blocks at an edge, by the producer warp after the boxes have landed.  Pages without
// a token that the item sees are not touched at all.
// Measured (GB300): four pieces of 2048 rows, window 4096, 32 heads over 8 kv heads x 128, 450-474 us, 1.2
// PFLOP/s (63 % of the library's matrix product): bound by the softmax of a block, about 1750 cycles
// for 128 x 128 scores (tensor pipe 54 %, issue 34 %, DRAM 16 %).
//
// Rounding: P to bf16, once, as in the prefill's attention (a second part would be work of the softmax, which bounds
// the kernel).  4-bit pages: n s has 11 significant bits.  Keys are held as two bf16 parts (of a 64th of n s),
// rounded and the three bits that this leaves, and S takes both (the reduction is twice as long, over the same
// queries).  Values are exact in fp16 where the scales of
// 32 tokens lie within 2^-14..2^6 (or are 0), and those tokens' P is rounded to fp16 too; else both
// are bf16.  The choice is one bit per 32 tokens that the dequantising warp leaves for the softmax
// (both CTAs see the same scales) and for the P.V instruction's descriptor.
// Measured: 64-row pieces of 8 sequences of 6-8 K tokens, against 64 bits relative to the result's norm,
// 1.7e-3, which is the result's own rounding, in 106 us.  (Keys, values and P in bf16: 3.6e-3, 76 us;
// only the keys in one bf16 part: 2.7e-3, 85 us.  Of the 29 us the second part's stores and products
// are 13, three stages instead of five 7, the look at the scales 8.  More run-ahead does not help: a
// ring of the keys' own, free after S, with four stages of values takes 111 us.)
#include <cmath>

#include <cuda_fp16.h>

#include "attn_tc.cuh"
#include "paged.cuh"

namespace blend {
namespace {

constexpr int TQ = 128;    // lanes of a tile
constexpr int TKEYS = 128;  // keys of a block
constexpr int Q_HALF = TQ * 128;    // 64 columns of a Q tile
constexpr int K_HALF = 64 * 128;    // 64 columns of a CTA's 64 keys
constexpr int NSBUF = 3;
constexpr uint32_t O_COL = 384;
constexpr int TMEM_COLS = 512;
// Warps: 0 producer, 1 TMEM + P.V issue, 2..5 softmax, 6 S issue; model pages: 7 edge blocks; 4-bit
// pages: 7..10 codes to operands, and in the second CTA warps 1 and 6 its blocks' signals
constexpr int S_WARP = 6;
constexpr int MAX_CLUSTERS = 76;
constexpr int MIN_QUOTA = 2;  // blocks of a cluster's share at least
constexpr int SNAP = 4;       // an item is not cut within so many blocks of its ends

template <bool I4, int D> struct TileCfg {
    static constexpr int NH = D / 64;
    static constexpr int THREADS = I4 ? 352 : 256;
    static constexpr int VCOL = D / 2;                      // V columns of a CTA
    static constexpr int QT = NH * Q_HALF;
    static constexpr int KB = (I4 ? 2 : 1) * NH * K_HALF;   // 4-bit pages: the keys as bf16, and what that leaves of them
    static constexpr int VB = TKEYS * VCOL * 2;
    static constexpr int STAGE = KB + VB;
    static constexpr int STAGES = D == 64 ? (I4 ? 6 : 8) : I4 ? 3 : 5;
    static constexpr int QB = I4 ? 1 : 2;  // Q buffers: 4-bit pages need the room for stages
    // 4-bit pages: raw rows on their way (this CTA's 64 keys, the 128 values, their scales)
    static constexpr int RAW_STAGES = 2;
    static constexpr int RB = D / 2, SB = D / 16;  // bytes of a row and of its scales
    static constexpr int RAW_V = 64 * RB, RAW_KS = RAW_V + TKEYS * RB, RAW_VS = RAW_KS + 64 * SB;
    static constexpr int RAW = I4 ? RAW_VS + TKEYS * SB : 0;
    static constexpr int SMEM = QB * QT + STAGES * STAGE + RAW_STAGES * RAW + 1024;
    // kind::f16, bf16 inputs, fp32 accumulate, M256 (the pair); S: N128, P.V: N = D with B MN-major
    static constexpr uint32_t IDESC_S = (1u << 4) | (1u << 7) | (1u << 10) | ((128u >> 3) << 17) | ((256u >> 4) << 24);
    static constexpr uint32_t IDESC_PV =
        (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | (((uint32_t)D >> 3) << 17) | ((256u >> 4) << 24);
    static constexpr uint32_t IDESC_PV_F16 = IDESC_PV & ~((1u << 7) | (1u << 10));
    // The exponent that P keeps in hand: fp16 holds P up to 2^15 (the largest sum of a block that is kept
    // without its maximum), and 2^5 above the maximum's own weight keeps 2^-30 of it.
    static constexpr float P_UP = I4 ? 5.f : 0.f;
    static constexpr float SUM_MAX = I4 ? 0x1p15f : 0x1p50f;
    // fp32 partial result of one tile: [D / 4][128 lanes][4], then maxima and sums per lane
    static constexpr size_t PART = (size_t)TQ * (D + 2);
};
static_assert(4 * MAX_CLUSTERS * TileCfg<false, 128>::PART * 4 <= paged_part_bytes(128), "workspace");
static_assert(4 * MAX_CLUSTERS * TileCfg<false, 64>::PART * 4 <= paged_part_bytes(64), "workspace");
static_assert(8 * MAX_CLUSTERS <= PAGED_MAX_CTAS, "arrival counters");
static_assert(2 * MAX_CLUSTERS * (size_t)(BLEND_MAX_SEQS + 1) <= PAGED_PRE_INTS, "prefix sums");

// MN-major B operand (V), a CTA's columns in one swizzle atom: 64 columns (128-byte swizzle, 8-key
// groups 1024 B apart) or 32 (64-byte swizzle, 512 B apart).
template <int D> __device__ __forceinline__ uint64_t desc_v(uint32_t a) {
    const uint64_t group = D == 128 ? 1024 : 512, layout = D == 128 ? 2 : 4;
    return (uint64_t)((a & 0x3FFFF) >> 4) | ((uint64_t)(16384 >> 4) << 16) | ((group >> 4) << 32) | ((uint64_t)1 << 46) |
           (layout << 61);
}
__device__ __forceinline__ void tma_4d_pair(void* dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
        "%4, %5, %6}], [%2];" ::"r"(su32(dst)),
        "l"((uint64_t)m), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}
// `bytes` (a multiple of 16, as both addresses) into this CTA's shared memory
__device__ __forceinline__ void bulk_copy(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(su32(dst)),
                 "l"(src), "r"(bytes), "r"(su32(bar))
                 : "memory");
}
// Arrival on the leader's barrier that publishes this thread's shared-memory writes to the pair.
__device__ __forceinline__ void arrive_leader_release(uint64_t* b) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(leader_addr(b)) : "memory");
}
// Warp-level bounded wait by polling: a blocking try_wait on a barrier that the other CTA's commits
// reach resumes late (see test_cl), which a producer cannot hide.
__device__ __forceinline__ bool warp_poll(uint64_t* b, uint32_t par, volatile int* abort_flag) {
    for (long long i = 0; i < 64 * SPIN_LIMIT; ++i) {
        if (__all_sync(0xffffffffu, test_cl(b, par))) return true;
        if ((i & 1023) == 1023 && __any_sync(0xffffffffu, *abort_flag != 0)) return false;
    }
    return false;
}
__device__ __forceinline__ void arrive_leader(uint64_t* b) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(leader_addr(b)) : "memory");
}
__device__ __forceinline__ bool wait_cl_acquire(uint64_t* b, uint32_t par, volatile int* abort_flag) {
    for (long long i = 0; i < 64 * SPIN_LIMIT; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}\n"
            : "=r"(ok)
            : "r"(su32(b)), "r"(par)
            : "memory");
        if (ok) return true;
        if ((i & 1023) == 1023 && *abort_flag) return false;
    }
    return false;
}
// A block that the second CTA's dequantising warps have written, signalled to the leader: a release to
// the cluster takes over 1000 cycles, so one thread per block does it for four warps (whose arrivals
// at the CTA's own barrier it has seen), and two warps that have nothing else to do take turns.
__device__ __forceinline__ bool pass_on(uint64_t* own, uint64_t* leader, uint32_t par, volatile int* abort_flag) {
    if (!warp_poll(own, par, abort_flag)) return false;
    if ((threadIdx.x & 31) == 0) arrive_leader_release(leader);
    __syncwarp();
    return true;
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ int tiles2(int n_q, int rows2) { return (n_q + rows2 - 1) / rows2; }
// Positions of item tp's rows (two tiles of rows2 rows) and its 128-key blocks; an item that sees
// nothing keeps one block, all masked, which gives its rows their zeros.
struct ItemRange {
    int p_lo, p_hi, n;
    KeyRange kr;
};
__device__ __forceinline__ ItemRange item_range(const PagedAttn& a, const SeqInfo& si, int tp, int rows2) {
    ItemRange r;
    const int first = si.len - si.n_q;
    r.p_lo = first + tp * rows2;
    r.p_hi = first + min(si.n_q, (tp + 1) * rows2) - 1;
    r.kr = key_range<TKEYS>(r.p_lo, r.p_hi, a.window, a.n_sink);
    r.n = max(1, r.kr.total());
    return r;
}

// A cluster's share of the line of blocks, item by item.  Every role walks its own.
struct Walk {
    const PagedAttn& a;
    const int* pre;
    const Shares sh;
    const int rows2, share, total;
    int seq, head, tp, i0;  // i0: first unit of the item
    SeqInfo si;
    ItemRange it;
    int b0, b1;  // this share's blocks of the item
    bool done;

    __device__ __forceinline__ Walk(const PagedAttn& a_, const int* pre_, const Shares& sh_, int rows2_, int share_, int total_)
        : a(a_), pre(pre_), sh(sh_), rows2(rows2_), share(share_), total(total_) {
        const int x = sh.start(share);
        int lo = 0, hi = a.pg.n_seq - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (pre[mid] <= x) lo = mid;
            else hi = mid - 1;
        }
        seq = lo;
        while (pre[seq + 1] <= x) ++seq;
        const int per_head = (pre[seq + 1] - pre[seq]) / a.pg.hkv;
        int rem = x - pre[seq];
        head = rem / per_head;
        rem -= head * per_head;
        si = seq_info(a, seq);
        tp = 0;
        it = item_range(a, si, 0, rows2);
        while (rem >= it.n) {
            rem -= it.n;
            it = item_range(a, si, ++tp, rows2);
        }
        i0 = x - rem;
        done = sh.first(i0, i0 + it.n) > share;
        while (!done && sh.last(i0, i0 + it.n) < share) next();
        if (!done) cut();
    }
    __device__ __forceinline__ void cut() {
        b0 = sh.begin(share, i0, i0 + it.n);
        b1 = sh.end(share, i0, i0 + it.n);
    }
    __device__ __forceinline__ bool more() const { return !done; }
    __device__ __forceinline__ void next() {
        i0 += it.n;
        done = i0 >= total;
        if (done) return;
        if (++tp == tiles2(si.n_q, rows2)) {
            tp = 0;
            if (++head == a.pg.hkv) {
                head = 0;
                do ++seq;
                while (pre[seq + 1] <= i0);
                si = seq_info(a, seq);
            }
        }
        it = item_range(a, si, tp, rows2);
        done = sh.first(i0, i0 + it.n) > share;
        cut();
    }
    __device__ __forceinline__ bool any_seen(int j0, int j1) const {
        return j0 <= it.p_hi && (j0 < a.n_sink || j1 > it.p_lo - a.window);
    }
    __device__ __forceinline__ bool all_seen(int j0, int j1) const {
        return j1 <= it.p_hi && (j1 < a.n_sink || j0 > it.p_lo - a.window);
    }
};

// Blocks of a whole share.
__device__ __forceinline__ int blocks_of(Walk w) {
    int n = 0;
    for (; w.more(); w.next()) n += w.b1 - w.b0;
    return n;
}

// A lane's row of 128 scores in TMEM: those of keys it does not see become -inf.  Seen are keys up to
// `hi` of the block that come after hi - window or before `sink`.
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }  // bits 0..n-1
__device__ __forceinline__ void mask_scores(uint32_t s_col, int hi, int window, int sink) {
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
        const uint32_t bits = below(hi + 1 - 32 * q) & (~below(hi - window + 1 - 32 * q) | below(sink - 32 * q));
        if (__all_sync(0xffffffffu, bits == 0xffffffffu)) continue;
        uint32_t v[32];
        TMEM_LD32(s_col + 32 * q, v);
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (!(bits & (1u << i))) v[i] = __float_as_uint(-INFINITY);
        TMEM_ST32(s_col + 32 * q, v);
    }
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ float row_max(uint32_t s_col) {
    float mx = -INFINITY;
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
        uint32_t v[32];
        TMEM_LD32(s_col + 32 * q, v);
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
        for (int i = 0; i < 32; i += 2) mx = max3f(mx, __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
    }
    return mx;
}

// The values n s of the codes at bits 0..3 and 16..19, rounded once.
__device__ __forceinline__ uint32_t pair_value(uint32_t w, uint32_t scale2) {
    const uint32_t n = code_ints(w);
    const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&n), *reinterpret_cast<__nv_bfloat162*>(&scale2));
    return *reinterpret_cast<const uint32_t*>(&v);
}
// A 64th of the values, which saves shifts (code_pair) and goes into the scores' factor, rounded once, and what
// the rounding leaves (three bits, exactly).
template <bool HI> __device__ __forceinline__ void pair_parts(uint32_t w, uint32_t scale2, uint32_t& value, uint32_t& rest) {
    const uint32_t n = code_pair<HI>(w);
    const __nv_bfloat162 n2 = *reinterpret_cast<const __nv_bfloat162*>(&n), s2 = *reinterpret_cast<__nv_bfloat162*>(&scale2);
    const __nv_bfloat162 v = __hmul2(n2, s2), r = __hfma2(n2, s2, __hneg2(v));
    value = *reinterpret_cast<const uint32_t*>(&v);
    rest = *reinterpret_cast<const uint32_t*>(&r);
}
// One of two bf16 scales, twice.
__device__ __forceinline__ uint32_t both(uint32_t w, int hi) { return __byte_perm(w, w, hi ? 0x3232 : 0x1010); }

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// The same in fp16, exact for scales that fit_f16 lets through: a code in the low bits of 1024 (the
// codes at bits 0 and 16) is 1024 + n + 8.
__device__ __forceinline__ uint32_t pair_f16(uint32_t w, uint32_t scale2) {
    uint32_t x = (w & 0x000F000Fu) | 0x64006400u;
    const uint32_t off = 0x64086408u;
    const __half2 v = __hmul2(__hsub2(*reinterpret_cast<__half2*>(&x), *reinterpret_cast<const __half2*>(&off)),
                              *reinterpret_cast<__half2*>(&scale2));
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t both_f16(uint32_t w, int hi) {
    const float f = __uint_as_float(hi ? w & 0xffff0000u : w << 16);
    return pack_f16x2(f, f);
}
// Both bf16 scales of w are 0 or within 2^-14..2^6: n s is exact in fp16 (2^-17..2^13 would do for
// that), and weights so small that fp16 loses them, under 2^-30 of a row's largest, cannot matter by
// having values that much larger.
__device__ __forceinline__ bool fit_f16(uint32_t w) {
    const uint32_t lo = w & 0xffffu, hi = w >> 16;
    return (lo == 0u || lo - 0x3880u <= 0x0A00u) && (hi == 0u || hi - 0x3880u <= 0x0A00u);
}
constexpr uint32_t ALL_F16 = 0x01010101u;
// P of a block with tokens whose values are bf16, 32 keys at a time from the row's reference (which
// holds the block's maximum): packed over the scores; returns the sum.
__device__ __forceinline__ float mixed_block(uint32_t s_col, uint32_t f16, float scale, float ref) {
    float sum = 0.f;
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
        uint32_t v[32];
        TMEM_LD32(s_col + 32 * q, v);
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
        const bool h = (f16 >> (8 * q)) & 1u;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float p0 = ex2(fmaf(__uint_as_float(v[2 * i]), scale, ref)), p1 = ex2(fmaf(__uint_as_float(v[2 * i + 1]), scale, ref));
            sum += p0 + p1;
            v[i] = h ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
        }
        TMEM_ST16(s_col + 16 * q, v);
    }
    return sum;
}

template <bool I4, int D>
__global__ void __launch_bounds__(TileCfg<I4, D>::THREADS, 1)
    k_paged_tile(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                 const __grid_constant__ CUtensorMap mapV, const __grid_constant__ PagedAttn a, int rpt) {
    using T = TileCfg<I4, D>;
    constexpr int NH = T::NH, STAGES = T::STAGES, STAGE = T::STAGE, QT = T::QT, KB = T::KB, VCOL = T::VCOL;
    constexpr int WARPS = T::THREADS / 32;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t q_full[2], q_empty[2], kv_full[STAGES], kv_empty[STAGES], s_full[NSBUF],
        p_full[NSBUF], o_full, o_free, edge_full[STAGES], own_full[STAGES],
        raw_full[T::RAW_STAGES], raw_empty[T::RAW_STAGES];
    __shared__ uint32_t tmem_sh;
    __shared__ volatile int abort_flag;
    __shared__ int pend_kv[STAGES], pend_q[2], pend_edge[STAGES], pend_raw[T::RAW_STAGES];
    __shared__ uint32_t v_f16[STAGES];  // 4-bit pages: byte q is 1 where tokens 32 q .. +31 of the stage are fp16
    __shared__ int3 raw_at[T::RAW_STAGES];  // first key of a raw block, positions of its item's first and last row
    // in the workspace (shared memory is full of stages); read again only where a role changes sequence
    int* pre = a.pre + (size_t)blockIdx.x * (BLEND_MAX_SEQS + 1);

    uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t* sQ = smem;              // Q buffer qb at qb * QT
    uint8_t* sKV = smem + T::QB * QT;    // stage s at s * STAGE: K column halves, V
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = (int)cta_rank();
    const int grp = (int)(blockIdx.x >> 1), n_grp = (int)(gridDim.x >> 1);
    const int rows2 = 2 * rpt, group = a.group, n_seq = a.pg.n_seq;

    // ---- the line of blocks: pre[s] = blocks of all items of sequences before s
    for (int s = warp; s < n_seq; s += WARPS) {
        const SeqInfo si = seq_info(a, s);
        int n = 0;
        if (si.n_q * group > a.short_pairs)  // the others are the split kernel's
            for (int tp = lane; tp < tiles2(si.n_q, rows2); tp += 32) n += item_range(a, si, tp, rows2).n;
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) pre[s + 1] = n * a.pg.hkv;
    }
    __syncthreads();
    if (warp == 0) {
        int base = 0;
        for (int s0 = 0; s0 < n_seq; s0 += 32) {
            const int s = s0 + lane;
            int v = s < n_seq ? pre[s + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v = add_capped(v, y, PAGED_MAX_UNITS);
            }
            v = add_capped(v, base, PAGED_MAX_UNITS);
            if (s < n_seq) pre[s + 1] = v;
            base = __shfl_sync(0xffffffffu, v, 31);
        }
        if (lane == 0) pre[0] = 0;
    }
    __syncthreads();
    const int total = pre[n_seq];
    if (total == 0) return;  // both CTAs of the cluster
    if (total == PAGED_MAX_UNITS) {  // sequences that claim the same rows again and again
        if (threadIdx.x == 0) set_error(a.err, BLEND_EDEVICE);
        return;
    }
    const int quota = max(MIN_QUOTA, Shares::parts(total, n_grp));
    const Shares sh(total, quota, min(SNAP, quota));
    if (grp >= sh.n) return;

    // Lanes of a tile past its rows read a Q of zeros
    for (int i = threadIdx.x; i < T::QB * QT / 16; i += T::THREADS) reinterpret_cast<uint4*>(sQ)[i] = make_uint4(0, 0, 0, 0);
    fence_async_smem();
    if (threadIdx.x == 0) {
        for (int b = 0; b < 2; ++b) {
            mbar_init(&q_full[b], 1);
            mbar_init(&q_empty[b], 1);
            pend_q[b] = -1;
        }
        for (int b = 0; b < NSBUF; ++b) {
            mbar_init(&s_full[b], 1);
            mbar_init(&p_full[b], 8);  // 4 softmax warps in each CTA
        }
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&kv_full[s], I4 ? 5 : 2);  // once from each CTA; 4-bit: the leader's four warps and the other CTA
            mbar_init(&edge_full[s], 1);
            pend_edge[s] = -1;
            mbar_init(&own_full[s], 4);  // 4-bit pages: this CTA's dequantising warps
            mbar_init(&kv_empty[s], 1);
            pend_kv[s] = -1;
        }
        for (int s = 0; s < T::RAW_STAGES; ++s) {
            mbar_init(&raw_full[s], 1);
            mbar_init(&raw_empty[s], 4);
            pend_raw[s] = -1;
        }
        mbar_init(&o_full, 1);
        mbar_init(&o_free, 8);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&tmem_sh)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before either signals the other's
    fence_after();
    const uint32_t tb = tmem_sh;

    if (warp == 0) {
        // ------------------------------------------------ producer warp (both CTAs): Q, model pages
        // Lane i owns one copy of every block: boxes of the CTA's 64 keys by pages and column halves, then
        // of the 128 keys' V columns by pages; or for 4-bit pages the key rows by pages, their scales, the
        // value rows, their scales.  The page of its next copy is read a block ahead.
        const int k_rows = min(1 << a.pg.shift, 64), v_rows = 1 << a.pg.shift;
        const int n_k = 64 / k_rows * (I4 ? 2 : NH), n_v = TKEYS / v_rows * (I4 ? 2 : 1);
        const bool is_k = lane < n_k, mine = lane < n_k + n_v;
        const int nth = is_k ? lane : lane - n_k;                       // of the keys' or the values' copies
        const int pieces = is_k ? 64 / k_rows : TKEYS / v_rows;
        const int piece = !I4 ? (is_k ? nth / NH : nth) : nth % pieces;
        const bool scale = I4 && nth >= pieces;
        const int rows = is_k ? k_rows : v_rows;
        const int tok = is_k ? 64 * rank + piece * k_rows : piece * v_rows;  // first token of the copy in a block
        const int col = is_k ? (nth % NH) * 64 : VCOL * rank;
        const int width = scale ? T::SB : T::RB;                        // 4-bit: bytes of a row
        const int box_at = !I4 ? (is_k ? (nth % NH) * K_HALF + piece * k_rows * 128 : KB + tok * VCOL * 2)
                               : (is_k ? (scale ? T::RAW_KS : 0) : (scale ? T::RAW_VS : T::RAW_V)) + piece * rows * width;
        const char* src = is_k ? (scale ? a.pg.ks : a.pg.k) : (scale ? a.pg.vs : a.pg.v);
        const int page_mask = (1 << a.pg.shift) - 1;
        uint32_t it = 0;
        bool ok = true;
        int tl = 0, page = 0, k0 = 0;
        bool need = false, edge = false;
        Walk w(a, pre, sh, rows2, grp, total);
        int b = w.more() ? w.b0 : 0;
        auto look = [&]() {  // this lane's box of block b: whether a row sees any of it, and its page
            k0 = w.it.kr.block(b) * TKEYS;
            edge = !w.all_seen(k0, k0 + TKEYS - 1);
            need = mine && w.any_seen(k0 + tok, k0 + tok + rows - 1);
            if (need) page = page_entry(a.pg, w.seq, k0 + tok);  // looked at when the stage is free
        };
        if (w.more()) look();
        while (ok && w.more()) {
            if (b == w.b0) {
                const int qb = tl % T::QB;
                ok = warp_poll(&q_empty[qb], ((tl / T::QB) & 1) ^ 1, &abort_flag);
                if (!ok) break;
                if (lane == 0) {
                    if (rank == 0) {
                        mbar_expect_tx(&q_full[qb], 2u * NH * 128u * (uint32_t)(group * rpt));  // both CTAs' tiles
                        pend_q[qb] = (tl / T::QB) & 1;
                    }
                    // an absent second tile reloads the first (finite data, never stored)
                    const int t_row = w.tp * rows2 + rank * rpt;
                    const int row = w.si.row0 + (t_row < w.si.n_q ? t_row : w.tp * rows2);
                    const uint32_t qf = leader_addr(&q_full[qb]);
#pragma unroll
                    for (int hh = 0; hh < NH; ++hh) tma_4d_pair(sQ + qb * QT + hh * Q_HALF, &mapQ, qf, hh * 64, 0, w.head, row);
                }
                __syncwarp();
                ++tl;
            }
            const int st = it % STAGES;
            if constexpr (I4) {
                const int rs = it % T::RAW_STAGES;
                ok = warp_poll(&raw_empty[rs], ((it / T::RAW_STAGES) & 1) ^ 1, &abort_flag);
                if (!ok) break;
                const uint32_t bytes = __reduce_add_sync(0xffffffffu, need ? (unsigned)(rows * width) : 0u);
                if (lane == 0) {
                    raw_at[rs] = make_int3(k0, w.it.p_lo, w.it.p_hi);
                    pend_raw[rs] = (int)((it / T::RAW_STAGES) & 1);
                    mbar_expect_tx(&raw_full[rs], bytes);
                }
                __syncwarp();
                if (need) {
                    const int pg = checked_page(a.pg, page, a.err);
                    bulk_copy(sKV + STAGES * STAGE + rs * T::RAW + box_at,
                              src + page_row(a.pg, pg, w.head, (k0 + tok) & page_mask) * width, (uint32_t)(rows * width), &raw_full[rs]);
                }
                __syncwarp();
            } else {
                ok = warp_poll(&kv_empty[st], ((it / STAGES) & 1) ^ 1, &abort_flag);
                if (!ok) break;
                uint8_t* dst = sKV + st * STAGE;
                if (lane == 0) {
                    if (rank == 0) pend_kv[st] = (int)((it / STAGES) & 1);
                    // a whole block: the leader expects both CTAs' boxes, the other CTA has nothing of its own
                    // to publish; an edge block is signalled by the edge warp, which first waits for V
                    if (!edge) {
                        if (rank == 0) mbar_expect_tx(&kv_full[st], 2u * (KB + T::VB));
                        else arrive_leader(&kv_full[st]);
                    }
                }
                if (edge) {
                    const unsigned v_seen = __ballot_sync(0xffffffffu, need && !is_k);
                    if (lane == 0 && v_seen) {
                        mbar_expect_tx(&edge_full[st], (uint32_t)__popc(v_seen) * (uint32_t)v_rows * VCOL * 2);
                        pend_edge[st] = 1;
                    }
                    __syncwarp();
                }
                if (need) {
                    const int pg = checked_page(a.pg, page, a.err);
                    const int c1 = (k0 + tok) & page_mask, c2 = pg * a.pg.hkv + w.head;
                    if (is_k) tma_3d_pair(dst + box_at, &mapK, leader_addr(&kv_full[st]), col, c1, c2);
                    else if (!edge) tma_3d_pair(dst + box_at, &mapV, leader_addr(&kv_full[st]), col, c1, c2);
                    else tma_3d(dst + box_at, &mapV, &edge_full[st], col, c1, c2);
                }
                __syncwarp();
            }
            ++it;
            if (++b == w.b1) {
                w.next();
                if (!w.more()) break;
                b = w.b0;
            }
            look();
        }
        if (!ok) {
            abort_flag = 1;
            if (lane == 0) set_error(a.err, BLEND_ETIMEOUT);
        }
    } else if (I4 && rank == 1 && (warp == 1 || warp == S_WARP)) {
        // ------------------------------------------------ the second CTA's blocks, signalled to the leader
        bool ok = true;
        const int n_blocks = blocks_of(Walk(a, pre, sh, rows2, grp, total));
        for (int i = warp == 1 ? 0 : 1; ok && i < n_blocks; i += 2)
            ok = pass_on(&own_full[i % STAGES], &kv_full[i % STAGES], (i / STAGES) & 1, &abort_flag);
        if (!ok) {
            abort_flag = 1;
            if (lane == 0) set_error(a.err, BLEND_ETIMEOUT);
        }
    } else if (warp == S_WARP && lane == 0 && rank == 0) {
        // ------------------------------------------------ S issuer (leader, for both CTAs)
        uint32_t it = 0;
        bool ok = true;
        int tl = 0;
        for (Walk w(a, pre, sh, rows2, grp, total); ok && w.more(); w.next(), ++tl) {
            const int qb = tl % T::QB;
            if (!wait_cl(&q_full[qb], (tl / T::QB) & 1, &abort_flag)) {
                ok = false;
                break;
            }
            pend_q[qb] = -1;
            const uint64_t qd = desc_k(su32(sQ + qb * QT));
            for (int b = w.b0; b < w.b1; ++b, ++it) {
                const int sb = it % NSBUF, st = it % STAGES;
                const uint32_t pv = it - NSBUF;  // the P.V that last read this buffer
                if ((it >= NSBUF && !wait_cl(&kv_empty[pv % STAGES], (pv / STAGES) & 1, &abort_flag)) ||
                    !wait_cl_acquire(&kv_full[st], (it / STAGES) & 1, &abort_flag)) {
                    ok = false;
                    break;
                }
                pend_kv[st] = -1;
                fence_after();
                const uint64_t kd = desc_k(su32(sKV + st * STAGE));
#pragma unroll
                for (int kk = 0; kk < (I4 ? 2 : 1) * D / 16; ++kk) {  // 4-bit pages: twice, with both parts of the keys
                    const uint32_t off = (kk & 3) * 32, half = kk >> 2;
                    umma_ss2(tb + sb * 128, qd + (((half % NH) * Q_HALF + off) >> 4), kd + ((half * K_HALF + off) >> 4),
                             T::IDESC_S, kk > 0 ? 1u : 0u);
                }
                commit2(&s_full[sb]);
            }
            if (!ok) break;
            commit2(&q_empty[qb]);
        }
        if (!ok) {
            abort_flag = 1;
            set_error(a.err, BLEND_ETIMEOUT);
        }
    } else if (warp == 1 && lane == 0 && rank == 0) {
        // ------------------------------------------------ P.V issuer (leader, for both CTAs)
        uint32_t it = 0;
        bool ok = true;
        int tl = 0;
        for (Walk w(a, pre, sh, rows2, grp, total); ok && w.more(); w.next(), ++tl) {
            for (int b = w.b0; b < w.b1; ++b, ++it) {
                const int sb = it % NSBUF, st = it % STAGES;
                if (!wait_cl(&p_full[sb], (it / NSBUF) & 1, &abort_flag) ||
                    (b == w.b0 && !wait_cl(&o_free, (tl & 1) ^ 1, &abort_flag))) {
                    ok = false;
                    break;
                }
                fence_after();
                const uint64_t vd = desc_v<D>(su32(sKV + st * STAGE + KB));
                const uint32_t pa = tb + sb * 128;
                const uint32_t f16 = I4 ? *(volatile uint32_t*)&v_f16[st] : 0u;
#pragma unroll
                for (int kk = 0; kk < TKEYS / 16; ++kk)
                    umma_ts2(tb + O_COL, pa + kk * 8, vd + ((kk * 16 * VCOL * 2) >> 4),
                             I4 && ((f16 >> (8 * (kk / 2))) & 1u) ? T::IDESC_PV_F16 : T::IDESC_PV, (b > w.b0 || kk > 0) ? 1u : 0u);
                commit2(&kv_empty[st]);
            }
            if (!ok) break;
            commit2(&o_full);
        }
        if (!ok) {
            abort_flag = 1;
            set_error(a.err, BLEND_ETIMEOUT);
        }
    } else if (warp >= 2 && warp < S_WARP) {
        // ------------------------------------------------ softmax of this CTA's tile + output
        const int sp = warp & 3;  // TMEM lane quarter of this warp
        const int r_in = sp * 32 + lane;
        const uint32_t lane_off = (uint32_t)(sp * 32) << 16;
        const uint32_t o_col = tb + lane_off + O_COL;
        const float scale = I4 ? a.scale_log2 * CODE_UNIT : a.scale_log2;
        const float2 sc2 = make_float2(scale, scale);
        bf16* out = reinterpret_cast<bf16*>(a.out);
        uint32_t it = 0;
        bool ok = true;
        int tl = 0;
        for (Walk w(a, pre, sh, rows2, grp, total); ok && w.more(); w.next(), ++tl) {
            const int t_row = w.tp * rows2 + rank * rpt;            // first row of this CTA's tile
            const int rows = min(rpt, w.si.n_q - t_row);            // <= 0: the tile is absent
            const bool valid = r_in < rows * group;
            const int row = t_row + (valid ? r_in / group : 0);
            const int first = w.si.len - w.si.n_q;
            const int t_lo = first + t_row, t_hi = t_lo + max(rows, 1) - 1;
            const int my_pos = valid ? first + row : t_lo;
            // lanes without a row never hold up their warp: a reference of 0 keeps them off the exact path
            float m_used = valid && my_pos >= 0 ? -INFINITY : 0.f, l = 0.f;
            for (int b = w.b0; b < w.b1; ++b, ++it) {
                const int sb = it % NSBUF;
                const uint32_t s_col = tb + lane_off + sb * 128;
                if (!warp_wait_cl(&s_full[sb], (it / NSBUF) & 1, &abort_flag)) {
                    ok = false;
                    break;
                }
                fence_after();
                const int k0 = w.it.kr.block(b) * TKEYS;
                const bool cut = !all_see(k0, k0 + TKEYS - 1, t_lo, t_hi, a.window, a.n_sink);
                if (cut) mask_scores(s_col, my_pos - k0, a.window, a.n_sink - k0);
                const uint32_t f16 = I4 ? *(volatile uint32_t*)&v_f16[it % STAGES] : ALL_F16;
                uint32_t s[128];
                float2 accs;
                bool rescale = false;
                float corr = 1.f;
                // as in k_attn_pair: without this block's maximum while its sum stays below 2^50.  What few
                // blocks need (masks, the maximum) works on TMEM in small loops, so that the path of the
                // others is short and straight (masks and maximum on the 128 registers, unrolled, put
                // some 15 KB of instructions into the middle of it: 468 instead of 457 us for four
                // prompt pieces of 2048 rows, window 4096, and 220 bytes of spills with 4-bit pages).
                auto raise = [&]() {
                    const float mxs = row_max(s_col) * scale;
                    const bool need = mxs > m_used + RESCALE_LOG2;
                    rescale = __any_sync(0xffffffffu, need);
                    if (rescale) {
                        const float m_new = need ? mxs - T::P_UP : m_used;
                        corr = need ? ex2(m_used - m_new) : 1.f;
                        l *= corr;
                        m_used = m_new;
                    }
                };
                const bool mixed = I4 && f16 != ALL_F16;
                if (mixed) {
                    raise();
                    accs = make_float2(mixed_block(s_col, f16, scale, m_used == -INFINITY ? 0.f : -m_used), 0.f);
                }
                bool exact = !__all_sync(0xffffffffu, m_used != -INFINITY);
#pragma unroll 1
                while (!mixed) {
                    if (exact) raise();
                    const float ref = m_used == -INFINITY ? 0.f : -m_used;
                    TMEM_LD32(s_col, s);
                    TMEM_LD32(s_col + 32, (s + 32));
                    TMEM_LD32(s_col + 64, (s + 64));
                    TMEM_LD32(s_col + 96, (s + 96));
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                    float2 acc2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    const float2 nm2 = make_float2(ref, ref);
#pragma unroll
                    for (int e = 0; e < 64; ++e) {
                        const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), sc2, nm2);
                        const float p0 = ex2(x.x), p1 = ex2(x.y);
                        acc2[e & 1] = __fadd2_rn(acc2[e & 1], make_float2(p0, p1));
                        s[e] = I4 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
                    }
                    accs = __fadd2_rn(acc2[0], acc2[1]);
                    if (exact || !__any_sync(0xffffffffu, !(accs.x + accs.y <= T::SUM_MAX))) break;
                    exact = true;  // P is not stored yet: once more, from the block's maximum
                }
                if (!mixed) {
                    TMEM_ST32(s_col, s);
                    TMEM_ST32(s_col + 32, (s + 32));
                }
                if (rescale && b > w.b0) {
                    const uint32_t pv = it - 1;  // O must hold every block before this one
                    if (!warp_wait_cl(&kv_empty[pv % STAGES], (pv / STAGES) & 1, &abort_flag)) {
                        ok = false;
                        break;
                    }
                    fence_after();
#pragma unroll 1
                    for (int e = 0; e < D; e += 32) {
                        uint32_t o[32];
                        TMEM_LD32(o_col + e, o);
                        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * corr);
                        TMEM_ST32(o_col + e, o);
                    }
                }
                l += accs.x + accs.y;
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                fence_before();
                warp_arrive_leader(&p_full[sb], rank);
            }
            if (!ok) break;
            if (!warp_wait_cl(&o_full, tl & 1, &abort_flag)) {
                ok = false;
                break;
            }
            fence_after();
            const bool whole = w.b0 == 0 && w.b1 == w.it.n;
            bf16* dst = out + ((long long)(w.si.row0 + row) * a.hq + w.head * group + (valid ? r_in % group : 0)) * D;
            if (whole) {
                const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
                for (int e = 0; e < D; e += 32) {
                    uint32_t o[32];
                    TMEM_LD32(o_col + e, o);
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                    if (valid) {
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            uint32_t w4[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                w4[i] = pack_bf16x2(__uint_as_float(o[v * 8 + 2 * i]) * inv,
                                                    __uint_as_float(o[v * 8 + 2 * i + 1]) * inv);
                            *reinterpret_cast<uint4*>(dst + e + v * 8) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
                        }
                    }
                }
                fence_before();
                warp_arrive_leader(&o_free, rank);
                continue;
            }
            // ---- part of an item: leave it, and join the parts of these 32 rows when last to arrive
            const int g_first = sh.first(w.i0, w.i0 + w.it.n), n_part = sh.last(w.i0, w.i0 + w.it.n) - g_first + 1;
            auto slot = [&](int g, int which) { return a.part + (size_t)((2 * g + which) * 2 + rank) * T::PART; };
            float* mine = slot(grp, w.b0 == 0 ? 1 : 0);
#pragma unroll
            for (int e = 0; e < D; e += 32) {
                uint32_t o[32];
                TMEM_LD32(o_col + e, o);
                asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                for (int v = 0; v < 8; ++v)
                    *reinterpret_cast<uint4*>(mine + (size_t)((e / 4 + v) * TQ + r_in) * 4) =
                        make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
            }
            mine[TQ * D + r_in] = m_used;
            mine[TQ * (D + 1) + r_in] = l;
            fence_before();
            warp_arrive_leader(&o_free, rank);  // O may be written again
            __threadfence();
            __syncwarp();
            int last = 0;
            int32_t* count = a.count + (g_first * 2 + rank) * 4 + sp;
            if (lane == 0) {
                last = atomicAdd(count, 1) == n_part - 1;
                if (last) *count = 0;  // ready for the next launch
            }
            last = __shfl_sync(0xffffffffu, last, 0);
            if (!last) continue;
            __threadfence();
            // part k lies with cluster g_first + k: in its slot 1 when the item starts there, else in slot 0
            float mx = -INFINITY, sum = 0.f;
#pragma unroll 4
            for (int k = 0; k < n_part; ++k) mx = max_nan(mx, __ldcg(slot(g_first + k, k == 0) + TQ * D + r_in));
            const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll 4
            for (int k = 0; k < n_part; ++k) {
                const float* p = slot(g_first + k, k == 0);
                sum += __ldcg(p + TQ * (D + 1) + r_in) * ex2(__ldcg(p + TQ * D + r_in) - ref);
            }
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            // 64 columns at a time, 16 loads on their way together
#pragma unroll 1
            for (int e = 0; e < D; e += 64) {
                float acc[64];
#pragma unroll
                for (int i = 0; i < 64; ++i) acc[i] = 0.f;
#pragma unroll 1
                for (int k = 0; k < n_part; ++k) {
                    const float* p = slot(g_first + k, k == 0);
                    const float f = ex2(__ldcg(p + TQ * D + r_in) - ref) * inv;
                    const float4* q = reinterpret_cast<const float4*>(p) + (e / 4) * TQ + r_in;
                    float4 v[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = __ldcg(q + i * TQ);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        acc[4 * i] = fmaf(v[i].x, f, acc[4 * i]);
                        acc[4 * i + 1] = fmaf(v[i].y, f, acc[4 * i + 1]);
                        acc[4 * i + 2] = fmaf(v[i].z, f, acc[4 * i + 2]);
                        acc[4 * i + 3] = fmaf(v[i].w, f, acc[4 * i + 3]);
                    }
                }
                if (valid) {
#pragma unroll
                    for (int v = 0; v < 8; ++v) {
                        uint32_t w4[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) w4[i] = pack_bf16x2(acc[v * 8 + 2 * i], acc[v * 8 + 2 * i + 1]);
                        *reinterpret_cast<uint4*>(dst + e + v * 8) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
                    }
                }
            }
        }
        if (!ok) {
            abort_flag = 1;
            if (lane == 0) set_error(a.err, BLEND_ETIMEOUT);
        }
    } else if (!I4 && warp > S_WARP) {
        // ------------------------------------------------ edge blocks of model pages (both CTAs)
        // V has its own barrier here; rows that no row sees are zeroed once it has landed, then the
        // block is signalled: the leader's own arrival carries the bytes of both CTAs' keys.
        const int k_rows = min(1 << a.pg.shift, 64), v_rows = 1 << a.pg.shift;
        uint32_t it = 0, phases = 0;  // phases: bit st, the parity of edge_full[st]
        bool ok = true;
        for (Walk w(a, pre, sh, rows2, grp, total); ok && w.more(); w.next())
            for (int b = w.b0; b < w.b1; ++b, ++it) {
                const int k0 = w.it.kr.block(b) * TKEYS;
                if (w.all_seen(k0, k0 + TKEYS - 1)) continue;
                const int st = it % STAGES;
                // the stage must be this block's before anything is written to it
                ok = warp_poll(&kv_empty[st], ((it / STAGES) & 1) ^ 1, &abort_flag);
                if (!ok) break;
                const unsigned k_seen = __ballot_sync(0xffffffffu, lane * k_rows < TKEYS && w.any_seen(k0 + lane * k_rows, k0 + (lane + 1) * k_rows - 1));
                const unsigned v_seen = __ballot_sync(0xffffffffu, lane * v_rows < TKEYS && w.any_seen(k0 + lane * v_rows, k0 + (lane + 1) * v_rows - 1));
                if (v_seen) {
                    ok = warp_poll(&edge_full[st], (phases >> st) & 1, &abort_flag);
                    if (!ok) break;
                    if (lane == 0) pend_edge[st] = -1;
                    phases ^= 1u << st;
                }
                uint8_t* dst = sKV + st * STAGE + KB;
                constexpr int CH = VCOL / 8;  // 16-byte chunks of a row (the swizzle stays within it)
                for (int i = lane; i < TKEYS * CH; i += 32) {
                    const int j = k0 + i / CH;
                    if (!w.any_seen(j, j)) *reinterpret_cast<uint4*>(dst + i * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (rank == 0) mbar_expect_tx(&kv_full[st], (uint32_t)__popc(k_seen) * (uint32_t)k_rows * D * 2);
                    else arrive_leader_release(&kv_full[st]);
                }
                __syncwarp();
            }
        if (!ok) {
            abort_flag = 1;
            if (lane == 0) set_error(a.err, BLEND_ETIMEOUT);
        }
    } else if (I4 && warp > S_WARP) {
        // ------------------------------------------------ 4-bit pages to bf16 operands (both CTAs)
        const int t = threadIdx.x - (S_WARP + 1) * 32;  // V: token t of the block; K: half a row of this CTA's token t / 2
        constexpr int RB = T::RB, SB = T::SB, RS = T::RAW_STAGES, G = D / 32;
        const int n_blocks = blocks_of(Walk(a, pre, sh, rows2, grp, total)), tk = t >> 1;
        bool ok = true;
        for (int i = 0; i < n_blocks; ++i) {
            const int st = i % STAGES, rs = i % RS;
            ok = warp_wait(&raw_full[rs], (i / RS) & 1, &abort_flag) && warp_poll(&kv_empty[st], ((i / STAGES) & 1) ^ 1, &abort_flag);
            if (!ok) break;
            if (t == 0) pend_raw[rs] = -1;
            const uint8_t* raw = sKV + STAGES * STAGE + rs * T::RAW;
            uint8_t* dk = sKV + st * STAGE;
            {
                const uint4* p = reinterpret_cast<const uint4*>(raw + t * (RB / 2));
                uint32_t kw[D / 16], sc[G];
#pragma unroll
                for (int q = 0; q < D / 64; ++q) {
                    const uint4 v = p[q];
                    kw[4 * q] = v.x; kw[4 * q + 1] = v.y; kw[4 * q + 2] = v.z; kw[4 * q + 3] = v.w;
                }
#pragma unroll
                for (int q = 0; q < G / 2; ++q) {
                    const uint32_t v = *reinterpret_cast<const uint32_t*>(raw + T::RAW_KS + tk * SB + 4 * q);
                    sc[2 * q] = both(v, 0);
                    sc[2 * q + 1] = both(v, 1);
                }
#pragma unroll
                for (int q = 0; q < D / 16; ++q) {
                    // word q of this half row: c = 2 (t & 1) + q / G, g = q % G  (G words per c)
                    const int c = 2 * (t & 1) + q / G, g = q % G, ch = 4 * (g & 1) + c;
                    const uint32_t w = kw[q], hi = w >> 8;
                    uint4 x, y;
                    pair_parts<false>(w, sc[g], x.x, y.x);
                    pair_parts<true>(w, sc[g], x.y, y.y);
                    pair_parts<false>(hi, sc[g], x.z, y.z);
                    pair_parts<true>(hi, sc[g], x.w, y.w);
                    uint8_t* to = dk + (g >> 1) * K_HALF + tk * 128 + ((ch ^ (tk & 7)) << 4);
                    *reinterpret_cast<uint4*>(to) = x;
                    *reinterpret_cast<uint4*>(to + NH * K_HALF) = y;
                }
            }
            uint8_t* dv = dk + KB;
            {
                const int3 at = raw_at[rs];
                const int j = at.x + t;
                const bool seen = j <= at.z && (j < a.n_sink || j > at.y - a.window);
                // a token that no row sees counts as zero whatever its scale (or the row, if it was not read)
                uint32_t sw[G / 2];
#pragma unroll
                for (int g = 0; g < G / 2; ++g) sw[g] = seen ? *reinterpret_cast<const uint32_t*>(raw + T::RAW_VS + t * SB + 4 * g) : 0u;
                const bool f16 = __all_sync(0xffffffffu, fit_f16(sw[0]) && fit_f16(sw[G / 2 - 1]));
                if (lane == 0) reinterpret_cast<volatile uint8_t*>(&v_f16[st])[t >> 5] = f16 ? 1 : 0;
                auto turn = [&](uint32_t s0, uint32_t s1, auto pair) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        // chunk c holds dims 8c.. of each group: halves r = 2c, 2c + 1; threads start at different
                        // chunks so that a warp's reads fall on distinct banks
                        const int c = (q + (t >> 1)) & 3;
                        uint32_t x, y;  // words of halves 2c, 2c + 1 with this CTA's groups
                        if constexpr (D == 128) {
                            const uint4 v = *reinterpret_cast<const uint4*>(raw + T::RAW_V + t * RB + c * 16);
                            x = rank ? v.y : v.x;
                            y = rank ? v.w : v.z;
                        } else {
                            const uint2 v = *reinterpret_cast<const uint2*>(raw + T::RAW_V + t * RB + c * 8);
                            x = rank ? v.x >> 16 : v.x;
                            y = rank ? v.y >> 16 : v.y;
                        }
#pragma unroll
                        for (int g = 0; g < D / 64; ++g) {  // low halves of x, y, then the high ones
                            const uint32_t h0 = g ? x >> 16 : x & 0xffffu, h1 = g ? y >> 16 : y & 0xffffu;
                            const uint32_t y0 = h0 | (h0 << 12), y1 = h1 | (h1 << 12);  // codes 0, 1 and 2, 3 as pairs at bits 0 and 8
                            const uint32_t sc = g ? s1 : s0;
                            const int ch = 4 * g + c;
                            const int to = D == 128 ? t * 128 + ((ch ^ (t & 7)) << 4) : t * 64 + ((ch ^ ((t >> 1) & 3)) << 4);
                            *reinterpret_cast<uint4*>(dv + to) = make_uint4(pair(y0, sc), pair(y0 >> 8, sc), pair(y1, sc), pair(y1 >> 8, sc));
                        }
                    }
                };
                const uint32_t vsc = sw[D == 128 ? rank : 0];
                const int first = D == 128 ? 0 : rank;
                if (f16) turn(both_f16(vsc, first), both_f16(vsc, 1), [](uint32_t w, uint32_t sc) { return pair_f16(w, sc); });
                else turn(both(vsc, first), both(vsc, 1), [](uint32_t w, uint32_t sc) { return pair_value(w, sc); });
            }
            warp_arrive(&raw_empty[rs]);
            fence_async_smem();
            warp_arrive(rank == 0 ? &kv_full[st] : &own_full[st]);
        }
        if (!ok) {
            abort_flag = 1;
            if (lane == 0) set_error(a.err, BLEND_ETIMEOUT);
        }
    }
    fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && abort_flag) {
        // let the copies still in flight land before the shared memory is released
        if (rank == 0 && !I4)
            for (int s = 0; s < STAGES; ++s)
                if (pend_kv[s] >= 0)
                    for (long long i = 0; i < SPIN_LIMIT && !mbar_try(&kv_full[s], (uint32_t)pend_kv[s]); ++i) {
                    }
        if (rank == 0)
            for (int b = 0; b < 2; ++b)
                if (pend_q[b] >= 0)
                    for (long long i = 0; i < SPIN_LIMIT && !mbar_try(&q_full[b], (uint32_t)pend_q[b]); ++i) {
                    }
        if (I4)
            for (int s = 0; s < T::RAW_STAGES; ++s)
                if (pend_raw[s] >= 0)
                    for (long long i = 0; i < SPIN_LIMIT && !mbar_try(&raw_full[s], (uint32_t)pend_raw[s]); ++i) {
                    }
        // (an edge barrier's parity is its warp's; it is waited for in both, which costs a bounded wait)
        for (int st = 0; st < STAGES; ++st)
            if (pend_edge[st] >= 0)
                for (int par = 0; par < 2; ++par)
                    for (long long i = 0; i < SPIN_LIMIT / 16 && !mbar_try(&edge_full[st], (uint32_t)par); ++i) {
                    }
    }
    __syncthreads();
    cluster_sync();  // neither CTA leaves while the other may still signal its barriers
    if (warp == 1) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tb), "r"(TMEM_COLS) : "memory");
    }
}

PFN_cuTensorMapEncodeTiled_v12000 g_enc = nullptr;

bool encode(CUtensorMap* map, int rank, const void* base, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box, CUtensorMapSwizzle swizzle) {
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return g_enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, es,
                 CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                 CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool I4, int D> int launch_tile(const PagedAttn& a, cudaStream_t s) {
    using T = TileCfg<I4, D>;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(T::THREADS);
    cfg.dynamicSmemBytes = T::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    static int clusters = -1;
    if (clusters < 0) {
        cudaFuncSetAttribute(k_paged_tile<I4, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, T::SMEM);
        cfg.gridDim = dim3(2 * MAX_CLUSTERS);
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, k_paged_tile<I4, D>, &cfg) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
        clusters = n < MAX_CLUSTERS ? n : MAX_CLUSTERS;
    }
    if (clusters <= 0) return BLEND_EUNSUPPORTED;
    const int rpt = TQ / a.group, page = 1 << a.pg.shift;
    CUtensorMap mq, mk, mv;
    const cuuint64_t qd[4] = {(cuuint64_t)D, (cuuint64_t)a.group, (cuuint64_t)a.pg.hkv, (cuuint64_t)a.max_rows};
    const cuuint64_t qs[3] = {(cuuint64_t)D * 2, (cuuint64_t)a.group * D * 2, (cuuint64_t)a.ld_q * 2};
    const cuuint32_t qb[4] = {64, (cuuint32_t)a.group, 1, (cuuint32_t)rpt};
    if (!encode(&mq, 4, a.q, qd, qs, qb, CU_TENSOR_MAP_SWIZZLE_128B)) return BLEND_EUNSUPPORTED;
    mk = mv = mq;  // not read for 4-bit pages
    if (!I4) {
        const cuuint64_t kd[3] = {(cuuint64_t)D, (cuuint64_t)page, (cuuint64_t)a.pg.hkv * a.pg.n_pages};
        const cuuint64_t ks[2] = {(cuuint64_t)D * 2, (cuuint64_t)page * D * 2};
        const cuuint32_t kb[3] = {64, (cuuint32_t)(page < 64 ? page : 64), 1};
        const cuuint32_t vb[3] = {(cuuint32_t)T::VCOL, (cuuint32_t)page, 1};
        if (!encode(&mk, 3, a.pg.k, kd, ks, kb, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !encode(&mv, 3, a.pg.v, kd, ks, vb, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
            return BLEND_EUNSUPPORTED;
    }
    cfg.gridDim = dim3(2 * clusters);
    if (cudaLaunchKernelEx(&cfg, k_paged_tile<I4, D>, mq, mk, mv, a, rpt) != cudaSuccess) return BLEND_ECUDA;
    note_launch(1);
    return BLEND_OK;
}

}  // namespace

int launch_paged_attn_tile(bool i4, const PagedAttn& a, int d, cudaStream_t s) {
    if (!g_enc) {
        cudaDriverEntryPointQueryResult qr;
        void* fn = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &qr) !=
                cudaSuccess ||
            qr != cudaDriverEntryPointSuccess || !fn)
            return BLEND_EUNSUPPORTED;
        g_enc = (PFN_cuTensorMapEncodeTiled_v12000)fn;
    }
    if (i4) return d == 64 ? launch_tile<true, 64>(a, s) : launch_tile<true, 128>(a, s);
    return d == 64 ? launch_tile<false, 64>(a, s) : launch_tile<false, 128>(a, s);
}

}  // namespace blend

// Paged KV cache of one layer: what the append, gather and attention kernels share.
#pragma once
#include "common.cuh"

namespace blend {

constexpr int PAGED_STEP = 16;       // keys of one step of the row-split kernels; every page holds whole steps
constexpr int PAGED_MAX_CTAS = 640;  // CTAs of a launch that may leave partial results
constexpr int PAGED_NO_WINDOW = 1 << 30;  // past every position, and position - window stays in 32 bits
constexpr int PAGED_MAX_TILE = 32;   // (row, head) pairs of one tile of those kernels
// fp32 partial results: two slots per CTA, each [pair][head_dim] sums, then maxima and sums per pair
constexpr size_t paged_slot_floats(int d) { return (size_t)PAGED_MAX_TILE * (d + 2); }
constexpr size_t PAGED_PRE_INTS = (size_t)152 * (BLEND_MAX_SEQS + 1);
constexpr size_t paged_part_bytes(int d) { return 2 * (size_t)PAGED_MAX_CTAS * paged_slot_floats(d) * 4; }

// The pages as the kernels see them (blend_pages with the model's head count).
struct PageView {
    const char* k;
    const char* v;
    const char* ks;  // 4-bit pages: bf16 scales [page][head][token][d/32]
    const char* vs;
    const int32_t* table;
    int n_pages, n_seq, max_pages;
    int shift;  // log2(tokens per page)
    int hkv;
};

__device__ __forceinline__ int page_entry(const PageView& p, int seq, int t) {
    return __ldg(p.table + (long long)seq * p.max_pages + (t >> p.shift));
}
// A table entry outside the pool is reported and page 0 read in its place.
__device__ __forceinline__ int checked_page(const PageView& p, int page, int32_t* err) {
    if ((unsigned)page < (unsigned)p.n_pages) return page;
    set_error(err, BLEND_EDEVICE);
    return 0;
}
// Row of (page, head, token in page) counted in rows of the pool: 64 bits, pools pass 2^31 elements.
__device__ __forceinline__ long long page_row(const PageView& p, int page, int head, int in_page) {
    return (((long long)page * p.hkv + head) << p.shift) + in_page;
}

// ---- packed 4-bit rows (layout in blend.h at BLEND_PAGES_INT4)
// Eight consecutive dims 32g + 8c .. +7 of a K row are one 32-bit word; dim e of them sits at
// bit 4 (e / 2) + 16 (e % 2), so (w >> 4 i) & 0x000F000F is the pair (2i, 2i + 1).
__device__ __forceinline__ int k4_word(int d, int g, int c) { return c * (d / 8) + 4 * g; }  // byte offset in the row
__device__ __forceinline__ int k4_bit(int e) { return 4 * (e >> 1) + 16 * (e & 1); }
// Four consecutive dims 32g + 4r .. +3 of a V row are one 16-bit word, dim e at bit 4 e.
__device__ __forceinline__ int v4_half(int d, int g, int r) { return r * (d / 16) + 2 * g; }

// Two codes as bf16 values (n - 8) / 64, exact.  A code n + 8 alone in the low bits of a bf16 is
// (n + 8) 2^-133, and alone at bits 4..7 it is 16 times that (bf16 is linear up to bit pattern 255),
// so a mask selects a pair and one multiply-add shifts and scales it; no bits are moved for half of
// the codes.  HI: the codes at bits 4..7 and 20..23.
constexpr float CODE_UNIT = 64.f;
template <bool HI> __device__ __forceinline__ uint32_t code_pair(uint32_t w) {
    uint32_t x = w & (HI ? 0x00F000F0u : 0x000F000Fu);
    const uint32_t up = HI ? 0x7D007D00u : 0x7F007F00u;  // 2^123, 2^127
    const uint32_t off = 0xBE00BE00u;                    // -1/8
    const __nv_bfloat162 r = __hfma2(*reinterpret_cast<__nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&up),
                                     *reinterpret_cast<const __nv_bfloat162*>(&off));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// Two codes at bits 0..3 and 16..19 as bf16 values n, exact: in the low bits of 128 a code is 128 + n + 8.
__device__ __forceinline__ uint32_t code_ints(uint32_t w) {
    uint32_t x = (w & 0x000F000Fu) | 0x43004300u;
    const uint32_t off = 0x43084308u;  // 136
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&off));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// Arguments of the attention kernels.
struct PagedAttn {
    PageView pg;
    const void* q;
    long long ld_q;  // elements between rows of q
    const int32_t* q_start;
    const int32_t* kv_len;
    int max_rows, max_q;
    int short_pairs;  // tile kernel: sequences of up to so many pairs are the split kernel's
    int hq, group;
    int window;  // PAGED_NO_WINDOW: none
    int n_sink;
    float scale_log2;  // log2(e) / sqrt(d)
    void* out;
    float* part;
    int32_t* count;
    int* pre;  // tile kernel: each CTA's prefix sums over the sequences
    int32_t* err;
};

// Query rows and length of one sequence; a bad entry is reported and gives no rows.
struct SeqInfo {
    int row0, n_q, len;
};
__device__ __forceinline__ SeqInfo seq_info(const PagedAttn& a, int s) {
    SeqInfo i;
    i.row0 = __ldg(a.q_start + s);
    const int end = __ldg(a.q_start + s + 1);
    i.len = __ldg(a.kv_len + s);
    i.n_q = end - i.row0;
    if (i.row0 < 0 || end < i.row0 || end > a.max_rows || i.n_q > a.max_q || i.len < 0 ||
        i.len > (a.pg.max_pages << a.pg.shift)) {
        set_error(a.err, BLEND_EDEVICE);
        i.row0 = 0;
        i.n_q = 0;
        i.len = 0;
    }
    return i;
}

// Sums over sequences are capped: bounds that go down and up again may claim the same rows many times, so
// that what the caller's sizes bound for ascending ones passes 32 bits.  Terms are at most `cap` < 2^31.
__host__ __device__ __forceinline__ int add_capped(int x, int y, int cap) {
    const unsigned s = (unsigned)x + (unsigned)y;
    return s < (unsigned)cap ? (int)s : cap;
}
constexpr int PAGED_MAX_UNITS = 0x7fffffff;  // work units of a call: fewer than this

// Keys that rows at positions p0..p1 of one sequence see, as blocks of BLK keys: the sinks'
// blocks 0..n_a-1, then blocks first_b.. of the window's range (n_b of them).
struct KeyRange {
    int n_a, first_b, n_b;
    __device__ __forceinline__ int total() const { return n_a + n_b; }
    __device__ __forceinline__ int block(int i) const { return i < n_a ? i : first_b + (i - n_a); }
};
template <int BLK>
__device__ __forceinline__ KeyRange key_range(int p0, int p1, int window, int n_sink) {
    KeyRange r{0, 0, 0};
    if (p1 < 0) return r;
    const int lo = max(0, max(p0, 0) - window + 1);
    r.first_b = lo / BLK;
    if (lo > 0) r.n_a = min((min(n_sink, p1 + 1) + BLK - 1) / BLK, r.first_b);
    r.n_b = p1 / BLK + 1 - r.first_b;
    return r;
}
// Key j is visible to a row at position p.
__device__ __forceinline__ bool sees(int j, int p, int window, int n_sink) {
    return j <= p && (j > p - window || j < n_sink);
}
// Key j is visible to some row at positions p0..p1.
__device__ __forceinline__ bool seen_by_any(int j, int p0, int p1, int window, int n_sink) {
    return j <= p1 && (j < n_sink || j > p0 - window);
}
// Every key of [j0, j1] is visible to every row at positions p0..p1.
__device__ __forceinline__ bool all_see(int j0, int j1, int p0, int p1, int window, int n_sink) {
    return j1 <= p0 && (j0 > p1 - window || j1 < n_sink);
}

// ---- cp.async
// BYTES from global to shared memory; zeros when !ok.
template <int BYTES> __device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool ok) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(ok ? BYTES : 0)
                     : "memory");
}
template <int BYTES> __device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
    if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Maximum that keeps a NaN: a running maximum that dropped one would give its row no weight
// when the shares of the keys are joined.
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// How the line of all items' units is shared out: share b takes units b quota .. (b + 1) quota - 1,
// except that a border within `snap` units of an item's end moves to that end (to the nearer one of a
// short item): a part costs its share a fixed time, and the join another.  So an item of fewer than
// 2 snap units is never cut.  Totals reach 2^31 - 1, so nothing here is rounded up by an addition to them.
struct Shares {
    int quota, snap, n;
    __host__ __device__ __forceinline__ Shares(int total, int quota_, int snap_)
        : quota(quota_), snap(snap_), n(parts(total, quota_)) {}
    static __host__ __device__ __forceinline__ int parts(int total, int of) { return (total - 1) / of + 1; }  // total >= 1
    // a unit from whose item on share b has to look for its own
    __host__ __device__ __forceinline__ int start(int b) const { return max(0, b * quota - (snap - 1)); }
    // first and last share of the item of units [i0, i1)
    __host__ __device__ __forceinline__ int first(int i0, int i1) const { return (i0 + min(snap, (int)(((unsigned)(i1 - i0) + 1u) >> 1)) - 1) / quota; }
    __host__ __device__ __forceinline__ int last(int i0, int i1) const { return max((i1 - snap) / quota, first(i0, i1)); }
    // share b's units of it, from i0
    __host__ __device__ __forceinline__ int begin(int b, int i0, int i1) const { return b == first(i0, i1) ? 0 : b * quota - i0; }
    __host__ __device__ __forceinline__ int end(int b, int i0, int i1) const { return b == last(i0, i1) ? i1 - i0 : (b + 1) * quota - i0; }
};

void launch_paged_append(int dtype, bool i4, const PageView& pg, int hq, int d, const void* k_new, long long ld_k,
                         const void* v_new, long long ld_v, const void* q, long long ld_q, void* q_out,
                         const int32_t* seq, const int32_t* pos, const int32_t* rot, const int32_t* n_dev, int max_n,
                         const float2* tab, int max_pos, int32_t* err, cudaStream_t s);
void launch_paged_gather(int dtype, bool i4, const PageView& pg, int d, const int32_t* seq, const int32_t* pos,
                         const int32_t* rot, const int32_t* n_dev, int max_n, void* k_out, void* v_out,
                         const float2* tab, int max_pos, int32_t* err, cudaStream_t s);
// Sequences of more than a.short_pairs (row, head) pairs, bf16 (paged_tile.cu); others are left alone.
// Returns BLEND_EUNSUPPORTED, with nothing launched, where no pair of CTAs fits or an operand has no
// tensor map, and BLEND_ECUDA (the error left to be read) when the launch fails.
int launch_paged_attn_tile(bool i4, const PagedAttn& a, int d, cudaStream_t s);
// Sequences of at most 32 (row, head) pairs, bf16 (paged_split.cu); others are left alone.
void launch_paged_attn_split(bool i4, const PagedAttn& a, int d, cudaStream_t s);
void launch_paged_attn_simt(int dtype, bool i4, const PagedAttn& a, int d, cudaStream_t s);
}  // namespace blend

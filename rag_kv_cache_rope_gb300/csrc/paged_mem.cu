// Paged KV cache: rows appended with their rotation, and read back (paged_append,
// paged_gather in blend.h).
//
// One thread owns the 16 dims i..i+7 and i+d/2..i+d/2+7 of one head of one row: the eight
// rotation pairs it needs sit in its own registers, and in the 4-bit form these are one
// 32-bit word of each of two 32-dim groups, whose maxima are shared by the four threads of a
// group (two shuffles).  The d/16 threads of a head sit side by side and a warp covers
// neighbouring heads of a row, so the loads are whole 128-byte lines.
// Both kernels are bound by HBM: rows in, rows out, nothing read twice but the rotation
// table, which stays in L2 (one row of it per position, shared by all heads).
//
// The rotation is (x1 c - x2 s, x2 c + x1 s) with every product and sum rounded to fp32 on
// its own (no contraction): the 4-bit codes are a rounding of these values, so their bits
// are part of the format and any program that repeats the steps gets the same codes.
#include "paged.cuh"

namespace blend {
namespace {

constexpr int MEM_THREADS = 256;

// Eight consecutive dims as fp32.
__device__ __forceinline__ void load8(const bf16* p, float* x) {
    const Vec<bf16> v = ld16(p);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = v.get(e);
}
__device__ __forceinline__ void load8(const float* p, float* x) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void store8(bf16* p, const float* x) {
    Vec<bf16> v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v.set(e, x[e]);
    st16(p, v);
}
__device__ __forceinline__ void store8(float* p, const float* x) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// Pairs (a[e], b[e]) of dims i0 + e, i0 + e + half rotated by `rot` positions; 0 leaves them
// bit for bit as they are (an infinity stays one).
__device__ __forceinline__ void rotate8(float* a, float* b, int rot, int i0, int half, const float2* tab) {
    if (rot == 0) return;
    const float4* cs = reinterpret_cast<const float4*>(tab + (long long)abs(rot) * half + i0);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float4 t = __ldg(cs + e);
        const float s0 = rot < 0 ? -t.y : t.y, s1 = rot < 0 ? -t.w : t.w;
        const float a0 = a[2 * e], b0 = b[2 * e], a1 = a[2 * e + 1], b1 = b[2 * e + 1];
        a[2 * e] = __fsub_rn(__fmul_rn(a0, t.x), __fmul_rn(b0, s0));
        b[2 * e] = __fadd_rn(__fmul_rn(b0, t.x), __fmul_rn(a0, s0));
        a[2 * e + 1] = __fsub_rn(__fmul_rn(a1, t.z), __fmul_rn(b1, s1));
        b[2 * e + 1] = __fadd_rn(__fmul_rn(b1, t.z), __fmul_rn(a1, s1));
    }
}

// Scale of the 32 dims that four neighbouring threads hold eight each of: bf16 of max / 7;
// NaN when one of them is not finite.  Call it with all 32 lanes.
__device__ __forceinline__ bf16 group_scale(const float* x) {
    float m = 0.f;
    bool fin = true;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        m = fmaxf(m, fabsf(x[e]));
        fin = fin && isfinite(x[e]);
    }
    m = fin ? m : INFINITY;
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    return __float2bfloat16_rn(isfinite(m) ? __fdiv_rn(m, 7.f) : __int_as_float(0x7fc00000));
}
// Code of x, 1..15 (value code - 8), 8 where the scale is zero or NaN.
__device__ __forceinline__ uint32_t code4(float x, float scale) {
    if (!(scale > 0.f)) return 8u;
    return (uint32_t)(8 + (int)fminf(fmaxf(rintf(__fdiv_rn(x, scale)), -7.f), 7.f));
}

struct RowAt {
    bool ok;
    int seq, pos, rot;
    long long at;  // pool row of head 0
};
// Place and rotation of row i; a negative sequence marks a row to leave alone, anything out
// of range is reported and left alone as well.
__device__ __forceinline__ RowAt row_at(const PageView& pg, const int32_t* seq, const int32_t* pos, const int32_t* rot,
                                        bool by_pos, int i, int max_pos, int32_t* err) {
    RowAt r;
    r.seq = __ldg(seq + i);
    r.pos = __ldg(pos + i);
    r.rot = rot ? __ldg(rot + i) : by_pos ? r.pos : 0;
    r.ok = r.seq >= 0;
    r.at = 0;
    if (!r.ok) return r;
    if (r.seq >= pg.n_seq || r.pos < 0 || r.pos >= (pg.max_pages << pg.shift) || r.rot <= -max_pos || r.rot >= max_pos) {
        set_error(err, BLEND_EDEVICE);
        r.ok = false;
        return r;
    }
    const int page = __ldg(pg.table + (long long)r.seq * pg.max_pages + (r.pos >> pg.shift));
    if ((unsigned)page >= (unsigned)pg.n_pages) {
        set_error(err, BLEND_EDEVICE);
        r.ok = false;
        return r;
    }
    r.at = page_row(pg, page, 0, r.pos & ((1 << pg.shift) - 1));
    return r;
}
__device__ __forceinline__ int checked_count(const int32_t* n_dev, int max_n, int32_t* err) {
    const int n = __ldg(n_dev);
    if (n < 0 || n > max_n) {
        if (blockIdx.x == 0 && threadIdx.x == 0) set_error(err, BLEND_EDEVICE);
        return n < 0 ? 0 : max_n;
    }
    return n;
}

// Head slots of a row: hkv keys, hkv values, then (with q) hq query heads.
template <typename T, bool I4, int D>
__global__ void __launch_bounds__(MEM_THREADS)
    k_paged_append(PageView pg, int hq, const T* __restrict__ k_new, long long ld_k, const T* __restrict__ v_new,
                   long long ld_v, const T* q, long long ld_q, T* q_out, const int32_t* __restrict__ seq,
                   const int32_t* __restrict__ pos, const int32_t* __restrict__ rot, const int32_t* __restrict__ n_dev,
                   int max_n, const float2* __restrict__ tab, int max_pos, int32_t* err) {
    constexpr int TPH = D / 16, HALF = D / 2;
    const int n = checked_count(n_dev, max_n, err);
    const int slots = 2 * pg.hkv + (q ? hq : 0);
    const long long unit = ((long long)blockIdx.x * MEM_THREADS + threadIdx.x) / TPH;
    const int i0 = (threadIdx.x % TPH) * 8;
    const long long row64 = unit / slots;
    const int slot = (int)(unit - row64 * slots);
    RowAt r{false, 0, 0, 0, 0};
    const int row = (int)row64;
    if (row64 < n) r = row_at(pg, seq, pos, rot, true, row, max_pos, err);
    const bool is_k = slot < pg.hkv, is_v = !is_k && slot < 2 * pg.hkv;
    const int head = is_k ? slot : is_v ? slot - pg.hkv : slot - 2 * pg.hkv;
    float a[8] = {}, b[8] = {};
    if (r.ok) {
        const T* src = (is_k ? k_new + row * ld_k : is_v ? v_new + row * ld_v : q + row * ld_q) + head * D;
        load8(src + i0, a);
        load8(src + i0 + HALF, b);
        if (!is_v) rotate8(a, b, r.rot, i0, HALF, tab);
    }
    if (!is_k && !is_v) {
        if (r.ok) {
            T* dst = q_out + ((long long)row * hq + head) * D;
            store8(dst + i0, a);
            store8(dst + i0 + HALF, b);
        }
        if (!I4) return;
    }
    const long long at = r.at + ((long long)head << pg.shift);
    char* base = const_cast<char*>(is_k ? pg.k : pg.v);
    if constexpr (!I4) {
        if (!r.ok) return;
        T* dst = reinterpret_cast<T*>(base) + at * D;
        store8(dst + i0, a);
        store8(dst + i0 + HALF, b);
    } else {
        // all lanes take part in the shuffles; the words are stored by those with a row
        const bf16 sa = group_scale(a), sb = group_scale(b);
        if (!r.ok || (!is_k && !is_v)) return;
        const float fa = __bfloat162float(sa), fb = __bfloat162float(sb);
        const int g = i0 / 32, g2 = (i0 + HALF) / 32, c = (i0 % 32) / 8;
        char* dst = base + at * (D / 2);
        uint32_t wa = 0, wb = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int bit = is_k ? k4_bit(e) : 4 * e;
            wa |= code4(a[e], fa) << bit;
            wb |= code4(b[e], fb) << bit;
        }
        if (is_k) {
            *reinterpret_cast<uint32_t*>(dst + k4_word(D, g, c)) = wa;
            *reinterpret_cast<uint32_t*>(dst + k4_word(D, g2, c)) = wb;
        } else {
            *reinterpret_cast<uint16_t*>(dst + v4_half(D, g, 2 * c)) = (uint16_t)wa;
            *reinterpret_cast<uint16_t*>(dst + v4_half(D, g, 2 * c + 1)) = (uint16_t)(wa >> 16);
            *reinterpret_cast<uint16_t*>(dst + v4_half(D, g2, 2 * c)) = (uint16_t)wb;
            *reinterpret_cast<uint16_t*>(dst + v4_half(D, g2, 2 * c + 1)) = (uint16_t)(wb >> 16);
        }
        if (c == 0) {
            bf16* sc = reinterpret_cast<bf16*>(const_cast<char*>(is_k ? pg.ks : pg.vs)) + at * (D / 32);
            sc[g] = sa;
            sc[g2] = sb;
        }
    }
}

template <typename T, bool I4, int D>
__global__ void __launch_bounds__(MEM_THREADS)
    k_paged_gather(PageView pg, const int32_t* __restrict__ seq, const int32_t* __restrict__ pos,
                   const int32_t* __restrict__ rot, const int32_t* __restrict__ n_dev, int max_n,
                   T* __restrict__ k_out, T* __restrict__ v_out, const float2* __restrict__ tab, int max_pos,
                   int32_t* err) {
    constexpr int TPH = D / 16, HALF = D / 2;
    const int n = checked_count(n_dev, max_n, err);
    const int slots = 2 * pg.hkv;
    const long long unit = ((long long)blockIdx.x * MEM_THREADS + threadIdx.x) / TPH;
    const int i0 = (threadIdx.x % TPH) * 8;
    const long long row64 = unit / slots;
    if (row64 >= n) return;
    const int row = (int)row64, slot = (int)(unit - row64 * slots);
    const RowAt r = row_at(pg, seq, pos, rot, false, row, max_pos, err);
    if (!r.ok) return;
    const bool is_k = slot < pg.hkv;
    const int head = is_k ? slot : slot - pg.hkv;
    const long long at = r.at + ((long long)head << pg.shift);
    const char* base = is_k ? pg.k : pg.v;
    float a[8], b[8];
    if constexpr (!I4) {
        const T* src = reinterpret_cast<const T*>(base) + at * D;
        load8(src + i0, a);
        load8(src + i0 + HALF, b);
    } else {
        const int g = i0 / 32, g2 = (i0 + HALF) / 32, c = (i0 % 32) / 8;
        const char* src = base + at * (D / 2);
        uint32_t wa, wb;
        if (is_k) {
            wa = *reinterpret_cast<const uint32_t*>(src + k4_word(D, g, c));
            wb = *reinterpret_cast<const uint32_t*>(src + k4_word(D, g2, c));
        } else {
            wa = *reinterpret_cast<const uint16_t*>(src + v4_half(D, g, 2 * c)) |
                 (uint32_t)*reinterpret_cast<const uint16_t*>(src + v4_half(D, g, 2 * c + 1)) << 16;
            wb = *reinterpret_cast<const uint16_t*>(src + v4_half(D, g2, 2 * c)) |
                 (uint32_t)*reinterpret_cast<const uint16_t*>(src + v4_half(D, g2, 2 * c + 1)) << 16;
        }
        const bf16* sc = reinterpret_cast<const bf16*>(is_k ? pg.ks : pg.vs) + at * (D / 32);
        const float fa = __bfloat162float(sc[g]), fb = __bfloat162float(sc[g2]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int bit = is_k ? k4_bit(e) : 4 * e;
            a[e] = __fmul_rn((float)((int)((wa >> bit) & 15u) - 8), fa);
            b[e] = __fmul_rn((float)((int)((wb >> bit) & 15u) - 8), fb);
        }
    }
    if (is_k) rotate8(a, b, r.rot, i0, HALF, tab);
    T* dst = (is_k ? k_out : v_out) + ((long long)row * pg.hkv + head) * D;
    store8(dst + i0, a);
    store8(dst + i0 + HALF, b);
}

template <typename T, bool I4, int D>
void append_d(const PageView& pg, int hq, const void* k_new, long long ld_k, const void* v_new, long long ld_v,
              const void* q, long long ld_q, void* q_out, const int32_t* seq, const int32_t* pos, const int32_t* rot,
              const int32_t* n_dev, int max_n, const float2* tab, int max_pos, int32_t* err, cudaStream_t s) {
    const long long threads = (long long)max_n * (2 * pg.hkv + (q ? hq : 0)) * (D / 16);
    const long long blocks = (threads + MEM_THREADS - 1) / MEM_THREADS;
    k_paged_append<T, I4, D><<<(unsigned)blocks, MEM_THREADS, 0, s>>>(
        pg, hq, (const T*)k_new, ld_k, (const T*)v_new, ld_v, (const T*)q, ld_q, (T*)q_out, seq, pos, rot, n_dev, max_n,
        tab, max_pos, err);
}
template <typename T, bool I4, int D>
void gather_d(const PageView& pg, const int32_t* seq, const int32_t* pos, const int32_t* rot, const int32_t* n_dev,
              int max_n, void* k_out, void* v_out, const float2* tab, int max_pos, int32_t* err, cudaStream_t s) {
    const long long threads = (long long)max_n * 2 * pg.hkv * (D / 16);
    const long long blocks = (threads + MEM_THREADS - 1) / MEM_THREADS;
    k_paged_gather<T, I4, D><<<(unsigned)blocks, MEM_THREADS, 0, s>>>(pg, seq, pos, rot, n_dev, max_n, (T*)k_out,
                                                                     (T*)v_out, tab, max_pos, err);
}

}  // namespace

void launch_paged_append(int dtype, bool i4, const PageView& pg, int hq, int d, const void* k_new, long long ld_k,
                         const void* v_new, long long ld_v, const void* q, long long ld_q, void* q_out,
                         const int32_t* seq, const int32_t* pos, const int32_t* rot, const int32_t* n_dev, int max_n,
                         const float2* tab, int max_pos, int32_t* err, cudaStream_t s) {
    if (max_n <= 0) return;
    auto f = dtype == BLEND_BF16
                 ? (i4 ? (d == 64 ? append_d<bf16, true, 64> : append_d<bf16, true, 128>)
                       : (d == 64 ? append_d<bf16, false, 64> : append_d<bf16, false, 128>))
                 : (i4 ? (d == 64 ? append_d<float, true, 64> : append_d<float, true, 128>)
                       : (d == 64 ? append_d<float, false, 64> : append_d<float, false, 128>));
    f(pg, hq, k_new, ld_k, v_new, ld_v, q, ld_q, q_out, seq, pos, rot, n_dev, max_n, tab, max_pos, err, s);
    note_launch(1);
}

void launch_paged_gather(int dtype, bool i4, const PageView& pg, int d, const int32_t* seq, const int32_t* pos,
                         const int32_t* rot, const int32_t* n_dev, int max_n, void* k_out, void* v_out,
                         const float2* tab, int max_pos, int32_t* err, cudaStream_t s) {
    if (max_n <= 0) return;
    auto f = dtype == BLEND_BF16
                 ? (i4 ? (d == 64 ? gather_d<bf16, true, 64> : gather_d<bf16, true, 128>)
                       : (d == 64 ? gather_d<bf16, false, 64> : gather_d<bf16, false, 128>))
                 : (i4 ? (d == 64 ? gather_d<float, true, 64> : gather_d<float, true, 128>)
                       : (d == 64 ? gather_d<float, false, 64> : gather_d<float, false, 128>));
    f(pg, seq, pos, rot, n_dev, max_n, k_out, v_out, tab, max_pos, err, s);
    note_launch(1);
}

}  // namespace blend

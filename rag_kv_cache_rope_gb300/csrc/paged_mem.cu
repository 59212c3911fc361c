// Paged KV cache: rows appended with their rotation, and read back (paged_append,
// paged_gather in blend.h).
//
// One thread owns the 16 dims i..i+7 and i+d/2..i+d/2+7 of one head's key and value (or of one query
// head) of one row: the eight rotation pairs it needs sit in its own registers, its four 16-byte
// loads are on their way together, and in the 4-bit form its dims are eight of each of two 32-dim
// groups, whose maxima the four threads of a group share by two shuffles.  The d/16 threads of a
// head sit side by side and a warp covers neighbouring heads of a row, so loads are whole 128-byte
// lines; 4-bit rows leave as 8 bytes per thread after one exchange between the two halves of a head.
// Rows in, rows out, nothing is read twice but the rotation table, which stays in L2 (one row of it per
// position, shared by all heads).  Measured (GB300, 6.8 TB/s copy rate), 16 064 rows of 8 heads x 128 into
// bf16 pages: 25 us, 5.2 TB/s, bound by HBM; out of 4-bit pages 20 us, 4.1 TB/s, where the chain count and
// entries, page, row is as long as the transfer (hence two rows a thread).  Into 4-bit pages the kernel
// is bound by instruction issue and its dependencies, 57 % of the slots: 57 K rows 92 us, 3.3 TB/s.
//
// The rotation is (x1 c - x2 s, x2 c + x1 s) with every product and sum rounded to fp32 on
// its own (no contraction): the 4-bit codes are a rounding of these values, so their bits
// are part of the format and any program that repeats the steps gets the same codes.
#include "paged.cuh"

namespace blend {
namespace {

constexpr int MEM_THREADS = 256;

// Eight consecutive dims from fp32.
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

// Eight consecutive dims as they are.
template <typename T> struct Raw8 {
    uint4 w[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ void store(T* p) const {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
    }
    __device__ __forceinline__ void get(float* x) const {
        const T* p = reinterpret_cast<const T*>(w);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = to_f<T>(p[e]);
    }
};

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

// Scales of the four 32-dim groups that four neighbouring threads hold eight dims each of: bf16 of
// max * (1/7 in fp32), NaN when a group is not finite, and their reciprocals.  Thread j of the four computes
// group j's (a product and a reciprocal each) and the others read them.  Call it with all 32 lanes.
struct Scale {
    uint32_t bits;  // the bf16
    float s, y;     // its value, and 1 / s
};
__device__ __forceinline__ float group_max(const float* x) {
    float m = fabsf(x[0]);
#pragma unroll
    for (int e = 1; e < 8; ++e) m = max_nan(m, fabsf(x[e]));
    m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
    return max_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
}
__device__ __forceinline__ void group_scales(const float* x0, const float* x1, const float* x2, const float* x3, Scale (&out)[4]) {
    const float m0 = group_max(x0), m1 = group_max(x1), m2 = group_max(x2), m3 = group_max(x3);
    const int j = threadIdx.x & 3;
    const float m = j == 0 ? m0 : j == 1 ? m1 : j == 2 ? m2 : m3;
    const bf16 s = __float2bfloat16_rn(isfinite(m) ? __fmul_rn(m, 1.f / 7.f) : __int_as_float(0x7fc00000));
    const uint32_t bits = __bfloat16_as_ushort(s);
    const float y = __frcp_rn(__bfloat162float(s));
    const int first = (threadIdx.x & 31) & ~3;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        out[k].bits = __shfl_sync(0xffffffffu, bits, first + k);
        out[k].s = __uint_as_float(out[k].bits << 16);
        out[k].y = __shfl_sync(0xffffffffu, y, first + k);
    }
}
// Codes n + 8 of eight values (n = round-to-even of the fp32 quotient x / s, -7..7), each in the low
// four bits of c[e], whose other bits below 22 are zero.  All are 8 where the scale is zero or NaN.
//
// The quotient has to be the correctly rounded one, since a code is a rounding of it.  With y = 1 / s
// correctly rounded, q = x y, r = x - q s (exact) and q + r y is x / s correctly rounded (Markstein's
// theorem, P. Markstein, IBM J. Res. Dev. 34, 1990) as long as nothing leaves the normal range: three
// operations a value instead of a division.  Scales outside 2^-100..2^100 divide.
__device__ __forceinline__ void codes8(const float* x, const Scale& sc, uint32_t (&c)[8]) {
    const float s = sc.s, y = sc.y;
    if (s >= 0x1p-100f && s <= 0x1p100f) {
        // (two values an instruction)
        const float2 y2 = make_float2(y, y), ns2 = make_float2(-s, -s), up2 = make_float2(12582920.f, 12582920.f);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const float2 x2 = make_float2(x[e], x[e + 1]), q = __fmul2_rn(x2, y2);
            // max |x| / s stays below 7.5 for such scales, so the code is in range without a clamp; adding
            // 1.5 2^23 rounds to an integer, ties to even (and the 8 keeps its parity)
            const float2 r = __fadd2_rn(__ffma2_rn(__ffma2_rn(q, ns2, x2), y2, q), up2);
            c[e] = __float_as_uint(r.x);
            c[e + 1] = __float_as_uint(r.y);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            c[e] = s > 0.f ? (uint32_t)(8 + (int)fminf(fmaxf(rintf(__fdiv_rn(x[e], s)), -7.f), 7.f)) : 8u;
    }
}
// Four codes to 16 bits, in the low half (what the codes carry from bit 22 up stays above).
__device__ __forceinline__ uint32_t four(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return a + b * 16u + c * 256u + d * 4096u;
}
// K: even codes in the low half of a word, odd ones in the high half.  V: in order.
__device__ __forceinline__ uint32_t k_word(const uint32_t (&c)[8]) {
    return __byte_perm(four(c[0], c[2], c[4], c[6]), four(c[1], c[3], c[5], c[7]), 0x5410);
}
__device__ __forceinline__ uint32_t v_word(const uint32_t (&c)[8]) {
    return __byte_perm(four(c[0], c[1], c[2], c[3]), four(c[4], c[5], c[6], c[7]), 0x5410);
}
// A K word's values n s, each a product of exact numbers rounded once.  (As (n / 64) (64 s), which saves the
// two shifts, scales from 2^122 on gave infinities, and NaN for a code of 0.)
__device__ __forceinline__ void k_values(uint32_t w, float s, float* x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t p = code_ints(w >> (4 * i));
        x[2 * i] = __fmul_rn(__uint_as_float(p << 16), s);
        x[2 * i + 1] = __fmul_rn(__uint_as_float(p & 0xffff0000u), s);
    }
}
// A V word's values: codes 0, 1 and 2, 3 of a half are pairs once the half is repeated 12 bits up.
__device__ __forceinline__ void v_values(uint32_t w, float s, float* x) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t c = h ? w >> 16 : w & 0xffffu, y = c | (c << 12);
        const uint32_t p[2] = {code_ints(y), code_ints(y >> 8)};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            x[4 * h + 2 * i] = __fmul_rn(__uint_as_float(p[i] << 16), s);
            x[4 * h + 2 * i + 1] = __fmul_rn(__uint_as_float(p[i] & 0xffff0000u), s);
        }
    }
}

// Where row i goes, in the three steps of its loads (so that two rows' loads can be on their way
// together): its entries; the page of its token; the place.  A negative sequence marks a row to
// leave alone, anything out of range is reported and left alone as well.
struct RowAt {
    bool ok;
    int seq, pos, rot, page;
    __device__ __forceinline__ void read(const int32_t* seq_, const int32_t* pos_, const int32_t* rot_, bool by_pos, long long i, bool in) {
        seq = in ? __ldg(seq_ + i) : -1;
        pos = in ? __ldg(pos_ + i) : 0;
        rot = rot_ ? (in ? __ldg(rot_ + i) : 0) : by_pos ? pos : 0;
    }
    __device__ __forceinline__ void find(const PageView& pg, int max_pos, bool live, int32_t* err) {
        ok = live && seq >= 0;
        const bool bad = seq >= pg.n_seq || pos < 0 || pos >= (pg.max_pages << pg.shift) || rot <= -max_pos || rot >= max_pos;
        if (ok && bad) set_error(err, BLEND_EDEVICE);
        ok = ok && !bad;
        page = ok ? page_entry(pg, seq, pos) : 0;
    }
    __device__ __forceinline__ long long place(const PageView& pg, int head, int32_t* err) {  // its pool row
        if ((unsigned)page >= (unsigned)pg.n_pages) {
            set_error(err, BLEND_EDEVICE);
            ok = false;
        }
        return ok ? page_row(pg, page, head, pos & ((1 << pg.shift) - 1)) : 0;
    }
};
__device__ __forceinline__ int checked_count(const int32_t* n_dev, int max_n, int32_t* err) {
    const int n = __ldg(n_dev);
    if (n < 0 || n > max_n) {
        if (blockIdx.x == 0 && threadIdx.x == 0) set_error(err, BLEND_EDEVICE);
        return n < 0 ? 0 : max_n;
    }
    return n;
}

// Slots of a row: hkv kv heads (key and value), then (with q) hq query heads.
template <typename T, bool I4, int D>
__global__ void __launch_bounds__(MEM_THREADS, 4)
    k_paged_append(PageView pg, int hq, const T* __restrict__ k_new, long long ld_k, const T* __restrict__ v_new,
                   long long ld_v, const T* q, long long ld_q, T* q_out, const int32_t* __restrict__ seq,
                   const int32_t* __restrict__ pos, const int32_t* __restrict__ rot, const int32_t* __restrict__ n_dev,
                   int max_n, long long row0, const float2* __restrict__ tab, int max_pos, int32_t* err) {
    constexpr int TPH = D / 16, HALF = D / 2;
    const int slots = pg.hkv + (q ? hq : 0);
    const unsigned unit = (blockIdx.x * MEM_THREADS + threadIdx.x) / TPH;  // below 2^32 / TPH (launcher)
    const int t = threadIdx.x % TPH, i0 = t * 8;
    const long long row = row0 + unit / (unsigned)slots;
    const int slot = (int)(unit % (unsigned)slots);
    const bool in = row < max_n, is_kv = slot < pg.hkv;
    const int head = is_kv ? slot : slot - pg.hkv;
    RowAt r;
    r.read(seq, pos, rot, true, row, in);
    Raw8<T> ra{}, rb{}, rva{}, rvb{};
    if (in) {  // (without waiting for the count)
        const T* src = is_kv ? k_new + row * ld_k + head * D : q + row * ld_q + head * D;
        ra.load(src + i0);
        rb.load(src + i0 + HALF);
        if (is_kv) {
            const T* sv = v_new + row * ld_v + head * D;
            rva.load(sv + i0);
            rvb.load(sv + i0 + HALF);
        }
    }
    r.find(pg, max_pos, row < checked_count(n_dev, max_n, err), err);
    const long long at = r.place(pg, head, err);
    float a[8], b[8];
    ra.get(a);
    rb.get(b);
    if (r.ok) rotate8(a, b, r.rot, i0, HALF, tab);
    if (!is_kv && r.ok) {
        T* dst = q_out + (row * hq + head) * D;
        store8(dst + i0, a);
        store8(dst + i0 + HALF, b);
    }
    const bool store = r.ok && is_kv;
    if constexpr (!I4) {
        if (!store) return;
        T* dk = reinterpret_cast<T*>(const_cast<char*>(pg.k)) + at * D;
        T* dv = reinterpret_cast<T*>(const_cast<char*>(pg.v)) + at * D;
        store8(dk + i0, a);
        store8(dk + i0 + HALF, b);
        rva.store(dv + i0);
        rvb.store(dv + i0 + HALF);
    } else {
        float va[8], vb[8];
        rva.get(va);
        rvb.get(vb);
        // all lanes take part in the shuffles
        Scale sc[4];
        group_scales(a, b, va, vb, sc);
        uint32_t c8[8];
        codes8(a, sc[0], c8);
        const uint32_t k0 = k_word(c8);  // word (c, g)
        codes8(b, sc[1], c8);
        const uint32_t k1 = k_word(c8);  // and (c, g + D / 64)
        codes8(va, sc[2], c8);
        const uint32_t w0 = v_word(c8);  // halves (g, 2c), (g, 2c + 1)
        codes8(vb, sc[3], c8);
        const uint32_t w1 = v_word(c8);  // and those of g + D / 64
        uint32_t v0 = __byte_perm(w0, w1, 0x5410), v1 = __byte_perm(w0, w1, 0x7632);  // by half: 2c, 2c + 1
        const uint32_t ks = sc[0].bits | sc[1].bits << 16, vs = sc[2].bits | sc[3].bits << 16;
        uint2 kw, vw, sk, sv;
        if constexpr (D == 128) {
            // thread t holds groups g = t / 4 and g + 2; t ^ 4 has the other two of the same dims.  The lower
            // thread takes words 0, 1 of chunk c and half 2c, the upper one words 2, 3 and half 2c + 1.
            const bool up = t >= 4;
            const uint32_t ko = __shfl_xor_sync(0xffffffffu, up ? k0 : k1, 4);
            kw = up ? make_uint2(ko, k1) : make_uint2(k0, ko);
            const uint32_t vo = __shfl_xor_sync(0xffffffffu, up ? v0 : v1, 4);  // groups (g, g + 2) of the partner
            const uint32_t mine = up ? v1 : v0, g02 = up ? vo : mine, g13 = up ? mine : vo;
            vw = make_uint2(__byte_perm(g02, g13, 0x5410), __byte_perm(g02, g13, 0x7632));
            const uint32_t k_up = __shfl_xor_sync(0xffffffffu, ks, 4), v_up = __shfl_xor_sync(0xffffffffu, vs, 4);
            sk = make_uint2(__byte_perm(ks, k_up, 0x5410), __byte_perm(ks, k_up, 0x7632));
            sv = make_uint2(__byte_perm(vs, v_up, 0x5410), __byte_perm(vs, v_up, 0x7632));
        } else {
            kw = make_uint2(k0, k1);
            vw = make_uint2(v0, v1);
            sk = make_uint2(ks, 0);
            sv = make_uint2(vs, 0);
        }
        if (!store) return;
        const int c = t & 3;
        char* dk = const_cast<char*>(pg.k) + at * (D / 2);
        char* dv = const_cast<char*>(pg.v) + at * (D / 2);
        *reinterpret_cast<uint2*>(dk + (D == 128 ? c * 16 + (t >> 2) * 8 : c * 8)) = kw;
        *reinterpret_cast<uint2*>(dv + (D == 128 ? (2 * c + (t >> 2)) * 8 : c * 8)) = vw;
        if (t == 0) {
            char* ds = const_cast<char*>(pg.ks) + at * (D / 16);
            char* dt = const_cast<char*>(pg.vs) + at * (D / 16);
            if constexpr (D == 128) {
                *reinterpret_cast<uint2*>(ds) = sk;
                *reinterpret_cast<uint2*>(dt) = sv;
            } else {
                *reinterpret_cast<uint32_t*>(ds) = sk.x;
                *reinterpret_cast<uint32_t*>(dt) = sv.x;
            }
        }
    }
}

// U rows of a thread, whose loads are on their way together.
template <typename T, bool I4, int D, int U>
__global__ void __launch_bounds__(MEM_THREADS, !I4 && U == 2 ? 3 : 4)
    k_paged_gather(PageView pg, const int32_t* __restrict__ seq, const int32_t* __restrict__ pos,
                   const int32_t* __restrict__ rot, const int32_t* __restrict__ n_dev, int max_n,
                   long long row0, T* __restrict__ k_out, T* __restrict__ v_out, const float2* __restrict__ tab,
                   int max_pos, int32_t* err) {
    constexpr int TPH = D / 16, HALF = D / 2;
    const int t = threadIdx.x % TPH, i0 = t * 8;
    RowAt r[U];
    long long at[U], row[U];
    int head[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const unsigned unit = (blockIdx.x * U + u) * (MEM_THREADS / TPH) + threadIdx.x / TPH;  // below 2^31 (launcher)
        row[u] = row0 + unit / (unsigned)pg.hkv;
        head[u] = (int)(unit % (unsigned)pg.hkv);
        r[u].read(seq, pos, rot, false, row[u], row[u] < max_n);
    }
    const int n = checked_count(n_dev, max_n, err);
#pragma unroll
    for (int u = 0; u < U; ++u) r[u].find(pg, max_pos, row[u] < n, err);
#pragma unroll
    for (int u = 0; u < U; ++u) at[u] = r[u].place(pg, head[u], err);
    if constexpr (!I4) {
        Raw8<T> ra[U], rb[U], rva[U], rvb[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (r[u].ok) {
                const T* sk = reinterpret_cast<const T*>(pg.k) + at[u] * D;
                const T* sv = reinterpret_cast<const T*>(pg.v) + at[u] * D;
                ra[u].load(sk + i0);
                rb[u].load(sk + i0 + HALF);
                rva[u].load(sv + i0);
                rvb[u].load(sv + i0 + HALF);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (r[u].ok) {
                const long long out = (row[u] * pg.hkv + head[u]) * D;
                rva[u].store(v_out + out + i0);
                rvb[u].store(v_out + out + i0 + HALF);
                float a[8], b[8];
                ra[u].get(a);
                rb[u].get(b);
                rotate8(a, b, r[u].rot, i0, HALF, tab);
                store8(k_out + out + i0, a);
                store8(k_out + out + i0 + HALF, b);
            }
    } else {
        // the layout and the exchange of k_paged_append, backwards
        const int c = t & 3;
        uint2 kw[U], vw[U], sk[U], sv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            kw[u] = vw[u] = sk[u] = sv[u] = make_uint2(0, 0);
            if (r[u].ok) {
                const char* pk = pg.k + at[u] * (D / 2);
                const char* pv = pg.v + at[u] * (D / 2);
                const char* ps = pg.ks + at[u] * (D / 16);
                const char* pt = pg.vs + at[u] * (D / 16);
                kw[u] = *reinterpret_cast<const uint2*>(pk + (D == 128 ? c * 16 + (t >> 2) * 8 : c * 8));
                vw[u] = *reinterpret_cast<const uint2*>(pv + (D == 128 ? (2 * c + (t >> 2)) * 8 : c * 8));
                if constexpr (D == 128) {
                    sk[u] = *reinterpret_cast<const uint2*>(ps);
                    sv[u] = *reinterpret_cast<const uint2*>(pt);
                } else {
                    sk[u].x = *reinterpret_cast<const uint32_t*>(ps);
                    sv[u].x = *reinterpret_cast<const uint32_t*>(pt);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            uint32_t k0, k1, w0, w1;
            float ka, kb, sa, sb;
            if constexpr (D == 128) {
                const bool up = t >= 4;
                const uint32_t ko = __shfl_xor_sync(0xffffffffu, up ? kw[u].x : kw[u].y, 4);
                k0 = up ? ko : kw[u].x;
                k1 = up ? kw[u].y : ko;
                const uint32_t g02 = __byte_perm(vw[u].x, vw[u].y, 0x5410), g13 = __byte_perm(vw[u].x, vw[u].y, 0x7632);
                const uint32_t vo = __shfl_xor_sync(0xffffffffu, up ? g02 : g13, 4);
                const uint32_t v0 = up ? vo : g02, v1 = up ? g13 : vo;  // this thread's groups by half: 2c, 2c + 1
                w0 = __byte_perm(v0, v1, 0x5410);
                w1 = __byte_perm(v0, v1, 0x7632);
                ka = __uint_as_float(up ? sk[u].x & 0xffff0000u : sk[u].x << 16);
                kb = __uint_as_float(up ? sk[u].y & 0xffff0000u : sk[u].y << 16);
                sa = __uint_as_float(up ? sv[u].x & 0xffff0000u : sv[u].x << 16);
                sb = __uint_as_float(up ? sv[u].y & 0xffff0000u : sv[u].y << 16);
            } else {
                k0 = kw[u].x;
                k1 = kw[u].y;
                w0 = __byte_perm(vw[u].x, vw[u].y, 0x5410);
                w1 = __byte_perm(vw[u].x, vw[u].y, 0x7632);
                ka = __uint_as_float(sk[u].x << 16);
                kb = __uint_as_float(sk[u].x & 0xffff0000u);
                sa = __uint_as_float(sv[u].x << 16);
                sb = __uint_as_float(sv[u].x & 0xffff0000u);
            }
            if (!r[u].ok) continue;
            const long long out = (row[u] * pg.hkv + head[u]) * D;
            float a[8], b[8];
            v_values(w0, sa, a);
            v_values(w1, sb, b);
            store8(v_out + out + i0, a);
            store8(v_out + out + i0 + HALF, b);
            k_values(k0, ka, a);
            k_values(k1, kb, b);
            rotate8(a, b, r[u].rot, i0, HALF, tab);
            store8(k_out + out + i0, a);
            store8(k_out + out + i0 + HALF, b);
        }
    }
}

// Rows of one launch: its threads count in 32 bits, and it ends with a whole pair of CTAs, so that no
// thread of it reaches a row of the next one (query heads may be rotated in place, and once only).
long long rows_of_launch(int slots, int d) {
    constexpr long long step = 2 * MEM_THREADS;
    const long long n = (1ll << 31) / ((long long)slots * (d / 16)) / step;
    return (n > 1 ? n : 1) * step;
}

template <typename T, bool I4, int D>
void append_d(const PageView& pg, int hq, const void* k_new, long long ld_k, const void* v_new, long long ld_v,
              const void* q, long long ld_q, void* q_out, const int32_t* seq, const int32_t* pos, const int32_t* rot,
              const int32_t* n_dev, int max_n, const float2* tab, int max_pos, int32_t* err, cudaStream_t s) {
    const int slots = pg.hkv + (q ? hq : 0);
    const long long most = rows_of_launch(slots, D);
    for (long long row0 = 0; row0 < max_n; row0 += most) {
        const long long threads = (max_n - row0 < most ? max_n - row0 : most) * slots * (D / 16);
        k_paged_append<T, I4, D><<<(unsigned)((threads + MEM_THREADS - 1) / MEM_THREADS), MEM_THREADS, 0, s>>>(
            pg, hq, (const T*)k_new, ld_k, (const T*)v_new, ld_v, (const T*)q, ld_q, (T*)q_out, seq, pos, rot, n_dev,
            max_n, row0, tab, max_pos, err);
        note_launch(1);
    }
}
template <typename T, bool I4, int D>
void gather_d(const PageView& pg, const int32_t* seq, const int32_t* pos, const int32_t* rot, const int32_t* n_dev,
              int max_n, void* k_out, void* v_out, const float2* tab, int max_pos, int32_t* err, cudaStream_t s) {
    const long long most = rows_of_launch(pg.hkv, D);
    for (long long row0 = 0; row0 < max_n; row0 += most) {
        const long long threads = (max_n - row0 < most ? max_n - row0 : most) * pg.hkv * (D / 16);
        const long long blocks = (threads + MEM_THREADS - 1) / MEM_THREADS;
        // two rows a thread once that still fills four CTAs on each of 152 SMs
        if (blocks >= 2 * 608)
            k_paged_gather<T, I4, D, 2><<<(unsigned)((blocks + 1) / 2), MEM_THREADS, 0, s>>>(
                pg, seq, pos, rot, n_dev, max_n, row0, (T*)k_out, (T*)v_out, tab, max_pos, err);
        else
            k_paged_gather<T, I4, D, 1><<<(unsigned)blocks, MEM_THREADS, 0, s>>>(
                pg, seq, pos, rot, n_dev, max_n, row0, (T*)k_out, (T*)v_out, tab, max_pos, err);
        note_launch(1);
    }
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
}

}  // namespace blend

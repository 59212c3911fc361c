// 4-bit weights with group scales: packing, reading back, and products for few rows (w4_pack,
// w4_unpack, w4_linear in blend.h).
//
// Products of few rows are bound by reading the codes.  mma.m16n8k16 with 16 weight rows against 8 input
// rows: a lane's sixteen bytes of a 64-byte chunk are its operands of four 32-input steps, so codes go from
// global memory to operands in registers, with one mask and one multiply-add for two of them (code_pair in
// paged.cuh: (code - 8) / 64, exact in bf16; the 64 goes into the sum's end).  The products of a group
// are summed in fp32 by the matrix unit, and one multiply-add per result and group applies the scale: neither
// codes nor scales are rounded.  fp32 inputs enter as three bf16 parts, which hold all 24 bits.
//
// Up to 8 rows come here (the instruction's other side has 8 columns), and fp32 rows of any number.  bf16, against the
// tcgen05 kernel: 8 x 27648 x 5120 (groups of 32, SwiGLU) 22 us and 34; 8 x 152064 x 5120 83 and 123; 8 x 5120 x 13824 19.7
// and 19.5; 9 rows in two blocks of this kernel 36.4 and 34.2 (27648 x 5120, groups of 32), 25.9 and 19.5 (5120 x 13824).
// fp32: 1 x 27648 x 5120 (groups of 32) 25 us, 8 rows 119 (three parts of the inputs, over two CTAs); many rows read all
// codes again for each block of eight rows or fewer, 500 x 5120 x 13824 2.1 ms.
#include "w4.cuh"

namespace blend {
namespace {

// ---------------------------------------------------------------- pack, unpack
// A warp takes a stretch of one row, a lane eight inputs (one word of codes) of it at a time, PACK_U times 32
// words together: loads and stores are whole lines, and nothing is divided to find a place.  Packing 27648 x 5120 bf16 in
// groups of 32 takes 82-83 us (4.4 TB/s), wherever source, codes and scales lie, bound by instruction issue (71 % of slots: a
// maximum, an exact quotient and a code for each weight), fp32 130 us (5.0 TB/s); reading back 57 us (6.4 TB/s), bound by HBM, to
// fp32 141 us (4.6 TB/s: a lane's eight values are two halves of a line).
constexpr int PACK_THREADS = 256, PACK_U = 4;
struct PackPlace {
    int row, w0, w1;  // words w0 .. w1 - 1 of the row, in input order
    __device__ __forceinline__ PackPlace(const W4View& w) {
        row = blockIdx.x * (PACK_THREADS / 32) + (threadIdx.x >> 5);
        const int runs = (w.chunks * 16 + 32 * PACK_U - 1) / (32 * PACK_U);  // of 32 PACK_U words
        w0 = runs * blockIdx.y / gridDim.y * (32 * PACK_U);
        w1 = min((int)(runs * (blockIdx.y + 1) / gridDim.y) * (32 * PACK_U), w.chunks * 16);
    }
};

// Codes 8 + n of eight values as a 32-bit word, see the layout.
//
// n is the exact quotient rounded to an integer.  With y = 1 / s correctly rounded, q = x y, r = x - q s (exact) and
// q + r y is x / s correctly rounded (Markstein's theorem, P. Markstein, IBM J. Res. Dev. 34, 1990) as long as
// nothing leaves the normal range; scales outside 2^-100..2^100 divide.  That fp32 quotient may lie half way
// between two integers where the exact one only lies beside it (not with bf16 inputs, whose quotients by a bf16 keep
// further away): then the remainder tells the side.
template <typename T> __device__ __forceinline__ uint32_t code_word(const float* x, float s) {
    uint32_t c[8];
    if (s >= 0x1p-100f && s <= 0x1p100f) {
        const float y = __frcp_rn(s);
        const float2 y2 = make_float2(y, y), ns2 = make_float2(-s, -s), up2 = make_float2(12582920.f, 12582920.f);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const float2 x2 = make_float2(x[e], x[e + 1]), q = __fmul2_rn(x2, y2);
            float2 d = __ffma2_rn(__ffma2_rn(q, ns2, x2), y2, q);
            if constexpr (sizeof(T) == 4) {
                // half way: a step of the quotient towards the exact one (|n| + 1/2 stays below 2^24)
                const float2 r = __ffma2_rn(d, ns2, x2);
                if (fabsf(d.x - rintf(d.x)) == 0.5f && r.x != 0.f) d.x = nextafterf(d.x, r.x > 0.f ? 100.f : -100.f);
                if (fabsf(d.y - rintf(d.y)) == 0.5f && r.y != 0.f) d.y = nextafterf(d.y, r.y > 0.f ? 100.f : -100.f);
            }
            // |x| / s stays below 7.5, so the code is in range without a clamp; adding 1.5 2^23 rounds to an
            // integer, ties to even (and the 8 keeps its parity)
            const float2 n = __fadd2_rn(d, up2);
            c[e] = __float_as_uint(n.x);
            c[e + 1] = __float_as_uint(n.y);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float n = 0.f;
            if (s > 0.f) {
                const float q = __fdiv_rn(x[e], s), r = fmaf(-q, s, x[e]);
                n = rintf(q);
                if (fabsf(q - n) == 0.5f && r != 0.f) n = r > 0.f ? ceilf(q) : floorf(q);
                n = fminf(fmaxf(n, -7.f), 7.f);
            }
            c[e] = (uint32_t)(8 + (int)n);
        }
    }
    // inputs 0, 2, 4, 6 to the low half, 1, 3, 5, 7 to the high one (what a code carries from bit 22 up stays above)
    const uint32_t lo = c[0] + c[2] * 16u + c[4] * 256u + c[6] * 4096u, hi = c[1] + c[3] * 16u + c[5] * 256u + c[7] * 4096u;
    return __byte_perm(lo, hi, 0x5410);
}

template <typename T>
__global__ void __launch_bounds__(PACK_THREADS)
    k_w4_pack(W4View w, const T* __restrict__ src, long long ld) {
    const PackPlace at(w);
    if (at.row >= w.n) return;
    constexpr int NV = 8 / Vec<T>::N;
    const int lane = threadIdx.x & 31;
    const T* in = src + at.row * ld;
    uint32_t* codes = (uint32_t*)w.codes + (long long)at.row * w.chunks * 16;
    bf16* scale = (bf16*)w.scale + (long long)at.row * w.chunks * (128 / w.group);
    const int k8 = w.k / 8, lanes = w.group / 8, log2_lanes = lanes == 4 ? 2 : lanes == 8 ? 3 : 4;
    for (int w0 = at.w0; w0 < at.w1; w0 += 32 * PACK_U) {
        Vec<T> v[PACK_U][NV];
#pragma unroll
        for (int u = 0; u < PACK_U; ++u) {
            const int i = w0 + u * 32 + lane;
#pragma unroll
            for (int n = 0; n < NV; ++n) v[u][n].raw = i < k8 ? *(const uint4*)(in + i * 8 + n * Vec<T>::N) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < PACK_U; ++u) {
            const int i = w0 + u * 32 + lane;
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = v[u][e / Vec<T>::N].get(e % Vec<T>::N);
            float m = fabsf(x[0]);
#pragma unroll
            for (int e = 1; e < 8; ++e) m = max_nan(m, fabsf(x[e]));
            m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
            if (lanes > 4) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 4));
            if (lanes > 8) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 8));
            // (the fp32 quotient by 7 is never half way between two bf16 unless the exact one is)
            const bf16 sb = __float2bfloat16_rn(isfinite(m) ? __fdiv_rn(m, 7.f) : __int_as_float(0x7fc00000));
            const uint32_t word = code_word<T>(x, __bfloat162float(sb));
            if (i >= at.w1) continue;
            // word 4 part + k32 of its chunk
            codes[(i & ~15) | (i & 3) << 2 | (i >> 2 & 3)] = word;
            if ((i & (lanes - 1)) == 0) scale[i >> log2_lanes] = sb;
        }
    }
}

// A lane reads sixteen bytes (four words, inputs 32 apart) and writes eight values of each.
__device__ __forceinline__ void put_values(bf16* p, uint32_t word, bf16 s) {
    const __nv_bfloat162 s2 = __halves2bfloat162(s, s);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t n = code_ints(word >> (4 * i));
        const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&n), s2);  // exact, rounded once
        o[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ void put_values(float* p, uint32_t word, bf16 sb) {
    const float s = __bfloat162float(sb);
    float o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t n = code_ints(word >> (4 * i));
        o[2 * i] = __fmul_rn(__uint_as_float(n << 16), s);
        o[2 * i + 1] = __fmul_rn(__uint_as_float(n & 0xffff0000u), s);
    }
    *reinterpret_cast<float4*>(p) = make_float4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(o[4], o[5], o[6], o[7]);
}
template <typename T>
__global__ void __launch_bounds__(PACK_THREADS)
    k_w4_unpack(W4View w, T* __restrict__ out, long long ld) {
    const PackPlace at(w);
    if (at.row >= w.n) return;
    const int lane = threadIdx.x & 31, spc = 128 / w.group, log2_spc = spc == 4 ? 2 : spc == 2 ? 1 : 0;
    T* dst = out + at.row * ld;
    const uint4* codes = w.codes + (long long)at.row * w.chunks * 4;
    const bf16* scale = w.scale + (long long)at.row * w.chunks * spc;
    for (int q0 = at.w0 / 4; q0 < at.w1 / 4; q0 += 32) {
        const int q = q0 + lane;  // piece of the row: part q % 4 of chunk q / 4
        if (q >= at.w1 / 4) continue;
        const uint4 v = __ldg(codes + q);
        bf16 s[4];
#pragma unroll
        for (int k32 = 0; k32 < 4; ++k32) s[k32] = scale[(q >> 2 << log2_spc) + (k32 * spc >> 2)];
#pragma unroll
        for (int k32 = 0; k32 < 4; ++k32) {
            const int i = (q >> 2) * 128 + k32 * 32 + (q & 3) * 8;
            if (i < w.k) put_values(dst + i, word_of(v, k32), s[k32]);
        }
    }
}

// ---------------------------------------------------------------- products
constexpr int LIN_WARPS = 16, LIN_THREADS = 32 * LIN_WARPS;
constexpr int LIN_ROWS = 8;         // input rows of a launch block; more of them go to the tcgen05 kernel
constexpr int LIN_RING = 3;         // chunks of 32 weight rows on their way per warp, at most (1 x 5120 x 13824: 15.2 us, with four
                                    // 16.8, since L1 then holds fewer of the scales' sectors)
constexpr int LIN_CODES = 32 * 64, LIN_STAGE = LIN_CODES + 32 * 8;  // bytes of one: codes, and eight bytes of scales a row
constexpr int LIN_MAX_CLUSTER = 8;  // CTAs that share a weight row's inputs
constexpr int LIN_SUMS = 32 * LIN_ROWS;  // results of a unit

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The first product of a group: added to nothing.
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Where a CTA's share of the inputs lies and how its rows are laid out in shared memory: rows of whole
// chunks and 64 bytes more, so that the two rows of a quarter warp's 16-byte reads use different banks.
__host__ __device__ __forceinline__ int lin_row_bytes(int chunks) { return chunks * 256 + 64; }
// A unit is 32 weight rows (two tiles of matrix instructions, for SWIGLU the gate and the up rows of 16 outputs)
// by all input rows.  The warps of a CTA, or each half of them, take a unit's chunks in turn and join their sums at
// its end: two halves work on a unit each where there are enough units, and share the inputs in shared memory.
//
// Codes come by TMA into a ring of each warp (no barrier of the CTA in the loop, 2 KB a copy, swizzled so that lanes
// read them without conflicts); the scales beside them by cp.async onto the same mbarrier.  4 x 152064 x 5120 in
// groups of 64: 79 us, 5.3 TB/s of codes and scales, 78 % of the copy rate; what is left there is issue (66 % of slots: 24
// instructions for a word of codes).  1 x 27648 x 5120 in groups of 32: 19.8 us, 4.0 TB/s: 5-6 us are the start (inputs to
// shared memory, the first codes) and the last units.  Inputs that do not fit beside the rings are split among a
// cluster (8 x 13824 bf16: two CTAs); joining the sums of a unit through distributed shared memory costs 2-3 us, so no
// more CTAs share a row than have to (8 x 5120 x 13824 with two 19.8 us, with four 31).
template <typename T, int G>
__global__ void __launch_bounds__(LIN_THREADS, 1)
    k_w4_linear(const __grid_constant__ CUtensorMap m_codes, const W4Linear a, int cluster, int row_cap, int depth, int halves) {
    constexpr int P = sizeof(T) == 4 ? 3 : 1;  // bf16 parts of an input
    constexpr int SPC = 128 / G, SUMS = LIN_SUMS;
    extern __shared__ __align__(1024) char smem[];
    // full: a chunk of codes has come; p: the sums of a unit of the cluster's CTAs are there, have been read
    __shared__ uint64_t full[LIN_WARPS][LIN_RING], p_full[2][2], p_free[2][2];
    __shared__ int abort_sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), g = lane >> 2, t4 = lane & 3;
    const int rank = blockIdx.y % cluster;
    const int per_half = LIN_WARPS / halves, half = warp / per_half, warp_in = warp - half * per_half;
    const int unit0 = blockIdx.y / cluster + half * (gridDim.y / cluster), units_step = gridDim.y / cluster * halves;
    const int row0 = blockIdx.x * row_cap, rows = min(row_cap, a.rows - row0);
    const int chunks = a.w.chunks;
    const int c0 = chunks * rank / cluster, c1 = chunks * (rank + 1) / cluster;
    const int row_bytes = lin_row_bytes((chunks + cluster - 1) / cluster);
    const int plane = row_cap * row_bytes;
    // rings of codes, [2][LIN_WARPS][SUMS] sums of warps, [2 halves][2][SUMS] of this CTA (cluster > 1), inputs
    char* ring = smem + warp * (depth * LIN_CODES);
    char* scale_ring = smem + LIN_WARPS * depth * LIN_CODES + warp * (depth * 256);
    float* red = (float*)(smem + LIN_WARPS * depth * LIN_STAGE);
    float* part = red + 2 * LIN_WARPS * SUMS;
    char* s_x = (char*)(part + (cluster > 1 ? 4 * SUMS : 0));
    const int units = (a.w.n + 31) / 32;
    const int my_units = unit0 < units ? (units - unit0 + units_step - 1) / units_step : 0;

    // this warp's chunks of a unit: c0 + warp_in, + per_half, ...
    const int per_unit = max(0, (c1 - c0 - warp_in + per_half - 1) / per_half);
    if (lane == 0) {
        for (int i = 0; i < depth; ++i) mbar_init(&full[warp][i], 1 + 32);
        if (warp == 0) {
            abort_sh = 0;
            for (int i = 0; i < 4; ++i) {
                mbar_init(&p_full[i >> 1][i & 1], cluster * per_half);
                mbar_init(&p_free[i >> 1][i & 1], cluster * per_half);
            }
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    int f_unit = 0, f_chunk = 0, asked = 0;  // the next chunk to ask for, and how many have been
    long long at_scale = 0;                  // where the scales of this lane's row begin in it, in bytes
    const long long scale_end = (long long)a.w.n * chunks * (SPC * 2);
    auto fetch = [&](int slot) {
        if (f_unit >= my_units) return;
        const int unit = unit0 + f_unit * units_step;
        if (f_chunk == 0) at_scale = ((long long)min(unit * 32 + lane, a.w.n - 1) * chunks + c0 + warp_in) * (SPC * 2);
        // a row's scales of the chunk; of one alone, the word that it lies in (as much of it as there is)
        const uint32_t to = su32(scale_ring + slot * 256 + lane * 8);
        const char* from = (const char*)a.w.scale + (SPC == 1 ? at_scale & ~3ll : at_scale);
        if constexpr (SPC == 4) asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
        else asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(SPC == 1 && (at_scale & ~3ll) + 4 > scale_end ? 2 : 4) : "memory");
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(su32(&full[warp][slot])) : "memory");
        if (elect_one()) {
            mbar_expect_tx(&full[warp][slot], LIN_CODES);
            tma_2d(ring + slot * LIN_CODES, &m_codes, &full[warp][slot], (c0 + warp_in + f_chunk * per_half) * 64, unit * 32);
        }
        __syncwarp();
        ++asked;
        at_scale += per_half * (SPC * 2);
        if (++f_chunk == per_unit) {
            f_chunk = 0;
            ++f_unit;
        }
    };
    if (per_unit > 0) fetch(0);
    // this CTA's inputs to shared memory, zeros behind k
    {
        const int vecs = (c1 - c0) * 16;  // of eight inputs
        for (int r = 0; r < rows; ++r) {
            const T* src = (const T*)a.x + (long long)(row0 + r) * a.ld_x + c0 * 128;
            char* dst = s_x + r * row_bytes;
            if constexpr (P == 1) {
                for (int v = tid; v < vecs; v += LIN_THREADS) {
                    const int bytes = c0 * 128 + v * 8 < a.w.k ? 16 : 0;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(su32(dst + v * 16)), "l"(bytes ? src + v * 8 : (const T*)a.x), "r"(bytes) : "memory");
                }
            } else {
#pragma unroll 2
                for (int v = tid; v < vecs; v += LIN_THREADS) {
                    const bool in = c0 * 128 + v * 8 < a.w.k;
                    float4 f[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) f[h] = in ? *(const float4*)(src + v * 8 + h * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
                    const float* x = (const float*)f;
                    uint32_t w[P][4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x0 = x[2 * e], x1 = x[2 * e + 1];
#pragma unroll
                        for (int p = 0; p < P; ++p) {
                            const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
                            w[p][e] = *(const uint32_t*)&h;
                            x0 -= __low2float(h);
                            x1 -= __high2float(h);
                        }
                    }
#pragma unroll
                    for (int p = 0; p < P; ++p) *(uint4*)(dst + p * plane + v * 16) = make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
                }
            }
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (per_unit > 0)
        for (int i = 1; i < depth; ++i) fetch(i);
    asm volatile("cp.async.wait_group 0;" ::: "memory");  // (the last scales are in no group yet)
    __syncthreads();
    if (cluster > 1) cluster_sync();  // all CTAs' barriers exist

    // lanes of rows that are not there read the last one's (their columns are not stored)
    const char* x_at = s_x + min(g, rows - 1) * row_bytes + t4 * 16 + warp_in * 256;

    float acc[2][4];
    auto expired = [&]() {
        // (the results would be wrong: the error word tells)
        set_error(a.err, BLEND_ETIMEOUT);
        abort_sh = 1;
        f_unit = my_units;
    };
    const int in_half = tid - half * per_half * 32, threads = per_half * 32;
    // The warps' sums of unit number i joined in order, and its results written (by as many threads as there are).
    auto finish = [&](int i) {
        const int b = i & 1;
        float* all = red + (b * LIN_WARPS + half * per_half) * SUMS;
#pragma unroll
        for (int m = 0; m < 2; ++m) *(float4*)(all + warp_in * SUMS + m * 128 + lane * 4) = make_float4(acc[m][0], acc[m][1], acc[m][2], acc[m][3]);
        asm volatile("barrier.sync %0, %1;" ::"r"(half + 1), "r"(threads) : "memory");
        // weight row m of tile t and input row col
        auto place = [&](int t, int m, int col) { return t * 128 + ((m & 7) * 4 + (col >> 1)) * 4 + (m >> 3) * 2 + (col & 1); };
        auto warps_sum = [&](int o) {
            float v = 0.f;
#pragma unroll 8
            for (int w = 0; w < per_half; ++w) v += all[w * SUMS + o];
            return v;
        };
        float* sums = part + (half * 2 + b) * SUMS;
        if (cluster > 1) {
            const uint32_t par = i >> 1 & 1;
            if (!cluster_phase(&p_free[half][b], par ^ 1, &abort_sh)) expired();
            for (int o = in_half; o < 32 * rows; o += threads) {
                const int at = place(o >> 4 & 1, o & 15, o >> 5);
                sums[at] = warps_sum(at);
            }
            meet(&p_full[half][b], 0, cluster);
            if (!cluster_phase(&p_full[half][b], par, &abort_sh)) expired();
        }
        auto value = [&](int t, int m, int col) {
            const int at = place(t, m, col);
            float v = 0.f;
            if (cluster > 1) {
                for (int c = 0; c < cluster; ++c) v += ld_peer(peer_addr(sums + at, c));
            } else
                v = warps_sum(at);
            return v * CODE_UNIT;
        };
        // neighbouring threads: neighbouring weight rows of one input row
        const int unit = unit0 + i * units_step;
        if (a.epi == BLEND_W4_SWIGLU) {
            const int o1 = 16 * rows * (rank + 1) / cluster;
            for (int o = 16 * rows * rank / cluster + in_half; o < o1; o += threads) {
                const int m = o & 15, col = o >> 4;
                const float gate = value(0, m, col), up = value(1, m, col);
                const float y = gate / (1.f + expf(-gate)) * up;
                const long long at = (long long)(row0 + col) * a.ld_y + unit * 16 + m;
                if (a.y_f32) ((float*)a.y)[at] = y;
                else ((bf16*)a.y)[at] = __float2bfloat16_rn(y);
            }
        } else {
            const int o1 = 32 * rows * (rank + 1) / cluster;
            for (int o = 32 * rows * rank / cluster + in_half; o < o1; o += threads) {
                const int m = o & 31, col = o >> 5, j = unit * 32 + m;
                const float v = value(m >> 4, m & 15, col);
                if (j >= a.w.n) continue;
                const long long at = (long long)(row0 + col) * a.ld_y + j;
                if (a.epi == BLEND_W4_ADD) ((float*)a.y)[at] += v;
                else if (a.y_f32) ((float*)a.y)[at] = v;
                else ((bf16*)a.y)[at] = __float2bfloat16_rn(v);
            }
        }
        __syncwarp();
        if (cluster > 1) meet(&p_free[half][b], 0, cluster);
    };

    int slot = 0;
    uint32_t phase = 0;
    // lane (g, t4): piece t4 of rows g, g + 8, g + 16, g + 24 (64-byte swizzle: rows 8 apart alike)
    const char* my_codes = ring + g * 64 + ((t4 ^ (g >> 1 & 3)) << 4);
    // (one copy of the loop's code: unrolled over the ring, fetching it took a fifth of the time)
#pragma unroll 1
    for (int unit = 0; unit < my_units; ++unit) {
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i >> 2][i & 3] = 0.f;
#pragma unroll 1
        for (int chunk = 0; chunk < per_unit; ++chunk) {
            if (!__all_sync(0xffffffffu, mbar_wait(&full[warp][slot], phase, &abort_sh))) expired();
            const char* x_chunk = x_at + chunk * per_half * 256;
            uint4 q[4];
            Scales<G> sc[4];
            // (rows 8 apart: their scales lie alike in their words)
            const int odd = (g * chunks + c0 + warp_in + chunk * per_half) & 1;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                q[i] = *(const uint4*)(my_codes + slot * LIN_CODES + i * 512);
                sc[i].load_shared(scale_ring + slot * 256 + (g + 8 * i) * 8, odd);
            }
            // groups that begin behind k have no scale (a chunk's first never does)
            const int live = a.w.k - (c0 + warp_in + chunk * per_half) * 128;
            float grp[2][4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint32_t lo[2][4], hi[2][4];
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const uint32_t ca = word_of(q[2 * m], w), cb = word_of(q[2 * m + 1], w);
                    lo[m][0] = code_pair<false>(ca);
                    lo[m][1] = code_pair<false>(cb);
                    lo[m][2] = code_pair<true>(ca);
                    lo[m][3] = code_pair<true>(cb);
                    hi[m][0] = code_pair<false>(ca >> 8);
                    hi[m][1] = code_pair<false>(cb >> 8);
                    hi[m][2] = code_pair<true>(ca >> 8);
                    hi[m][3] = code_pair<true>(cb >> 8);
                }
#pragma unroll
                for (int p = P - 1; p >= 0; --p) {
                    const uint4 x = *(const uint4*)(x_chunk + p * plane + w * 64);
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        if (w % (G / 32) == 0 && p == P - 1) mma_first(grp[m], lo[m], x.x, x.y);
                        else mma(grp[m], lo[m], x.x, x.y);
                        mma(grp[m], hi[m], x.z, x.w);
                    }
                }
                if (w % (G / 32) == G / 32 - 1) {
                    float s[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[i] = G == 128 || w * 32 / G * G < live ? sc[i].get(w * 32 / G) : 0.f;
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        acc[m][0] = fmaf(s[2 * m], grp[m][0], acc[m][0]);
                        acc[m][1] = fmaf(s[2 * m], grp[m][1], acc[m][1]);
                        acc[m][2] = fmaf(s[2 * m + 1], grp[m][2], acc[m][2]);
                        acc[m][3] = fmaf(s[2 * m + 1], grp[m][3], acc[m][3]);
                    }
                }
            }
            __syncwarp();  // all lanes have read the slot
            fetch(slot);
            if (++slot == depth) {
                slot = 0;
                phase ^= 1;
            }
        }
        finish(unit);
    }
    if (*(volatile int*)&abort_sh) {
        // after a wait that ran out: the copies still on their way
        int never = 0;
        for (int i = max(0, asked - depth); i < asked; ++i) mbar_wait(&full[warp][i % depth], i / depth & 1, &never);
    }
    if (cluster > 1) {
        __syncwarp();
        cluster_sync();  // the others may still read this CTA's sums
    }
}

PFN_cuTensorMapEncodeTiled_v12000 g_enc = nullptr;

bool encode(CUtensorMap* map, CUtensorMapDataType dt, const void* base, cuuint64_t inner, cuuint64_t outer, cuuint64_t stride,
            cuuint32_t box_inner, cuuint32_t box_outer, CUtensorMapSwizzle swizzle) {
    if (!g_enc) {
        cudaDriverEntryPointQueryResult qr;
        void* fn = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &qr) != cudaSuccess ||
            qr != cudaDriverEntryPointSuccess || !fn) {
            cudaGetLastError();
            return false;
        }
        g_enc = (PFN_cuTensorMapEncodeTiled_v12000)fn;
    }
    const cuuint64_t dims[2] = {inner, outer}, strides[1] = {stride};
    const cuuint32_t box[2] = {box_inner, box_outer}, es[2] = {1, 1};
    return g_enc(map, dt, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int G> int go(const W4Linear& a, cudaStream_t s) {
    constexpr int P = sizeof(T) == 4 ? 3 : 1;
    constexpr int SMEM_MAX = 225 * 1024;
    auto* kern = k_w4_linear<T, G>;
    struct Set {
        bool ok = false;
    };
    static PerDevice<Set> set;
    if (!set.get([&] { return Set{cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MAX) == cudaSuccess}; }))
        return BLEND_ECUDA;
    // Input rows of a launch block, CTAs that share a weight row's inputs and chunks on their way per warp: the
    // first of them that fit in shared memory, fewer chunks before more CTAs before fewer rows.
    const int units = (a.w.n + 31) / 32;
    int cluster = 0, depth = 0, row_cap = a.rows < LIN_ROWS ? a.rows : LIN_ROWS;
    size_t smem = 0;
    for (;; row_cap = (row_cap + 1) / 2) {
        for (int c = 1; c <= LIN_MAX_CLUSTER && c <= a.w.chunks && !cluster; c *= 2)
            for (int d = LIN_RING; d >= 2 && !cluster; --d) {
                smem = (size_t)LIN_WARPS * d * LIN_STAGE + (size_t)(2 * LIN_WARPS + (c > 1 ? 4 : 0)) * LIN_SUMS * 4 +
                       (size_t)P * row_cap * lin_row_bytes((a.w.chunks + c - 1) / c);
                if (smem <= SMEM_MAX) {
                    cluster = c;
                    depth = d;
                }
            }
        if (cluster || row_cap == 1) break;
    }
    if (!cluster) return BLEND_EUNSUPPORTED;
    const int row_blocks = (a.rows + row_cap - 1) / row_cap, fit = 152 / cluster / row_blocks > 0 ? 152 / cluster / row_blocks : 1;
    // halves with a unit each: where whole CTAs would need a second round anyway (1 x 27648 x 5120 20.8 us for 24.0; 1 x 4096 x
    // 14336, one round of whole CTAs, 11.2 for 10.8)
    const int halves = units > fit ? 2 : 1;
    const int clusters = std::min(units, fit);
    // (no more on their way than a warp has: small calls start sooner with less shared memory)
    const int of_warp = (units + clusters * halves - 1) / (clusters * halves) *
                        (((a.w.chunks + cluster - 1) / cluster + LIN_WARPS / halves - 1) / (LIN_WARPS / halves));
    if (of_warp < depth) {
        smem -= (size_t)LIN_WARPS * (depth - of_warp) * LIN_STAGE;
        depth = of_warp;
    }
    CUtensorMap mc;
    if (!w4_encode_codes(&mc, a.w, 32)) return BLEND_EUNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)row_blocks, (unsigned)(clusters * cluster));  // (row blocks may pass 65535)
    cfg.blockDim = dim3(LIN_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.y = (unsigned)cluster;
    attr.val.clusterDim.x = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, kern, mc, a, cluster, row_cap, depth, halves) != cudaSuccess) return BLEND_ECUDA;
    note_launch();
    return BLEND_OK;
}
template <typename T> int go_group(const W4Linear& a, cudaStream_t s) {
    return a.w.group == 32 ? go<T, 32>(a, s) : a.w.group == 64 ? go<T, 64>(a, s) : go<T, 128>(a, s);
}

// Rows, and parts of a row where they are few: warps for 152 SMs of 32.
dim3 pack_grid(const W4View& w) {
    const int blocks = (w.n + PACK_THREADS / 32 - 1) / (PACK_THREADS / 32), runs = (w.chunks * 16 + 32 * PACK_U - 1) / (32 * PACK_U);
    int parts = (152 * 4 + blocks - 1) / blocks;
    parts = parts < runs ? parts : runs;
    return dim3((unsigned)blocks, (unsigned)parts);
}

}  // namespace

bool w4_encode_codes(CUtensorMap* map, const W4View& w, int rows) {
    const cuuint64_t bytes = (cuuint64_t)w.chunks * 64;
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, w.codes, bytes, (cuuint64_t)w.n, bytes, 64, (cuuint32_t)rows, CU_TENSOR_MAP_SWIZZLE_64B);
}
bool w4_encode_inputs(CUtensorMap* map, const W4Linear& a, int rows) {
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.x, (cuuint64_t)a.w.k, (cuuint64_t)a.rows, (cuuint64_t)a.ld_x * 2, 64, (cuuint32_t)rows,
                  CU_TENSOR_MAP_SWIZZLE_128B);
}

void launch_w4_pack(int dtype, const W4View& w, const void* src, long long ld, cudaStream_t s) {
    if (dtype == BLEND_BF16) k_w4_pack<bf16><<<pack_grid(w), PACK_THREADS, 0, s>>>(w, (const bf16*)src, ld);
    else k_w4_pack<float><<<pack_grid(w), PACK_THREADS, 0, s>>>(w, (const float*)src, ld);
    note_launch();
}
void launch_w4_unpack(int dtype, const W4View& w, void* out, long long ld, cudaStream_t s) {
    if (dtype == BLEND_BF16) k_w4_unpack<bf16><<<pack_grid(w), PACK_THREADS, 0, s>>>(w, (bf16*)out, ld);
    else k_w4_unpack<float><<<pack_grid(w), PACK_THREADS, 0, s>>>(w, (float*)out, ld);
    note_launch();
}

int launch_w4_linear(int dtype, const W4Linear& a, cudaStream_t s) {
    if (dtype == BLEND_BF16 && a.tc && a.rows > LIN_ROWS && a.w.n >= 128 && a.w.k >= 64) {
        const int rc = launch_w4_tile(a, s);
        if (rc != BLEND_EUNSUPPORTED) return rc;
    }
    return dtype == BLEND_BF16 ? go_group<bf16>(a, s) : go_group<float>(a, s);
}

}  // namespace blend

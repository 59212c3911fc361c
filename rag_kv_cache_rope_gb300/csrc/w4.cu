// 4-bit weights with group scales: packing, reading back, and products for few rows (w4_pack,
// w4_unpack, w4_linear in blend.h).
//
// Products of few rows are bound by reading the codes.  mma.m16n8k16 with 16 weight rows against 8 input
// rows: a lane's sixteen bytes of a 64-byte chunk are its operands of four 32-input steps, so codes go from
// global memory to operands in registers, with one mask and one multiply-add for two of them (code_pair in
// paged.cuh: (code - 8) / 64, exact in bf16; the 64 goes into the sum's end).  The products of a group
// are summed in fp32 by the matrix unit, and one multiply-add per result and group applies the scale: neither
// codes nor scales are rounded.  fp32 inputs enter as three bf16 parts, which hold all 24 bits.
#include <cooperative_groups.h>

#include "w4.cuh"

namespace cg = cooperative_groups;

namespace blend {
namespace {

// ---------------------------------------------------------------- pack, unpack
// A warp takes a stretch of one row, a lane eight inputs (one word of codes) of it at a time, PACK_U times 32
// words together: loads and stores are whole lines, and nothing is divided to find a place.
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
constexpr int LIN_WARPS = 8, LIN_THREADS = 32 * LIN_WARPS;
constexpr int LIN_RING = 4;         // chunks on their way per warp
constexpr int LIN_TILE_ROWS = 16;   // more rows of inputs go to the tcgen05 kernel
constexpr int LIN_MAX_CLUSTER = 8;  // CTAs that share a weight row's inputs

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Where a CTA's share of the inputs lies and how its rows are laid out in shared memory: rows of whole
// chunks and 64 bytes more, so that the two rows of a quarter warp's 16-byte reads use different banks.
__host__ __device__ __forceinline__ int lin_row_bytes(int chunks) { return chunks * 256 + 64; }

template <typename T, int NT, int G>
__global__ void __launch_bounds__(LIN_THREADS, 2)
    k_w4_linear(const W4Linear a, int cluster, int row_cap) {
    constexpr int P = sizeof(T) == 4 ? 3 : 1;  // bf16 parts of an input
    constexpr int COLS = 8 * NT, SPC = 128 / G;
    extern __shared__ __align__(128) char smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
    const int rank = cluster > 1 ? (int)cg::this_cluster().block_rank() : 0;
    const int unit0 = blockIdx.x / cluster, units_step = gridDim.x / cluster;
    const int row0 = blockIdx.y * COLS, rows = min(COLS, a.rows - row0);
    const int c0 = (int)((long long)a.w.chunks * rank / cluster), c1 = (int)((long long)a.w.chunks * (rank + 1) / cluster);
    const int row_bytes = lin_row_bytes((a.w.chunks + cluster - 1) / cluster);
    const int plane = row_cap * row_bytes;
    float* red = (float*)(smem + P * plane);              // [2][LIN_WARPS][NT][128]
    float* part = red + 2 * LIN_WARPS * NT * 128;         // [2][NT][128]: this CTA's sums (cluster > 1)

    // tiles of 16 weight rows: a gate tile, then its up tile
    const bool glu = a.epi == BLEND_W4_SWIGLU;
    const int tiles = (a.w.n + 15) / 16;
    const int units = glu ? tiles / 2 : tiles;
    const int my_units = unit0 < units ? (units - unit0 + units_step - 1) / units_step : 0;
    const int my_tiles = glu ? 2 * my_units : my_units;
    auto tile_at = [&](int i) { return glu ? 2 * (unit0 + (i >> 1) * units_step) + (i & 1) : unit0 + i * units_step; };

    // this warp's chunks of a tile: c0 + warp, + LIN_WARPS, ...
    const int per_tile = max(0, (c1 - c0 - warp + LIN_WARPS - 1) / LIN_WARPS);
    uint4 qa[LIN_RING], qb[LIN_RING];
    Scales<G> sa[LIN_RING], sb[LIN_RING];
    int f_tile = 0, f_chunk = 0;  // the next chunk to ask for
    auto fetch = [&](int slot) {
        if (f_tile >= my_tiles) return;
        const int tile = tile_at(f_tile), c = c0 + warp + f_chunk * LIN_WARPS;
        const long long ra = min(tile * 16 + g, a.w.n - 1), rb = min(tile * 16 + g + 8, a.w.n - 1);
        qa[slot] = __ldg(a.w.codes + (ra * a.w.chunks + c) * 4 + t4);
        qb[slot] = __ldg(a.w.codes + (rb * a.w.chunks + c) * 4 + t4);
        sa[slot].load(a.w.scale + (ra * a.w.chunks + c) * SPC);
        sb[slot].load(a.w.scale + (rb * a.w.chunks + c) * SPC);
        if (++f_chunk == per_tile) {
            f_chunk = 0;
            ++f_tile;
        }
    };
    if (per_tile > 0) {
#pragma unroll
        for (int i = 0; i < LIN_RING; ++i) fetch(i);
    }

    // this CTA's inputs to shared memory, zeros behind k
    {
        const int vecs = (c1 - c0) * 16;  // of eight inputs
        for (int i = tid; i < rows * vecs; i += LIN_THREADS) {
            const int r = i / vecs, v = i - r * vecs, at = c0 * 128 + v * 8;
            char* dst = smem + r * row_bytes + v * 16;
            const T* src = (const T*)a.x + (long long)(row0 + r) * a.ld_x + at;
            if constexpr (P == 1) {
                *(uint4*)dst = at < a.w.k ? *(const uint4*)src : make_uint4(0, 0, 0, 0);
            } else {
                uint32_t w[P][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float2 x = at < a.w.k ? *(const float2*)(src + 2 * e) : make_float2(0.f, 0.f);
#pragma unroll
                    for (int p = 0; p < P; ++p) {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
                        w[p][e] = *(const uint32_t*)&h;
                        x.x -= __low2float(h);
                        x.y -= __high2float(h);
                    }
                }
#pragma unroll
                for (int p = 0; p < P; ++p) *(uint4*)(dst + p * plane) = make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
            }
        }
    }
    __syncthreads();

    // lanes of rows that are not there read the last one's (their columns are not stored)
    int x_at[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) x_at[nt] = min(nt * 8 + g, rows - 1) * row_bytes + t4 * 16;

    float acc[NT][4];
    auto clear = [&]() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[nt][i] = 0.f;
    };
    float gate[(NT * 128 + LIN_THREADS - 1) / LIN_THREADS];
    // The warps' sums of tile number i joined in order, and its results written.
    auto finish = [&](int i) {
        float* mine = red + (i & 1) * (LIN_WARPS * NT * 128);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) *(float4*)(mine + (warp * NT + nt) * 128 + lane * 4) = make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
        clear();
        // (warps come here from different places: a barrier by number, not by place)
        asm volatile("barrier.sync 0;" ::: "memory");
        float* sums = part + (i & 1) * (NT * 128);
        const int tile = tile_at(i);
        auto warps_sum = [&](int o) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < LIN_WARPS; ++w) v += mine[w * NT * 128 + o];
            return v;
        };
        if (cluster > 1) {
            for (int o = tid; o < NT * 128; o += LIN_THREADS) sums[o] = warps_sum(o);
            cg::this_cluster().sync();
        }
        const int o0 = NT * 128 * rank / cluster, o1 = NT * 128 * (rank + 1) / cluster;
#pragma unroll
        for (int u = 0; u < (int)(sizeof(gate) / sizeof(float)); ++u) {
            const int q = o0 + u * LIN_THREADS + tid;
            if (q >= o1) break;
            // neighbouring threads: neighbouring weight rows of one input row
            const int m = q & 15, col = (q >> 4) & 7, nt = q >> 7;
            const int o = nt * 128 + ((m & 7) * 4 + (col >> 1)) * 4 + (m >> 3) * 2 + (col & 1);
            float v = 0.f;
            if (cluster > 1) {
                for (int c = 0; c < cluster; ++c) v += cg::this_cluster().map_shared_rank(sums, c)[o];
            } else
                v = warps_sum(o);
            v *= CODE_UNIT;
            const int r = nt * 8 + col, j = tile * 16 + m;
            if (r >= rows || j >= a.w.n) continue;
            const long long at = (long long)(row0 + r) * a.ld_y;
            if (glu) {
                if ((i & 1) == 0) {
                    gate[u] = v;
                    continue;
                }
                const float y = gate[u] / (1.f + __expf(-gate[u])) * v;
                const long long jj = at + (tile >> 1) * 16 + m;
                if (a.y_f32) ((float*)a.y)[jj] = y;
                else ((bf16*)a.y)[jj] = __float2bfloat16_rn(y);
            } else if (a.epi == BLEND_W4_ADD)
                ((float*)a.y)[at + j] += v;
            else if (a.y_f32)
                ((float*)a.y)[at + j] = v;
            else
                ((bf16*)a.y)[at + j] = __float2bfloat16_rn(v);
        }
        __syncwarp();
    };

    clear();
    if (per_tile == 0) {
        for (int i = 0; i < my_tiles; ++i) finish(i);
    } else {
        int tile = 0, chunk = 0;
        while (tile < my_tiles) {
#pragma unroll
            for (int slot = 0; slot < LIN_RING; ++slot) {
                if (tile >= my_tiles) break;
                const int c = c0 + warp + chunk * LIN_WARPS;
                const uint4 wa = qa[slot], wb = qb[slot];
                const Scales<G> ka = sa[slot], kb = sb[slot];
                fetch(slot);
                const char* xs = smem + (c - c0) * 256;
                float grp[NT][4];
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    if (w % (G / 32) == 0) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int i = 0; i < 4; ++i) grp[nt][i] = 0.f;
                    }
                    const uint32_t ca = word_of(wa, w), cb = word_of(wb, w);
                    const uint32_t a0[4] = {code_pair<false>(ca), code_pair<false>(cb), code_pair<true>(ca), code_pair<true>(cb)};
                    const uint32_t a1[4] = {code_pair<false>(ca >> 8), code_pair<false>(cb >> 8), code_pair<true>(ca >> 8), code_pair<true>(cb >> 8)};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int p = P - 1; p >= 0; --p) {
                            const uint4 x = *(const uint4*)(xs + p * plane + x_at[nt] + w * 64);
                            mma(grp[nt], a0, x.x, x.y);
                            mma(grp[nt], a1, x.z, x.w);
                        }
                    if (w % (G / 32) == G / 32 - 1) {
                        // a group behind k has no scale
                        const bool live = (c * 128 + w * 32) / G * G < a.w.k;
                        const float s0 = live ? ka.get(w * 32 / G) : 0.f, s1 = live ? kb.get(w * 32 / G) : 0.f;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            acc[nt][0] = fmaf(s0, grp[nt][0], acc[nt][0]);
                            acc[nt][1] = fmaf(s0, grp[nt][1], acc[nt][1]);
                            acc[nt][2] = fmaf(s1, grp[nt][2], acc[nt][2]);
                            acc[nt][3] = fmaf(s1, grp[nt][3], acc[nt][3]);
                        }
                    }
                }
                if (++chunk == per_tile) {
                    finish(tile);
                    chunk = 0;
                    ++tile;
                }
            }
        }
    }
    if (cluster > 1) cg::this_cluster().sync();  // the others may still read this CTA's sums
}

template <typename T, int NT, int G> int go(const W4Linear& a, cudaStream_t s) {
    constexpr int P = sizeof(T) == 4 ? 3 : 1;
    constexpr int SMEM_MAX = 224 * 1024;
    auto* kern = k_w4_linear<T, NT, G>;
    static const cudaError_t set = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MAX);
    if (set != cudaSuccess) return BLEND_ECUDA;
    const int row_cap = a.rows < 8 * NT ? a.rows : 8 * NT;
    // CTAs that share a weight row: until the inputs' share leaves room for two CTAs per SM, and until there
    // are tiles for all SMs
    const int tiles = a.epi == BLEND_W4_SWIGLU ? a.w.n / 32 : (a.w.n + 15) / 16;
    int cluster = 1;
    auto bytes = [&](int c) {
        return (size_t)P * row_cap * lin_row_bytes((a.w.chunks + c - 1) / c) + (size_t)(2 * LIN_WARPS + 2) * NT * 128 * 4;
    };
    while (cluster < LIN_MAX_CLUSTER && (bytes(cluster) > SMEM_MAX / 2 || (tiles * cluster < 304 && a.w.chunks / (2 * cluster) >= LIN_WARPS)))
        cluster *= 2;
    const size_t smem = bytes(cluster);
    if (smem > SMEM_MAX) return BLEND_EUNSUPPORTED;
    const int row_blocks = (a.rows + 8 * NT - 1) / (8 * NT);
    int clusters = 152 * 2 / cluster;
    clusters = clusters < tiles ? clusters : tiles;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * cluster), (unsigned)row_blocks);
    cfg.blockDim = dim3(LIN_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, kern, a, cluster, row_cap) != cudaSuccess) return BLEND_ECUDA;
    note_launch();
    return BLEND_OK;
}
template <typename T, int NT> int go_group(const W4Linear& a, cudaStream_t s) {
    return a.w.group == 32 ? go<T, NT, 32>(a, s) : a.w.group == 64 ? go<T, NT, 64>(a, s) : go<T, NT, 128>(a, s);
}

// Rows, and parts of a row where they are few: warps for 152 SMs of 32.
dim3 pack_grid(const W4View& w) {
    const int blocks = (w.n + PACK_THREADS / 32 - 1) / (PACK_THREADS / 32), runs = (w.chunks * 16 + 32 * PACK_U - 1) / (32 * PACK_U);
    int parts = (152 * 4 + blocks - 1) / blocks;
    parts = parts < runs ? parts : runs;
    return dim3((unsigned)blocks, (unsigned)parts);
}

}  // namespace

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
    if (dtype == BLEND_BF16 && a.tc && a.rows > LIN_TILE_ROWS && a.w.n >= 128 && a.w.k >= 64) {
        const int rc = launch_w4_tile(a, s);
        if (rc != BLEND_EUNSUPPORTED) return rc;
    }
    if (dtype == BLEND_BF16) return a.rows <= 8 ? go_group<bf16, 1>(a, s) : go_group<bf16, 2>(a, s);
    return go_group<float, 1>(a, s);
}

}  // namespace blend

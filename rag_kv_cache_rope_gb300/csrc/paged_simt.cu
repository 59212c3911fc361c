// Attention over a paged cache on CUDA cores (paged_attention in blend.h): every page form and
// element type, fp32 throughout.  fp32 models run here (their 1e-4 parity has no room for bf16
// products), and bf16 models with tensor cores switched off.
//
//   o = sum_j 2^(c q.k_j - m) v_j / sum_j 2^(c q.k_j - m),  c = log2(e) / sqrt(d), m the running maximum
//
// A CTA takes one tile of SR (row, head) pairs of one kv head (1, 4 or 8: no more than a sequence's rows
// fill, since empty places cost as much as others) and one of `splits` shares of the keys they see; its
// eight warps take 32-key blocks in turn, each with its own running maximum, sums and outputs in
// registers, and join through shared memory.  With splits > 1 the
// joined results go to the workspace, and the CTA that arrives last at the item's counter joins
// them in split order, so the result does not depend on the order of arrival.
// Bound by latency and issue, not bandwidth.  Measured (GB300, 6.8 TB/s copy rate, fp32, in a captured
// graph): 32 tokens over 2000 each, 32 heads over 8 x 128, 103 us (75 % of the copy rate); one over 64 K with
// 40 heads 250 (32 %); two over 11-64 K, 9 heads over 3 x 64, 76 (39 %); 4-bit pages, 27 behind a window of
// 159, 9 heads over 3 x 64, 21.  Values are loaded four keys at a time without a branch between them (203, 340 and 105 us one by
// one).  Before that: tiles of eight for four pairs 439 instead of 241; one CTA per SM, with the 144
// registers that the compiler takes unasked for eight pairs, 566 instead of 339; d = 64 with three and two
// CTAs per SM 160 and 183 instead of 104; 4-bit pages with two 38.  Keys come sixteen at a time in the same
// way for up to four pairs (117 and 78 before); two times four for eight pairs spills (2.5 ms instead of 1.4
// for two pieces of 200 rows).
// Keys that no row of the tile sees are never loaded, and a weight of zero adds nothing, so what
// lies in masked slots (an infinity, a NaN) has no effect on any row.
#include "paged.cuh"

namespace blend {
namespace {

constexpr int SW = 8;      // warps
constexpr int SKEYS = 32;  // keys of a warp's block

// Four dims 4 i4 .. +3 of a K row / of a V row as fp32.
template <typename T, bool I4, int D> struct Row;
template <int D> struct Row<float, false, D> {
    static __device__ __forceinline__ void k4(const char* p, long long row, int i4, float, float* x) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(p + row * D * 4) + i4);
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    }
    static __device__ __forceinline__ void v4(const char* p, long long row, int i4, float, float* x) { k4(p, row, i4, 0.f, x); }
};
template <int D> struct Row<bf16, false, D> {
    static __device__ __forceinline__ void k4(const char* p, long long row, int i4, float, float* x) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(p + row * D * 2) + i4);
        x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xffff0000u);
        x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xffff0000u);
    }
    static __device__ __forceinline__ void v4(const char* p, long long row, int i4, float, float* x) { k4(p, row, i4, 0.f, x); }
};
template <typename T, int D> struct Row<T, true, D> {
    static __device__ __forceinline__ void k4(const char* p, long long row, int i4, float sc, float* x) {
        const int g = i4 >> 3, e8 = i4 & 7;  // dims 32 g + 4 e8 ..
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(p + row * (D / 2) + k4_word(D, g, e8 >> 1)));
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = sc * (float)((int)((w >> k4_bit(4 * (e8 & 1) + e)) & 15u) - 8);
    }
    static __device__ __forceinline__ void v4(const char* p, long long row, int i4, float sc, float* x) {
        const int g = i4 >> 3, r = i4 & 7;
        const uint32_t w = __ldg(reinterpret_cast<const uint16_t*>(p + row * (D / 2) + v4_half(D, g, r)));
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = sc * (float)((int)((w >> (4 * e)) & 15u) - 8);
    }
};
template <bool I4, int D> __device__ __forceinline__ float scale_of(const char* p, long long row, int i4) {
    return I4 ? __bfloat162float(__ldg(reinterpret_cast<const bf16*>(p) + row * (D / 32) + (i4 >> 3))) : 1.f;
}

// The tile with index `tile` among all sequences' tiles of SR pairs: its sequence and its index
// there; seq -1 when there are fewer.  All threads of the CTA take part.
struct Found {
    int seq, tile;
};
template <int SR>
__device__ __forceinline__ Found find_tile(const PagedAttn& a, int tile, int* sh) {
    constexpr int CAP = (1 << 30) - 1;  // a sequence has at most 2^26 tiles, a launch 2^26 + 1024
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    if (t == 0) sh[SW] = -1;
    int base = 0;
    for (int s0 = 0; s0 < a.pg.n_seq; s0 += SW * 32) {
        const int s = s0 + t;
        const int mine = s < a.pg.n_seq ? (seq_info(a, s).n_q * a.group + SR - 1) / SR : 0;
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl = add_capped(incl, y, CAP);
        }
        if (lane == 31) sh[warp] = incl;
        __syncthreads();
        int before = base, all = base;
        for (int w = 0; w < SW; ++w) {
            if (w < warp) before = add_capped(before, sh[w], CAP);
            all = add_capped(all, sh[w], CAP);
        }
        const int excl = before + incl - mine;
        if (tile >= excl && tile < excl + mine) {
            sh[SW] = s;
            sh[SW + 1] = tile - excl;
        }
        __syncthreads();
        base = all;
        if (tile < base) break;
    }
    return Found{sh[SW], sh[SW + 1]};
}

// CTAs that an SM should hold: loads in flight against registers, as measured (fp32 models, GB300; see above).
constexpr int simt_ctas(bool i4, int d, int sr) { return sr == 8 ? 2 : sr == 1 || d == 64 ? 4 : i4 ? 3 : 2; }

template <typename T, bool I4, int D, int SR>
__global__ void __launch_bounds__(SW * 32, simt_ctas(I4, D, SR))
    k_paged_simt(const PagedAttn a, int splits) {
    constexpr int NI = D / 32;  // four-dim pieces of a key that a lane of eight takes
    constexpr int DV = D / 32;  // output dims of a lane
    __shared__ __align__(16) float sq[SR][D];
    __shared__ __align__(16) float sc[SW][SR][SKEYS];
    __shared__ float so[SW][SR][D];
    __shared__ float sml[SW][SR][2];
    __shared__ int sh[SW + 4];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int item = blockIdx.x / splits, split = blockIdx.x % splits;
    const int head = item % a.pg.hkv;
    const Found f = find_tile<SR>(a, item / a.pg.hkv, sh);
    if (f.seq < 0) return;
    const SeqInfo si = seq_info(a, f.seq);
    const int pair0 = f.tile * SR, npair = min(SR, si.n_q * a.group - pair0);
    const int first = si.len - si.n_q;  // position of the sequence's first query row
    const int p0 = first + pair0 / a.group, p1 = first + (pair0 + npair - 1) / a.group;
    for (int i = tid; i < SR * D; i += SW * 32) {
        const int r = i / D, e = i % D;
        float x = 0.f;
        if (r < npair) {
            const int row = si.row0 + (pair0 + r) / a.group, h = head * a.group + (pair0 + r) % a.group;
            x = to_f<T>(reinterpret_cast<const T*>(a.q)[row * a.ld_q + h * D + e]) * a.scale_log2;
        }
        sq[r][e] = x;
    }
    __syncthreads();
    int rp[SR];
#pragma unroll
    for (int r = 0; r < SR; ++r) rp[r] = first + (pair0 + r) / a.group;
    const KeyRange kr = key_range<SKEYS>(p0, p1, a.window, a.n_sink);
    const int b0 = (int)((long long)kr.total() * split / splits), b1 = (int)((long long)kr.total() * (split + 1) / splits);
    float m[SR], l[SR], acc[SR][DV];
#pragma unroll
    for (int r = 0; r < SR; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int e = 0; e < DV; ++e) acc[r][e] = 0.f;
    }
    const int kk = lane >> 3, part = lane & 7;
    // the table entry of the next block's keys is read a block ahead
    auto entry_of = [&](int b) {
        const int j = kr.block(b) * SKEYS + lane;
        return b < b1 && seen_by_any(j, p0, p1, a.window, a.n_sink) ? page_entry(a.pg, f.seq, j) : 0;
    };
    int entry = entry_of(b0 + warp);
    for (int b = b0 + warp; b < b1; b += SW) {
        const int j0 = kr.block(b) * SKEYS, j = j0 + lane;
        const bool seen = seen_by_any(j, p0, p1, a.window, a.n_sink);
        const unsigned mask = __ballot_sync(0xffffffffu, seen);
        long long row = 0;
        if (seen) row = page_row(a.pg, checked_page(a.pg, entry, a.err), head, j & ((1 << a.pg.shift) - 1));
        entry = entry_of(b + SW);
        auto add = [&](float (&dot)[SR], const float (&x)[NI][4]) {
#pragma unroll
            for (int r = 0; r < SR; ++r)
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const float4 qv = *reinterpret_cast<const float4*>(&sq[r][4 * (part + 8 * i)]);
                    dot[r] += qv.x * x[i][0] + qv.y * x[i][1] + qv.z * x[i][2] + qv.w * x[i][3];
                }
        };
        auto keep = [&](float (&dot)[SR], int key) {
#pragma unroll
            for (int r = 0; r < SR; ++r) {
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) dot[r] += __shfl_xor_sync(0xffffffffu, dot[r], o);
                if (part == r) sc[warp][r][key] = dot[r];
            }
        };
        if constexpr (!I4) {
            // passes of four keys, for few pairs the loads of four passes on their way together; eight pairs have no
            // registers for that and branch around keys that no row sees
            constexpr int U = SR < 8 ? 4 : 1;
#pragma unroll (U == 4 ? 1 : 2)
            for (int ps = 0; ps < SKEYS / 4; ps += U) {
                float x[U][NI][4];
                auto seen_key = [&](int u) { return (mask >> (4 * (ps + u) + kk)) & 1u; };
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const long long kr_row = __shfl_sync(0xffffffffu, row, 4 * (ps + u) + kk);
#pragma unroll
                    for (int i = 0; i < NI; ++i) {
                        if (seen_key(u)) Row<T, I4, D>::k4(a.pg.k, kr_row, part + 8 * i, 1.f, x[u][i]);
                        else if (U > 1) x[u][i][0] = x[u][i][1] = x[u][i][2] = x[u][i][3] = 0.f;
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float dot[SR] = {};
                    if (U > 1 || seen_key(u)) add(dot, x[u]);
                    keep(dot, 4 * (ps + u) + kk);
                }
            }
        } else {
            // 4-bit pages: one branch around a key's loads and products (a branch each, as above: 24 instead of 21 us for
            // 27 tokens behind a window; eight pairs over model pages are 2-4 % faster with those)
#pragma unroll (SR == 8 ? 2 : 4)
            for (int ps = 0; ps < SKEYS / 4; ++ps) {
                const int key = 4 * ps + kk;
                const long long kr_row = __shfl_sync(0xffffffffu, row, key);
                float dot[SR] = {};
                if ((mask >> key) & 1u) {
                    float x[NI][4];
#pragma unroll
                    for (int i = 0; i < NI; ++i)
                        Row<T, I4, D>::k4(a.pg.k, kr_row, part + 8 * i, scale_of<I4, D>(a.pg.ks, kr_row, part + 8 * i), x[i]);
                    add(dot, x);
                }
                keep(dot, key);
            }
        }
        __syncwarp();
#pragma unroll
        for (int r = 0; r < SR; ++r) {
            float x = sc[warp][r][lane];
            if (r >= npair || !sees(j, rp[r], a.window, a.n_sink)) x = -INFINITY;
            float mx = x;
#pragma unroll
            for (int o = 16; o; o >>= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            mx = max_nan(mx, m[r]);
            const float ms = mx == -INFINITY ? 0.f : mx;
            const float w = exp2f(x - ms), corr = exp2f(m[r] - ms);
            m[r] = mx;
            l[r] = l[r] * corr + w;
#pragma unroll
            for (int e = 0; e < DV; ++e) acc[r][e] *= corr;
            sc[warp][r][lane] = w;
        }
        __syncwarp();
#pragma unroll (SR == 8 ? 1 : 2)
        for (int k0 = 0; k0 < SKEYS; k0 += 4) {  // four keys, whose weights are one load per pair
            float x[4][DV];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const long long v_row = __shfl_sync(0xffffffffu, row, k0 + u);
                if (!((mask >> (k0 + u)) & 1u)) {
#pragma unroll
                    for (int e = 0; e < DV; ++e) x[u][e] = 0.f;
                } else if constexpr (DV == 4) {
                    Row<T, I4, D>::v4(a.pg.v, v_row, lane, scale_of<I4, D>(a.pg.vs, v_row, lane), x[u]);
                } else {
                    float y[4];
                    Row<T, I4, D>::v4(a.pg.v, v_row, lane >> 1, scale_of<I4, D>(a.pg.vs, v_row, lane >> 1), y);
                    x[u][0] = (lane & 1) ? y[2] : y[0];
                    x[u][1] = (lane & 1) ? y[3] : y[1];
                }
            }
#pragma unroll
            for (int r = 0; r < SR; ++r) {
                const float4 w4 = *reinterpret_cast<const float4*>(&sc[warp][r][k0]);
                const float w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int e = 0; e < DV; ++e) acc[r][e] = w[u] != 0.f ? fmaf(w[u], x[u][e], acc[r][e]) : acc[r][e];
            }
        }
        __syncwarp();
    }
#pragma unroll
    for (int r = 0; r < SR; ++r) {
#pragma unroll
        for (int o = 16; o; o >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
        if (lane == 0) {
            sml[warp][r][0] = m[r];
            sml[warp][r][1] = l[r];
        }
#pragma unroll
        for (int e = 0; e < DV; ++e) so[warp][r][lane * DV + e] = acc[r][e];
    }
    __syncthreads();
    T* out = reinterpret_cast<T*>(a.out);
    const size_t slot_floats = paged_slot_floats(D);
    for (int i = tid; i < npair * D; i += SW * 32) {
        const int r = i / D, e = i % D;
        float mx = -INFINITY, L = 0.f, o = 0.f;
        for (int w = 0; w < SW; ++w) mx = max_nan(mx, sml[w][r][0]);
        const float ms = mx == -INFINITY ? 0.f : mx;
        for (int w = 0; w < SW; ++w) {
            const float c = exp2f(sml[w][r][0] - ms);
            if (c == 0.f) continue;
            L += sml[w][r][1] * c;
            o += so[w][r][e] * c;
        }
        if (splits == 1) {
            const int row = si.row0 + (pair0 + r) / a.group, h = head * a.group + (pair0 + r) % a.group;
            out[((long long)row * a.hq + h) * D + e] = from_f<T>(L == 0.f ? 0.f : o / L);
        } else {
            float* part_o = a.part + (size_t)blockIdx.x * slot_floats;
            part_o[i] = o;
            if (e == 0) {
                part_o[PAGED_MAX_TILE * D + r] = mx;
                part_o[PAGED_MAX_TILE * (D + 1) + r] = L;
            }
        }
    }
    if (splits == 1) return;
    __threadfence();
    __syncthreads();
    if (tid == 0) {
        const int before = atomicAdd(a.count + item, 1);
        sh[0] = before == splits - 1;
        if (sh[0]) a.count[item] = 0;  // ready for the next launch
    }
    __syncthreads();
    if (!sh[0]) return;
    __threadfence();
    const float* base = a.part + (size_t)item * splits * slot_floats;
    for (int i = tid; i < npair * D; i += SW * 32) {
        const int r = i / D, e = i % D;
        float mx = -INFINITY, L = 0.f, o = 0.f;
        for (int s = 0; s < splits; ++s) mx = max_nan(mx, __ldcg(base + s * slot_floats + PAGED_MAX_TILE * D + r));
        const float ms = mx == -INFINITY ? 0.f : mx;
        for (int s = 0; s < splits; ++s) {
            const float* p = base + s * slot_floats;
            const float c = exp2f(__ldcg(p + PAGED_MAX_TILE * D + r) - ms);
            if (c == 0.f) continue;
            L += __ldcg(p + PAGED_MAX_TILE * (D + 1) + r) * c;
            o += __ldcg(p + i) * c;
        }
        const int row = si.row0 + (pair0 + r) / a.group, h = head * a.group + (pair0 + r) % a.group;
        out[((long long)row * a.hq + h) * D + e] = from_f<T>(L == 0.f ? 0.f : o / L);
    }
}

template <typename T, bool I4, int D> void (*simt_kernel(int sr))(PagedAttn, int) {
    if constexpr (sizeof(T) == 4) {
        if (sr == 1) return k_paged_simt<T, I4, D, 1>;
        if (sr == 4) return k_paged_simt<T, I4, D, 4>;
    }
    return k_paged_simt<T, I4, D, 8>;
}

}  // namespace

void launch_paged_attn_simt(int dtype, bool i4, const PagedAttn& a, int d, cudaStream_t s) {
    // Pairs of a tile: as few as every sequence's rows fill (fp32: bf16 models come here with tensor cores
    // off alone).
    const long long pairs = (long long)a.max_q * a.group;
    const int sr = dtype == BLEND_BF16 || pairs > 4 ? 8 : pairs > 1 ? 4 : 1;
    const long long per_seq = (pairs + sr - 1) / sr;
    long long tiles = (long long)a.max_rows * a.group / sr + a.pg.n_seq;
    tiles = tiles < per_seq * a.pg.n_seq ? tiles : per_seq * a.pg.n_seq;
    const long long items = tiles * a.pg.hkv;
    if (items <= 0) return;
    // Shares of the keys: only while the tiles alone do not fill two CTAs on each of 152 SMs, and
    // no share under one 32-key block per warp at the longest length the table allows.
    const long long longest = (long long)a.pg.max_pages << a.pg.shift;
    long long splits = 1;
    if (items < 304) {
        splits = 608 / items;
        if (splits > PAGED_MAX_CTAS / items) splits = PAGED_MAX_CTAS / items;
        const long long most = (longest + SW * SKEYS - 1) / (SW * SKEYS);
        if (splits > most) splits = most;
        if (splits < 1) splits = 1;
    }
    auto kern = dtype == BLEND_BF16
                    ? (i4 ? (d == 64 ? simt_kernel<bf16, true, 64>(sr) : simt_kernel<bf16, true, 128>(sr))
                          : (d == 64 ? simt_kernel<bf16, false, 64>(sr) : simt_kernel<bf16, false, 128>(sr)))
                    : (i4 ? (d == 64 ? simt_kernel<float, true, 64>(sr) : simt_kernel<float, true, 128>(sr))
                          : (d == 64 ? simt_kernel<float, false, 64>(sr) : simt_kernel<float, false, 128>(sr)));
    kern<<<(unsigned)(items * splits), SW * 32, 0, s>>>(a, (int)splits);
    note_launch(1);
}

}  // namespace blend

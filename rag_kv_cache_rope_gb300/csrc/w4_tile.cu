// Products of many rows with 4-bit weights on tcgen05 (w4_linear in blend.h), bf16 inputs.
//
// A tile is 128 weight rows (M, the lanes of TMEM) by up to 128 input rows (N).  Weights are the A operand, in TMEM:
// their codes come by TMA as 128 x 64 bytes a chunk of 128 inputs, four warps turn them into bf16
// integers (code - 8) / 64, which are exact, one lane a weight row, and store them to TMEM, so they never pass
// through shared memory a second time and need no swizzle.  Inputs are the B operand, by TMA as they are.
// Scales are not rounded into an operand: the products of one group are summed in a TMEM accumulator of
// their own, and eight warps add it, times the row's scale, to sums in registers while the next group's products
// run.  So a result is what the few rows' kernel gives up to the order of fp32 sums.  (Scales inside the operand
// take 11 bits: two bf16 parts and twice the products.)
//   warp 0      TMA: codes and inputs            warp 1      tcgen05.mma of one lane, TMEM
//   warps 4-7   codes to TMEM                    warps 8-15  scales, sums, results
// Few tiles share their inputs' length among the CTAs of a cluster, which join their sums in order through
// distributed shared memory.  All waits are bounded: on expiry the error word gets BLEND_ETIMEOUT, copies and
// products in flight are waited for and TMEM is freed.
#include <cooperative_groups.h>

#include "attn_tc.cuh"
#include "w4.cuh"

namespace cg = cooperative_groups;

namespace blend {
namespace {

constexpr int TILE_M = 128, TILE_THREADS = 512;
constexpr int X_STAGES = 6;   // of 64 inputs
constexpr int C_STAGES = 6;   // of 128 inputs' codes
constexpr int A_STAGES = 4;   // of 64 inputs in TMEM, 32 columns each
constexpr int D_STAGES = 2;   // accumulators of a group
constexpr int CODE_BYTES = TILE_M * 64;
constexpr int A_COL = 256, TILE_COLS = 512;
constexpr int TILE_MAX_CLUSTER = 8;

template <int NT> constexpr int tile_smem(bool joined) {
    return X_STAGES * NT * 128 + C_STAGES * CODE_BYTES + (joined ? NT * TILE_M * 4 : 0) + 1024;
}

__device__ __forceinline__ void tmem_ld16(uint32_t t, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(t));
}

// NT: input rows of a tile; G: inputs of a group.
template <int NT, int G>
__global__ void __launch_bounds__(TILE_THREADS, 1)
    k_w4_tile(const __grid_constant__ CUtensorMap m_codes, const __grid_constant__ CUtensorMap m_x, const W4Linear a, int cluster) {
    constexpr uint32_t IDESC = (1u << 4) | (1u << 7) | (1u << 10) | ((NT >> 3) << 17) | ((TILE_M >> 4) << 24);
    constexpr int SPC = 128 / G, CW = NT / 2;  // groups of a chunk; columns of an epilogue thread
    extern __shared__ char smem_raw[];
    __shared__ uint64_t x_full[X_STAGES], x_empty[X_STAGES], c_full[C_STAGES], c_empty[C_STAGES], a_full[A_STAGES],
        a_empty[A_STAGES], d_full[D_STAGES], d_empty[D_STAGES], drain;
    __shared__ uint32_t tmem_sh;
    __shared__ int abort_sh;
    volatile int* abort_flag = &abort_sh;
    char* smem = (char*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    char* s_x = smem;
    char* s_codes = smem + X_STAGES * NT * 128;
    float* part = (float*)(s_codes + C_STAGES * CODE_BYTES);  // [NT][128]: this CTA's sums (cluster > 1)
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < X_STAGES; ++i) {
            mbar_init(&x_full[i], 1);
            mbar_init(&x_empty[i], 1);
        }
        for (int i = 0; i < C_STAGES; ++i) {
            mbar_init(&c_full[i], 1);
            mbar_init(&c_empty[i], 4);
        }
        for (int i = 0; i < A_STAGES; ++i) {
            mbar_init(&a_full[i], 4);
            mbar_init(&a_empty[i], 1);
        }
        for (int i = 0; i < D_STAGES; ++i) {
            mbar_init(&d_full[i], 1);
            mbar_init(&d_empty[i], 8);
        }
        mbar_init(&drain, 1);
        abort_sh = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&tmem_sh)), "r"(TILE_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tb = tmem_sh;

    const int rank = cluster > 1 ? (int)cta_rank() : 0;
    const int n_t = (a.rows + NT - 1) / NT, total = (a.w.n + TILE_M - 1) / TILE_M * n_t;
    const int tile0 = blockIdx.x / cluster, tile_step = gridDim.x / cluster;
    const int c0 = a.w.chunks * rank / cluster, c1 = a.w.chunks * (rank + 1) / cluster;
    bool ok = true;  // this warp's waits
    auto give_up = [&]() {
        ok = false;
        if (lane == 0) {
            *abort_flag = 1;
            set_error(a.err, BLEND_ETIMEOUT);
        }
    };
    uint32_t it_x = 0, it_c = 0, it_a = 0, it_d = 0;  // uses of the rings so far, by role

    for (int tile = tile0; tile < total; tile += tile_step) {
        const int wt = tile / n_t, tt = tile - wt * n_t;
        if (warp == 0) {
            if (lane == 0) {
                for (int c = c0; c < c1 && ok; ++c) {
                    const int sc = it_c % C_STAGES;
                    if (!mbar_wait(&c_empty[sc], (it_c / C_STAGES & 1) ^ 1, abort_flag)) {
                        give_up();
                        break;
                    }
                    mbar_expect_tx(&c_full[sc], CODE_BYTES);
                    tma_2d(s_codes + sc * CODE_BYTES, &m_codes, &c_full[sc], c * 64, wt * TILE_M);
                    ++it_c;
                    for (int h = 0; h < 2 && ok; ++h) {
                        const int sx = it_x % X_STAGES;
                        if (!mbar_wait(&x_empty[sx], (it_x / X_STAGES & 1) ^ 1, abort_flag)) {
                            give_up();
                            break;
                        }
                        mbar_expect_tx(&x_full[sx], NT * 128);
                        tma_2d(s_x + sx * NT * 128, &m_x, &x_full[sx], c * 128 + h * 64, tt * NT);
                        ++it_x;
                    }
                }
            }
            __syncwarp();
        } else if (warp == 1) {
            if (lane == 0) {
                for (int c = c0; c < c1 && ok; ++c) {
                    for (int h = 0; h < 2 && ok; ++h) {
                        const int sx = it_x % X_STAGES, sa = it_a % A_STAGES;
                        if (!mbar_wait(&x_full[sx], it_x / X_STAGES & 1, abort_flag) ||
                            !mbar_wait(&a_full[sa], it_a / A_STAGES & 1, abort_flag)) {
                            give_up();
                            break;
                        }
                        fence_after();
                        const uint64_t xd = desc_k(su32(s_x + sx * NT * 128));
                        const uint32_t at = tb + A_COL + sa * 32;
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            const int k = h * 64 + kk * 16, sd = it_d % D_STAGES;
                            if (k % G == 0) {
                                if (!mbar_wait(&d_empty[sd], (it_d / D_STAGES & 1) ^ 1, abort_flag)) {
                                    give_up();
                                    break;
                                }
                                fence_after();
                            }
                            umma_ts(tb + sd * NT, at + kk * 8, xd + (kk * 32 >> 4), IDESC, k % G ? 1u : 0u);
                            if ((k + 16) % G == 0) {
                                commit(&d_full[sd]);
                                ++it_d;
                            }
                        }
                        commit(&x_empty[sx]);
                        commit(&a_empty[sa]);
                        ++it_x;
                        ++it_a;
                    }
                }
            }
            __syncwarp();
        } else if (warp >= 4 && warp < 8) {
            const int r = (warp - 4) * 32 + lane;
            const uint32_t t_row = (uint32_t)(warp - 4) << 21;  // lanes 32 (warp - 4) .. of TMEM
            for (int c = c0; c < c1 && ok; ++c) {
                const int sc = it_c % C_STAGES;
                if (!warp_wait(&c_full[sc], it_c / C_STAGES & 1, abort_flag)) {
                    give_up();
                    break;
                }
                // piece t of the row's 64 bytes: words of inputs 32 w + 8 t (64-byte swizzle)
                uint4 q[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) q[t] = *(const uint4*)(s_codes + sc * CODE_BYTES + r * 64 + ((t ^ (r >> 1 & 3)) << 4));
                warp_arrive(&c_empty[sc]);
                ++it_c;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int sa = it_a % A_STAGES;
                    if (!warp_wait(&a_empty[sa], (it_a / A_STAGES & 1) ^ 1, abort_flag)) {
                        give_up();
                        break;
                    }
                    fence_after();
                    uint32_t v[32];
#pragma unroll
                    for (int w = 0; w < 2; ++w)
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            const uint32_t x = word_of(q[t], 2 * h + w);
                            uint32_t* o = v + 16 * w + 4 * t;
                            o[0] = code_pair<false>(x);
                            o[1] = code_pair<true>(x);
                            o[2] = code_pair<false>(x >> 8);
                            o[3] = code_pair<true>(x >> 8);
                        }
                    TMEM_ST32(tb + t_row + A_COL + sa * 32, v);
                    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                    fence_before();
                    warp_arrive(&a_full[sa]);
                    ++it_a;
                }
            }
        } else if (warp >= 8) {
            const int quarter = warp & 3, half = (warp - 8) >> 2;
            const int r = quarter * 32 + lane, j = wt * TILE_M + r;
            const uint32_t t_at = tb + ((uint32_t)quarter << 21) + half * CW;
            const bf16* sp = a.w.scale + (long long)min(j, a.w.n - 1) * a.w.chunks * SPC;
            float2 acc[CW / 2];
#pragma unroll
            for (int i = 0; i < CW / 2; ++i) acc[i] = make_float2(0.f, 0.f);
            Scales<G> next;
            next.load(sp + (long long)c0 * SPC);
            for (int c = c0; c < c1 && ok; ++c) {
                const Scales<G> sc = next;
                if (c + 1 < c1) next.load(sp + (long long)(c + 1) * SPC);
#pragma unroll
                for (int g = 0; g < SPC; ++g) {
                    const int sd = it_d % D_STAGES;
                    if (!warp_wait(&d_full[sd], it_d / D_STAGES & 1, abort_flag)) {
                        give_up();
                        break;
                    }
                    fence_after();
                    // (a group behind k has no scale)
                    const float s = c * 128 + g * G < a.w.k ? sc.get(g) : 0.f;
                    const float2 s2 = make_float2(s, s);
                    constexpr int B = CW < 32 ? CW : 32;
#pragma unroll
                    for (int b = 0; b < CW; b += B) {
                        uint32_t v[B];
#pragma unroll
                        for (int i = 0; i < B; i += 16) tmem_ld16(t_at + sd * NT + b + i, v + i);
                        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                        if (b + B == CW) {
                            fence_before();
                            warp_arrive(&d_empty[sd]);
                        }
#pragma unroll
                        for (int i = 0; i < B; i += 2)
                            acc[(b + i) / 2] = __ffma2_rn(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), s2, acc[(b + i) / 2]);
                    }
                    ++it_d;
                }
            }
            auto value = [&](int i) { return CODE_UNIT * (i & 1 ? acc[i / 2].y : acc[i / 2].x); };
            // one column of the tile: the weight rows' results for one row of inputs (all lanes)
            auto store = [&](int col, float v) {
                const int t = tt * NT + half * CW + col;
                if (t >= a.rows) return;
                if (a.epi == BLEND_W4_SWIGLU) {
                    // lanes 0..15 hold gate rows, 16..31 the up rows that go with them
                    const float up = __shfl_down_sync(0xffffffffu, v, 16);
                    if (lane >= 16 || j >= a.w.n) return;
                    const float y = v / (1.f + __expf(-v)) * up;
                    const long long at = (long long)t * a.ld_y + (wt * TILE_M + quarter * 32) / 2 + lane;
                    if (a.y_f32) ((float*)a.y)[at] = y;
                    else ((bf16*)a.y)[at] = __float2bfloat16_rn(y);
                    return;
                }
                if (j >= a.w.n) return;
                const long long at = (long long)t * a.ld_y + j;
                if (a.epi == BLEND_W4_ADD) ((float*)a.y)[at] += v;
                else if (a.y_f32) ((float*)a.y)[at] = v;
                else ((bf16*)a.y)[at] = __float2bfloat16_rn(v);
            };
            if (cluster == 1) {
                if (ok) {
#pragma unroll
                    for (int i = 0; i < CW; ++i) store(i, value(i));
                }
            } else {
#pragma unroll
                for (int i = 0; i < CW; ++i) part[(half * CW + i) * TILE_M + r] = value(i);
                __syncwarp();
                cluster_sync();
                if (ok) {
                    const int i0 = CW * rank / cluster, i1 = CW * (rank + 1) / cluster;
                    for (int i = i0; i < i1; ++i) {
                        float v = 0.f;
                        for (int q = 0; q < cluster; ++q)
                            v += cg::this_cluster().map_shared_rank(part, q)[(half * CW + i) * TILE_M + r];
                        store(i, v);
                    }
                }
                __syncwarp();
                cluster_sync();
            }
        }
        if (cluster > 1 && warp < 8) {
            // the epilogue's two meetings
            cluster_sync();
            cluster_sync();
        }
    }
    // After a wait that ran out, what is still in flight: copies, then products.
    __syncthreads();
    if (*abort_flag) {
        int never = 0;
        if (warp == 0 && lane == 0) {
            for (uint32_t i = it_c > C_STAGES ? it_c - C_STAGES : 0; i < it_c; ++i) mbar_wait(&c_full[i % C_STAGES], i / C_STAGES & 1, &never);
            for (uint32_t i = it_x > X_STAGES ? it_x - X_STAGES : 0; i < it_x; ++i) mbar_wait(&x_full[i % X_STAGES], i / X_STAGES & 1, &never);
        }
        if (warp == 1 && lane == 0) {
            commit(&drain);
            mbar_wait(&drain, 0, &never);
        }
        __syncwarp();
    }
    fence_before();
    __syncthreads();
    if (warp == 1) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tb), "r"(TILE_COLS) : "memory");
    }
}

PFN_cuTensorMapEncodeTiled_v12000 g_enc = nullptr;

bool encode(CUtensorMap* map, CUtensorMapDataType dt, const void* base, cuuint64_t inner, cuuint64_t outer, cuuint64_t stride,
            cuuint32_t box_inner, cuuint32_t box_outer, CUtensorMapSwizzle swizzle) {
    const cuuint64_t dims[2] = {inner, outer}, strides[1] = {stride};
    const cuuint32_t box[2] = {box_inner, box_outer}, es[2] = {1, 1};
    return g_enc(map, dt, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NT, int G> int go_tile(const W4Linear& a, cudaStream_t s) {
    auto* kern = k_w4_tile<NT, G>;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(TILE_THREADS);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    // clusters of 1..8 CTAs that run side by side
    static int fit[TILE_MAX_CLUSTER + 1] = {-1};
    if (fit[0] < 0) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, tile_smem<NT>(true)) != cudaSuccess) return BLEND_ECUDA;
        for (int c = 1; c <= TILE_MAX_CLUSTER; ++c) {
            attr.val.clusterDim.x = (unsigned)c;
            cfg.numAttrs = 1;
            cfg.gridDim = dim3(152u / c * c);
            cfg.dynamicSmemBytes = tile_smem<NT>(c > 1);
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
                cudaGetLastError();
                n = 0;
            }
            fit[c] = n < 152 / c ? n : 152 / c;
        }
        fit[0] = 0;
    }
    const int tiles = (a.w.n + TILE_M - 1) / TILE_M * ((a.rows + NT - 1) / NT);
    // CTAs of a tile: what takes the fewest chunks in a row, a tile's start and end counted as eight
    int cluster = 0;
    long long best = 0;
    for (int c = 1; c <= TILE_MAX_CLUSTER && c <= a.w.chunks; ++c) {
        if (fit[c] <= 0) continue;
        const long long cost = (long long)((tiles + fit[c] - 1) / fit[c]) * ((a.w.chunks + c - 1) / c + 8);
        if (!cluster || cost < best) {
            best = cost;
            cluster = c;
        }
    }
    if (!cluster) return BLEND_EUNSUPPORTED;
    CUtensorMap mc, mx;
    if (!encode(&mc, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w.codes, (cuuint64_t)a.w.chunks * 64, (cuuint64_t)a.w.n, (cuuint64_t)a.w.chunks * 64, 64,
                TILE_M, CU_TENSOR_MAP_SWIZZLE_64B) ||
        !encode(&mx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.x, (cuuint64_t)a.w.k, (cuuint64_t)a.rows, (cuuint64_t)a.ld_x * 2, 64, NT,
                CU_TENSOR_MAP_SWIZZLE_128B))
        return BLEND_EUNSUPPORTED;
    attr.val.clusterDim.x = (unsigned)cluster;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    cfg.gridDim = dim3((unsigned)((tiles < fit[cluster] ? tiles : fit[cluster]) * cluster));
    cfg.dynamicSmemBytes = tile_smem<NT>(cluster > 1);
    if (cudaLaunchKernelEx(&cfg, kern, mc, mx, a, cluster) != cudaSuccess) return BLEND_ECUDA;
    note_launch();
    return BLEND_OK;
}
template <int NT> int go_tile_group(const W4Linear& a, cudaStream_t s) {
    return a.w.group == 32 ? go_tile<NT, 32>(a, s) : a.w.group == 64 ? go_tile<NT, 64>(a, s) : go_tile<NT, 128>(a, s);
}

}  // namespace

int launch_w4_tile(const W4Linear& a, cudaStream_t s) {
    if (!g_enc) {
        cudaDriverEntryPointQueryResult qr;
        void* fn = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &qr) != cudaSuccess ||
            qr != cudaDriverEntryPointSuccess || !fn) {
            cudaGetLastError();
            return BLEND_EUNSUPPORTED;
        }
        g_enc = (PFN_cuTensorMapEncodeTiled_v12000)fn;
    }
    return a.rows <= 32 ? go_tile_group<32>(a, s) : a.rows <= 64 ? go_tile_group<64>(a, s) : go_tile_group<128>(a, s);
}

}  // namespace blend

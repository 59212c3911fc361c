// Products of many rows with 4-bit weights on tcgen05 (w4_linear in blend.h), bf16 inputs.
//
// A tile is 128 weight rows (M, the lanes of TMEM) by up to 128 input rows (N).  Weights are the A operand, in TMEM:
// their codes come by TMA as 128 x 64 bytes a chunk of 128 inputs, eight warps turn them into bf16
// integers (code - 8) / 64, which are exact, one lane a weight row, and store them to TMEM, so they never pass
// through shared memory a second time and need no swizzle.  Inputs are the B operand, by TMA as they are.
// Scales are not rounded into an operand: the products of one group are summed in a TMEM accumulator of
// their own, and eight warps add it, times the row's scale, to sums in registers while the next group's products
// run.  So a result is what the few rows' kernel gives up to the order of fp32 sums.  (Scales inside the operand
// take 11 bits: two bf16 parts, exact, and twice the products.)
//
// What bounds it is that hand-over: a group's accumulators are awaited, read, released and added one after the
// other by the same warps, about 480 cycles of 128 columns, where the products of 32 inputs take 128 and those of
// 128 inputs 512.  So groups of 128 run near the products' rate and smaller groups do not: 500 x 27648 x 5120 in groups of 128, 64
// and 32 takes 111, 160 and 253 us (1.28, 0.88 and 0.56 PFLOP/s), 2048 rows in groups of 128 412 us (1.41 PFLOP/s).  16 to
// 128 rows are bound by turning codes into operands, about 600 cycles a chunk whatever its rows: 16 x 27648 x 5120 27 us,
// 64 rows 31, 128 rows 37.  Tiles of 32 and 64 rows for as few rows: 29 us for 35, 33 for 37.
//
//   warp 0      TMA: codes                       warp 1      tcgen05.mma of one lane, TMEM
//   warp 2      TMA: inputs                      warp 3      products too, with tiles of 128 rows
//   warps 4-11  codes to TMEM                    warps 12-19 scales, sums, results
// Few tiles share their inputs' length among the CTAs of a cluster, which join their sums in order through
// distributed shared memory (16 x 5120 x 13824: 19 us for 38).  Tiles that do not come out even over the SMs are a line of
// chunks to a cluster, of which each CTA takes a stretch (500 x 5120 x 13824, 160 tiles on 152 SMs: 62 us for 91; 389 x 5120 x
// 8192: 43 for 58; 128 x 27648 x 5120: 37 for 41.6).  All waits are bounded: on expiry the error word gets BLEND_ETIMEOUT, copies and
// products in flight are waited for and TMEM is freed.
#include "w4.cuh"

namespace blend {
namespace {

constexpr int TILE_M = 128, TILE_THREADS = 640, EPI_WARPS = 8;
constexpr int STAGES = 4;     // chunks of 128 inputs on their way: operands in TMEM, inputs
// The same of codes.
template <int NT> constexpr int C_STAGES = NT == 128 ? 4 : 8;
constexpr int CODE_BYTES = TILE_M * 64;
constexpr int A_COL = 256, TILE_COLS = 512;  // accumulators, then 64 columns a stage
constexpr int TILE_MAX_CLUSTER = 8;

template <int NT> constexpr int tile_smem() {
    return STAGES * NT * 256 + C_STAGES<NT> * CODE_BYTES + NT * TILE_M * 4 + 1024;
}

// C columns of a warp's lanes: 16, 32 or 64.
template <int C> __device__ __forceinline__ void tmem_ld(uint32_t t, uint32_t (&r)[C]) {
    if constexpr (C == 64) {
        TMEM_LD32(t, r);
        uint32_t* h = r + 32;
        TMEM_LD32(t + 32, h);
    } else if constexpr (C == 32) {
        TMEM_LD32(t, r);
    } else {
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
              "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(t));
    }
}
// Bounded wait, of one thread or of whole warps, in few instructions: the roles' loops are short and run side by
// side, and what limited a first version was fetching their unrolled code.
__device__ __forceinline__ bool phase_wait(uint64_t* b, uint32_t par, volatile int* abort_flag) {
#pragma unroll 1
    for (int i = 0; i < WAIT_LIMIT; ++i) {
        if (mbar_try(b, par)) return true;
        if (*abort_flag) return false;
    }
    return false;
}
// A warp's wait for one to three phases: a look at a barrier takes 70 cycles, so they are looked at together.
// (One lane looking for its warp took 300.)
__device__ __forceinline__ bool warp_phases(volatile int* abort_flag, uint64_t* b0, uint32_t p0, uint64_t* b1 = nullptr, uint32_t p1 = 0,
                                            uint64_t* b2 = nullptr, uint32_t p2 = 0) {
    bool done = mbar_try(b0, p0);
    if (b1) done &= mbar_try(b1, p1);
    if (b2) done &= mbar_try(b2, p2);
    if (__all_sync(0xffffffffu, done)) return true;
    done = phase_wait(b0, p0, abort_flag);
    if (b1) done = done && phase_wait(b1, p1, abort_flag);
    if (b2) done = done && phase_wait(b2, p2, abort_flag);
    return __all_sync(0xffffffffu, done);
}
// A look that does not block, whose answer is asked for later: a phase that has ended stays so until its reader is done.
__device__ __forceinline__ bool phase_look(uint64_t* b, uint32_t par) {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}\n"
                 : "=r"(p)
                 : "r"(su32(b)), "r"(par)
                 : "memory");
    return p != 0;
}
// A place in a ring of N stages.
template <int N> struct Ring {
    int at = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void step() {
        if (++at == N) {
            at = 0;
            phase ^= 1;
        }
    }
};

// NT: input rows of a tile; G: inputs of a group; split: CTAs take stretches of a line of tiles (a form of its own: in one
// with the other, 500 x 27648 x 5120 took 113 us for 110).
template <int NT, int G, bool split>
__global__ void __launch_bounds__(TILE_THREADS, 1)
    k_w4_tile(const __grid_constant__ CUtensorMap m_codes, const __grid_constant__ CUtensorMap m_x, const W4Linear a, int cluster) {
    constexpr uint32_t IDESC = (1u << 4) | (1u << 7) | (1u << 10) | ((NT >> 3) << 17) | ((TILE_M >> 4) << 24);
    constexpr int SPC = 128 / G, CW = NT / 2;  // groups of a chunk; columns of an epilogue thread
    constexpr int GB = SPC < 128 / NT ? SPC : 128 / NT;  // groups whose accumulators make a stage
    constexpr int D_COLS = GB * NT, D_STAGES = A_COL / D_COLS;
    constexpr int PER = SPC / GB;              // accumulator stages of a chunk
    constexpr int MMAS = NT == 128 ? 2 : 1;    // warps that issue products
    static_assert(MMAS == 1 || (D_STAGES % 2 == 0 && STAGES % 2 == 0 && (PER == 1 || PER % 2 == 0)), "each MMA warp keeps to its own stages");
    constexpr int X_BYTES = NT * 256;          // two halves of 64 inputs
    extern __shared__ char smem_raw[];
    constexpr int CS = C_STAGES<NT>;
    // c_full, in: codes, inputs have come; full: four warps' operands; empty: their products are done
    __shared__ uint64_t c_full[CS], c_empty[CS], in[STAGES], full[STAGES], empty[STAGES], d_full[D_STAGES], d_empty[D_STAGES],
        p_full[2], p_empty[2], drain;  // p: sums of the cluster's CTAs; split: of the neighbours below and above
    __shared__ uint32_t tmem_sh;
    __shared__ int abort_sh;
    volatile int* abort_flag = &abort_sh;
    char* smem = (char*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    char* s_x = smem;
    char* s_codes = smem + STAGES * X_BYTES;
    float* part = (float*)(s_codes + CS * CODE_BYTES);  // [NT][128]: this CTA's sums
    const int tid = threadIdx.x, lane = tid & 31;
    // (the same for all lanes, and known to be: the roles' loops run in uniform registers, where the operands of
    // tcgen05.mma and TMA have to be; with a loop of lane 0 alone each product took 100 cycles to issue)
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    if (tid == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&in[i], 1);
            mbar_init(&full[i], 4);
            mbar_init(&empty[i], PER == 1 ? 1 : MMAS);
        }
        for (int i = 0; i < CS; ++i) {
            mbar_init(&c_full[i], 1);
            mbar_init(&c_empty[i], 4);
        }
        for (int i = 0; i < D_STAGES; ++i) {
            mbar_init(&d_full[i], 1);
            mbar_init(&d_empty[i], EPI_WARPS);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&p_full[i], EPI_WARPS * (split ? 1 : cluster));
            mbar_init(&p_empty[i], EPI_WARPS * (split ? 1 : cluster));
        }
        mbar_init(&drain, MMAS);
        abort_sh = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        // (never waits: by its registers no other CTA that uses TMEM fits on the SM beside this one)
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&tmem_sh)), "r"(TILE_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    if (cluster > 1) cluster_sync();  // all CTAs' barriers exist
    fence_after();
    // (all of TMEM: the columns begin at 0)
    constexpr uint32_t tb = 0;

    const int rank = blockIdx.x % cluster;
    const int n_t = (a.rows + NT - 1) / NT, total = (a.w.n + TILE_M - 1) / TILE_M * n_t;
    // The cluster's tiles: of each a share of the chunks for every CTA or, split, one line of chunks of which a CTA
    // takes a stretch (whole tiles and a part at either end). Even ranks walk up the line, odd ones down, so that neighbours
    // both begin or both end with the tile that they share. Who has the smaller part of it leaves its sums in shared memory,
    // which it needs again a whole tile later, and the other, who comes last, finishes the tile: nobody waits.
    const int first_tile = blockIdx.x / cluster, tile_step = gridDim.x / cluster, chunks = a.w.chunks;
    const int tiles = first_tile < total ? (total - first_tile + tile_step - 1) / tile_step : 0;
    const int lo = split ? tiles * chunks * rank / cluster : 0, hi = split ? tiles * chunks * (rank + 1) / cluster : 0;
    const int pieces = split ? (hi - 1) / chunks - lo / chunks + 1 : tiles;
    struct Piece {
        int tile, c0, c1;
    };
    auto piece = [&](int p) {
        if (!split) return Piece{first_tile + p * tile_step, chunks * rank / cluster, chunks * (rank + 1) / cluster};
        const int t = rank & 1 ? (hi - 1) / chunks - p : lo / chunks + p;
        return Piece{first_tile + t * tile_step, max(lo - t * chunks, 0), min(hi - t * chunks, chunks)};
    };
    bool ok = true;  // this warp's waits
    auto give_up = [&]() {
        ok = false;
        if (lane == 0) {
            *abort_flag = 1;
            set_error(a.err, BLEND_ETIMEOUT);
        }
    };
    Ring<STAGES> st;   // this role's stages
    Ring<CS> sc;
    Ring<D_STAGES> sd;
    Ring<1> met;

    // The roles' ends are their own, with no code in common: what runs on fewer registers stays within them.
    auto end_of_work = [&]() {
        fence_before();
        asm volatile("barrier.sync 0;" ::: "memory");
    };
    auto end_of_cluster = [&]() {
        fence_before();
        asm volatile("barrier.sync 0;" ::: "memory");
        if (cluster > 1) cluster_sync();  // no CTA leaves while another reads its sums
    };
    // Each role walks over the tiles by itself; registers go from the first four warps to the epilogue's.
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 0) {
            for (int p = 0; p < pieces; ++p) {
                const Piece at = piece(p);
                const int wt = at.tile / n_t;
#pragma unroll 1
                for (int c = at.c0; c < at.c1 && ok; ++c) {
                    if (!warp_phases(abort_flag, &c_empty[sc.at], sc.phase ^ 1)) {
                        give_up();
                        break;
                    }
                    if (elect_one()) {
                        mbar_expect_tx(&c_full[sc.at], CODE_BYTES);
                        tma_2d(s_codes + sc.at * CODE_BYTES, &m_codes, &c_full[sc.at], c * 64, wt * TILE_M);
                    }
                    __syncwarp();
                    sc.step();
                }
            }
        } else if (warp == 2) {
            for (int p = 0; p < pieces; ++p) {
                const Piece at = piece(p);
                const int tt = at.tile % n_t;
#pragma unroll 1
                for (int c = at.c0; c < at.c1 && ok; ++c) {
                    if (!warp_phases(abort_flag, &empty[st.at], st.phase ^ 1)) {
                        give_up();
                        break;
                    }
                    if (elect_one()) {
                        char* x = s_x + st.at * X_BYTES;
                        mbar_expect_tx(&in[st.at], X_BYTES);
                        tma_2d(x, &m_x, &in[st.at], c * 128, tt * NT);
                        tma_2d(x + X_BYTES / 2, &m_x, &in[st.at], c * 128 + 64, tt * NT);
                    }
                    __syncwarp();
                    st.step();
                }
            }
        } else if (warp < 2 * MMAS) {
            // Each of the two has the accumulator stages of one parity, so that one looks at its barriers while the
            // other's products run.
            const int mine = warp >> 1;
            for (int p = 0; p < pieces; ++p) {
                const Piece of = piece(p);
#pragma unroll 1
                for (int c = of.c0; c < of.c1 && ok; ++c, st.step()) {
                    if (MMAS == 2 && PER == 1 && (sd.at & 1) != mine) {
                        sd.step();
                        continue;
                    }
                    if (MMAS == 2 && PER > 1 && mine) sd.step();
                    if (!warp_phases(abort_flag, &in[st.at], st.phase, &full[st.at], st.phase, &d_empty[sd.at], sd.phase ^ 1)) {
                        give_up();
                        break;
                    }
                    const uint64_t xd = desc_k(su32(s_x + st.at * X_BYTES));
                    const uint32_t at = tb + A_COL + st.at * 64;
#pragma unroll
                    for (int b = 0; b < PER; ++b) {
                        if (MMAS == 2 && PER > 1 && (b & 1) != mine) continue;
                        if (b >= MMAS && !warp_phases(abort_flag, &d_empty[sd.at], sd.phase ^ 1)) {
                            give_up();
                            break;
                        }
                        fence_after();
                        const uint32_t d = tb + sd.at * D_COLS;
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < GB * G / 16; ++kk) {
                                const int k = b * GB * G + kk * 16;  // (the second 64 inputs are NT rows of 128 bytes behind)
                                umma_ts(d + kk * 16 / G * NT, at + k / 2, xd + ((k / 64 * NT * 128 + k % 64 * 2) >> 4), IDESC, k % G ? 1u : 0u);
                            }
                            commit(&d_full[sd.at]);
                            if (b + MMAS >= PER) commit(&empty[st.at]);
                        }
                        __syncwarp();
                        sd.step();
                        if (MMAS == 2 && PER > 1 && b + 2 < PER) sd.step();
                    }
                    if (MMAS == 2 && PER > 1 && !mine) sd.step();
                }
            }
        }
        end_of_work();
        if (*abort_flag) {
            // after a wait that ran out, what is still in flight: copies, then products
            int never = 0;
            // (stages before the next one were filled in this turn of the ring, the others in the last)
            if (warp == 0) {
#pragma unroll 1
                for (int i = 0; i < CS; ++i) phase_wait(&c_full[i], i < sc.at ? sc.phase : sc.phase ^ 1, &never);
            }
            if (warp == 2) {
#pragma unroll 1
                for (int i = 0; i < STAGES; ++i) phase_wait(&in[i], i < st.at ? st.phase : st.phase ^ 1, &never);
            }
            if ((warp & 1) && warp < 2 * MMAS) {
                if (elect_one()) commit(&drain);
                __syncwarp();
                phase_wait(&drain, 0, &never);
            }
            __syncwarp();
        }
        end_of_cluster();
        if (warp == 1) {
            fence_after();
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_sh), "r"(TILE_COLS) : "memory");
        }
    } else if (warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        // two sets of four warps take every second chunk
        const int r = (warp & 3) * 32 + lane, set = (warp >> 2) & 1;
        const uint32_t t_row = tb + ((uint32_t)(warp & 3) << 21) + A_COL;  // lanes 32 (warp % 4) .. of TMEM
        int turn = 1;
        for (int p = 0; p < pieces; ++p) {
            const Piece at = piece(p);
#pragma unroll 1
            for (int c = at.c0; c < at.c1 && ok; ++c, st.step(), sc.step()) {
                turn ^= 1;
                if (turn != set) continue;
                if (!warp_phases(abort_flag, &c_full[sc.at], sc.phase, &empty[st.at], st.phase ^ 1)) {
                    give_up();
                    break;
                }
                // piece t of the row's 64 bytes: words of inputs 32 w + 8 t (64-byte swizzle)
                uint4 q[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) q[t] = *(const uint4*)(s_codes + sc.at * CODE_BYTES + r * 64 + ((t ^ (r >> 1 & 3)) << 4));
                fence_after();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
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
                    TMEM_ST32(t_row + st.at * 64 + h * 32, v);
                }
                warp_arrive(&c_empty[sc.at]);
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                fence_before();
                warp_arrive(&full[st.at]);
            }
        }
        end_of_work();
        end_of_cluster();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
        // Many small groups: the next accumulators are looked for before the last are added (groups of 32: 264 -> 251 us at
        // 500 x 27648 x 5120; of 64 and 128: 2-4 % longer).
        constexpr bool EARLY = PER > 2;
        bool early = false;
        // results of y sixteen bytes at a time
        const bool vec = (((uintptr_t)a.y | (uintptr_t)a.ld_y * (a.y_f32 ? 4 : 2)) & 15) == 0;
        int left_at = -1;  // the side of the neighbour who has still to read the sums that were left
        for (int p = 0; p < pieces; ++p) {
            const Piece of = piece(p);
            const int wt = of.tile / n_t, tt = of.tile - wt * n_t, c0 = of.c0, c1 = of.c1;
            const int quarter = warp & 3, cols = (warp - 12) >> 2;
            const int r = quarter * 32 + lane, j = wt * TILE_M + r;
            const uint32_t t_at = tb + ((uint32_t)quarter << 21) + cols * CW;
            const bf16* sp = a.w.scale + (long long)min(j, a.w.n - 1) * a.w.chunks * SPC;
            float2 acc[CW / 2];
#pragma unroll
            for (int i = 0; i < CW / 2; ++i) acc[i] = make_float2(0.f, 0.f);
            Scales<G> next;
            next.load(sp + (long long)c0 * SPC);
#pragma unroll 1
            for (int c = c0; c < c1 && ok; ++c) {
                const Scales<G> sc = next;
                if (c + 1 < c1) next.load(sp + (long long)(c + 1) * SPC);
#pragma unroll 1
                for (int b = 0; b < PER; ++b) {
                    if (!(EARLY && __all_sync(0xffffffffu, early)) && !warp_phases(abort_flag, &d_full[sd.at], sd.phase)) {
                        give_up();
                        break;
                    }
                    fence_after();
#pragma unroll
                    for (int gb = 0; gb < GB; ++gb) {
                        const int g = b * GB + gb;
                        // (a group behind k has no scale)
                        const float s = c * 128 + g * G < a.w.k ? sc.get(g) : 0.f;
                        uint32_t v[CW];
                        tmem_ld<CW>(t_at + sd.at * D_COLS + gb * NT, v);
                        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                        if (gb == GB - 1) {
                            fence_before();
                            warp_arrive(&d_empty[sd.at]);
                            if (EARLY) {
                                Ring<D_STAGES> next_d = sd;
                                next_d.step();
                                early = phase_look(&d_full[next_d.at], next_d.phase);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < CW; i += 2) {
                            // (packed in pairs: 500 rows 110.8 us for 109.0, 64 rows 35.1 for 36.5)
                            float2& sum = acc[i / 2];
                            const float2 x = make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
                            sum = NT == 128 ? make_float2(fmaf(x.x, s, sum.x), fmaf(x.y, s, sum.y)) : __ffma2_rn(x, make_float2(s, s), sum);
                        }
                    }
                    sd.step();
                }
            }
            // This CTA's sums to shared memory, [column][weight row]; then a thread takes eight neighbouring results of one
            // row of y from there, of columns i0 .. i1 - 1 of its half: all, or this CTA's share, joined with the other CTAs'
            // sums in their order. (The neighbour's sums of a split tile are added before.)
            float* mine = part + cols * CW * TILE_M;
            const bool shared = split && c1 - c0 < chunks;
            const int other = c0 > 0 ? rank - 1 : rank + 1, side = c0 > 0 ? 0 : 1;  // (for it, this CTA is at side ^ 1)
            const bool finishes = !shared || 2 * (c1 - c0) > chunks || (2 * (c1 - c0) == chunks && rank < other);
            const int i0 = split ? 0 : CW * rank / cluster, i1 = min(split ? CW : CW * (rank + 1) / cluster, a.rows - tt * NT - cols * CW);
            // what was there has been read, by the other CTAs and by this one
            if (split && left_at >= 0 && ok && !cluster_phase(&p_empty[left_at], 0, abort_flag)) give_up();
            if (!split && cluster > 1 && ok && !cluster_phase(&p_empty[0], met.phase ^ 1, abort_flag)) give_up();
            asm volatile("barrier.sync %0, 128;" ::"r"(1 + cols) : "memory");
#pragma unroll
            for (int i = 0; i < CW; ++i) mine[i * TILE_M + r] = i & 1 ? acc[i / 2].y : acc[i / 2].x;
            left_at = finishes ? -1 : side;
            if (!finishes) {
                meet(&p_full[side ^ 1], other, 1);
                continue;
            }
            if (shared) {
                if (ok && !cluster_phase(&p_full[side], 0, abort_flag)) give_up();
                const uint32_t from = peer_addr(mine + r, other);
#pragma unroll 1
                for (int i = 0; i < CW; i += 16) {
                    float v[16];
#pragma unroll
                    for (int u = 0; u < 16; ++u) v[u] = ld_peer(from + (i + u) * TILE_M * 4);
#pragma unroll
                    for (int u = 0; u < 16; ++u) mine[(i + u) * TILE_M + r] += v[u];
                }
                meet(&p_empty[side ^ 1], other, 1);
            }
            if (cluster == 1 || split) asm volatile("barrier.sync %0, 128;" ::"r"(1 + cols) : "memory");
            else {
                meet(&p_full[0], 0, cluster);
                if (ok && !cluster_phase(&p_full[0], met.phase, abort_flag)) give_up();
            }
            auto sums = [&](int at, float (&v)[8]) {
                if (cluster == 1 || split) {
                    *(float4*)v = *(const float4*)(mine + at);
                    *(float4*)(v + 4) = *(const float4*)(mine + at + 4);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = 0.f;
#pragma unroll 1
                    for (int c = 0; c < cluster; c += 4) {
                        float4 q[4][2];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const uint32_t from = peer_addr(mine + at, min(c + u, cluster - 1));
                            q[u][0] = ld_peer4(from);
                            q[u][1] = ld_peer4(from + 16);
                        }
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            if (c + u < cluster) {
#pragma unroll
                                for (int e = 0; e < 8; ++e) v[e] += ((const float*)q[u])[e];
                            }
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= CODE_UNIT;
            };
            const bool swiglu = a.epi == BLEND_W4_SWIGLU;
            const int per_log2 = swiglu ? 3 : 4, wide = swiglu ? a.w.n / 2 : a.w.n;
#pragma unroll 1
            for (int o = quarter * 32 + lane; ok && o < (i1 - i0) << per_log2; o += 128) {
                const int col = i0 + (o >> per_log2), p = o & ((1 << per_log2) - 1);
                float v[8];
                if (swiglu) {
                    // sixteen gate rows, then the sixteen up rows that go with them
                    const int at = col * TILE_M + (p >> 1) * 32 + (p & 1) * 8;
                    float up[8];
                    sums(at, v);
                    sums(at + 16, up);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = v[e] / (1.f + expf(-v[e])) * up[e];
                } else
                    sums(col * TILE_M + p * 8, v);
                const int j0 = (wt * TILE_M >> (swiglu ? 1 : 0)) + p * 8;
                const long long at = (long long)(tt * NT + cols * CW + col) * a.ld_y + j0;
                if (vec && j0 + 8 <= wide) {
                    if (a.y_f32) {
                        float4* y = (float4*)((float*)a.y + at);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float4 x = make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
                            if (a.epi == BLEND_W4_ADD) {
                                const float4 old = y[h];
                                x = make_float4(old.x + x.x, old.y + x.y, old.z + x.z, old.w + x.w);
                            }
                            y[h] = x;
                        }
                    } else {
                        Vec<bf16> x;
#pragma unroll
                        for (int e = 0; e < 8; ++e) x.set(e, v[e]);
                        *(uint4*)((bf16*)a.y + at) = x.raw;
                    }
                } else {
#pragma unroll 1
                    for (int e = 0; e < 8 && j0 + e < wide; ++e) {
                        const float x = v[0];
#pragma unroll
                        for (int i = 0; i < 7; ++i) v[i] = v[i + 1];
                        if (a.epi == BLEND_W4_ADD) ((float*)a.y)[at + e] += x;
                        else if (a.y_f32) ((float*)a.y)[at + e] = x;
                        else ((bf16*)a.y)[at + e] = __float2bfloat16_rn(x);
                    }
                }
            }
            if (!split && cluster > 1) {
                meet(&p_empty[0], 0, cluster);
                met.step();
            }
        }
        end_of_work();
        end_of_cluster();
    }
}

template <int NT, int G> int go_tile(const W4Linear& a, cudaStream_t s) {
    auto *kern = k_w4_tile<NT, G, false>, *kern_split = k_w4_tile<NT, G, true>;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(TILE_THREADS);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    // clusters of 1..8 CTAs that run side by side, asked for once on a device
    struct Fit {
        int of[TILE_MAX_CLUSTER + 1] = {};
        bool ok = false;
    };
    static PerDevice<Fit> fits;
    const Fit* here = fits.get([&] {
        Fit f;
        f.ok = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, tile_smem<NT>()) == cudaSuccess &&
               cudaFuncSetAttribute(kern_split, cudaFuncAttributeMaxDynamicSharedMemorySize, tile_smem<NT>()) == cudaSuccess;
        for (int c = 1; c <= TILE_MAX_CLUSTER && f.ok; ++c) {
            attr.val.clusterDim.x = (unsigned)c;
            cfg.numAttrs = 1;
            cfg.gridDim = dim3(152u / c * c);
            cfg.dynamicSmemBytes = tile_smem<NT>();
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
                cudaGetLastError();
                n = 0;
            }
            f.of[c] = n < 152 / c ? n : 152 / c;
        }
        return f;
    });
    if (!here) return BLEND_ECUDA;
    const int* fit = here->of;
    const int tiles = (a.w.n + TILE_M - 1) / TILE_M * ((a.rows + NT - 1) / NT);
    // (the other form takes the same room)
    // CTAs of a cluster, and whether they split its tiles: what takes the fewest chunks in a row, a tile's end counted as
    // four, with sums to join as sixteen. (A split tile belongs to two CTAs: a cluster has as many tiles as CTAs.)
    int cluster = 0, split = 0;
    long long best = 0;
    for (int c = 1; c <= TILE_MAX_CLUSTER && c <= a.w.chunks; ++c) {
        if (fit[c] <= 0) continue;
        const long long rounds = (tiles + fit[c] - 1) / fit[c];
        for (int sp = 0; sp <= (c > 1 && tiles / fit[c] >= c && rounds * a.w.chunks < (1 << 24)); ++sp) {
            const long long cost = sp ? (rounds * a.w.chunks + c - 1) / c + (rounds + c - 1) / c * 4 + 16
                                      : rounds * ((a.w.chunks + c - 1) / c + (c == 1 ? 4 : 16));
            if (!cluster || cost < best) {
                best = cost;
                cluster = c;
                split = sp;
            }
        }
    }
    if (!cluster) return BLEND_EUNSUPPORTED;
    CUtensorMap mc, mx;
    if (!w4_encode_codes(&mc, a.w, TILE_M) || !w4_encode_inputs(&mx, a, NT)) return BLEND_EUNSUPPORTED;
    attr.val.clusterDim.x = (unsigned)cluster;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    cfg.gridDim = dim3((unsigned)((tiles < fit[cluster] ? tiles : fit[cluster]) * cluster));
    cfg.dynamicSmemBytes = tile_smem<NT>();
    if (cudaLaunchKernelEx(&cfg, split ? kern_split : kern, mc, mx, a, cluster) != cudaSuccess) return BLEND_ECUDA;
    note_launch();
    return BLEND_OK;
}
template <int NT> int go_tile_group(const W4Linear& a, cudaStream_t s) {
    return a.w.group == 32 ? go_tile<NT, 32>(a, s) : a.w.group == 64 ? go_tile<NT, 64>(a, s) : go_tile<NT, 128>(a, s);
}

}  // namespace

int launch_w4_tile(const W4Linear& a, cudaStream_t s) {
    return a.rows <= 32 ? go_tile_group<32>(a, s) : a.rows <= 64 ? go_tile_group<64>(a, s) : go_tile_group<128>(a, s);
}

}  // namespace blend

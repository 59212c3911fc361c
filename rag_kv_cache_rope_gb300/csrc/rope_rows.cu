// Rotary positions of every layout and scaling (rope_rows in blend.h).
//
// One thread owns a unit of 16 dims of a head and walks over heads and layers with it: the eight pairs'
// sines and cosines are computed once and stay in registers.  A unit is the dims i..i+7 and
// i+rot/2..i+rot/2+7 (half layout), sixteen neighbouring dims (interleaved), or sixteen dims behind the
// rotated ones, which are copied.  The d/16 threads of a head sit side by side and a warp covers
// neighbouring heads of a row, so loads and stores are whole lines.
//
// Angles: a pair's frequency is a 64-bit fraction of a turn, so rot * freq modulo 2^64 is the angle modulo
// a turn with an error of |rot| * 2^-53 of the frequency and no reduction: one integer multiplication
// where fp64 angles would need a division by 2 pi.  The fraction is cut into a quarter turn and a
// rest of at most an eighth, whose sine and cosine are fp32.
//
// Cached keys of 16064 rows over 8 layers, 8 x 128 bf16: 87 us, 6.0 TB/s, 90 % of the copy rate, bound by HBM.  4099 rows of
// 40 + 8 heads: 19.5 us (half of the dims, interleaved) to 20.8, 5 TB/s: the angles of a row are in the way of its first
// loads.  One row: 2.6 us.  fp32: 16064 rows 179 us (half layout) and 206 (interleaved), 157 at the copy rate.
#include "tokens.cuh"

namespace blend {
namespace {

constexpr int ROPE_THREADS = 256;

// cos and sin of `turn` 2^-64 turns.
__device__ __forceinline__ float2 unit_circle(uint64_t turn) {
    const uint32_t quarter = (uint32_t)((turn + (1ull << 61)) >> 62);
    const int32_t rest = (int32_t)((turn - ((uint64_t)quarter << 62)) >> 32);  // -2^29 .. 2^29, in 2^-32 turns
    float s, c;
    sincospif((float)rest * 0x1p-31f, &s, &c);
    const float x = quarter & 1 ? s : c, y = quarter & 1 ? c : s;
    return make_float2((quarter + 1) & 2 ? -x : x, quarter & 2 ? -y : y);
}

// Sixteen dims of a head as two runs of eight.
template <typename T> struct Unit16 {
    static constexpr int V = sizeof(T) / 2;  // 16-byte vectors of eight dims
    uint4 a[V], b[V];
    __device__ __forceinline__ void load(const T* pa, const T* pb) {
#pragma unroll
        for (int i = 0; i < V; ++i) a[i] = reinterpret_cast<const uint4*>(pa)[i];
#pragma unroll
        for (int i = 0; i < V; ++i) b[i] = reinterpret_cast<const uint4*>(pb)[i];
    }
    __device__ __forceinline__ void store(T* pa, T* pb) const {
#pragma unroll
        for (int i = 0; i < V; ++i) reinterpret_cast<uint4*>(pa)[i] = a[i];
#pragma unroll
        for (int i = 0; i < V; ++i) reinterpret_cast<uint4*>(pb)[i] = b[i];
    }
    __device__ __forceinline__ float get(int i) const {
        return to_f<T>(reinterpret_cast<const T*>(i < 8 ? a : b)[i & 7]);
    }
    __device__ __forceinline__ void set(int i, float x) {
        reinterpret_cast<T*>(i < 8 ? a : b)[i & 7] = from_f<T>(x);
    }
};

// Slots: the (layer, head) pairs of part 0, then those of part 1.
struct Slot {
    const char* src;
    char* dst;
};
template <typename T>
__device__ __forceinline__ Slot find_slot(const RopeArgs& a, int slot, int slots0, long long row) {
    const bool second = slot >= slots0;
    const blend_rope_rows& p = a.part[second ? 1 : 0];
    const unsigned at = (unsigned)(second ? slot - slots0 : slot);
    const unsigned layer = p.n_layers == 1 ? 0u : at / (unsigned)p.heads, head = at - layer * (unsigned)p.heads;
    return {(const char*)((const T*)p.src + layer * p.src_layer + row * p.src_row + (long long)head * a.head_dim),
            (char*)((T*)p.dst + layer * p.dst_layer + row * p.dst_row + (long long)head * a.head_dim)};
}

// heads_in: slots that a row's threads work on side by side (a power of two); each thread takes every
// heads_in-th slot.
template <typename T, bool PAIRS>
__global__ void __launch_bounds__(ROPE_THREADS, 4)
    k_rope_rows(const __grid_constant__ RopeArgs a, int units_log2, int heads_in_log2, int slots, int slots0) {
    const long long t = (long long)blockIdx.x * ROPE_THREADS + threadIdx.x;
    const int unit = (int)t & ((1 << units_log2) - 1);
    const int first = (int)(t >> units_log2) & ((1 << heads_in_log2) - 1);
    const long long row = t >> (units_log2 + heads_in_log2);
    if (row >= a.max_n) return;
    const int rot = __ldg(a.rot + row);
    int n = __ldg(a.n);
    if (n < 0 || n > a.max_n) {
        if (t == 0) set_error(a.err, BLEND_EDEVICE);
        n = n < 0 ? 0 : a.max_n;
    }
    if (row >= n) return;
    if (rot > ROPE_MAX_SHIFT || rot < -ROPE_MAX_SHIFT) {
        set_error(a.err, BLEND_EDEVICE);
        return;
    }
    const int rot_units = a.rot_dim / 16;
    const bool turned = unit < rot_units && !(rot == 0 && a.magnitude == 1.f);
    const int ia = !PAIRS && unit < rot_units ? unit * 8 : unit * 16;
    const int ib = !PAIRS && unit < rot_units ? ia + a.rot_dim / 2 : ia + 8;
    float2 cs[8];
    if (turned) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            cs[i] = unit_circle((uint64_t)(int64_t)rot * a.freq[unit * 8 + i]);
            cs[i].x *= a.magnitude;
            cs[i].y *= a.magnitude;
        }
    }
    if (!turned && a.part[0].src == a.part[0].dst && (a.n_parts == 1 || a.part[1].src == a.part[1].dst)) return;
    // U slots' loads are on their way together
    constexpr int U = 2;
    const int step = 1 << heads_in_log2;
    auto turn = [&](Unit16<T>& x) {
        if (!turned) return;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int j1 = PAIRS ? 2 * i : i, j2 = PAIRS ? 2 * i + 1 : i + 8;
            const float x1 = x.get(j1), x2 = x.get(j2);
            x.set(j1, x1 * cs[i].x - x2 * cs[i].y);
            x.set(j2, x2 * cs[i].x + x1 * cs[i].y);
        }
    };
    int slot = first;
    for (; slot + (U - 1) * step < slots; slot += U * step) {
        Unit16<T> x[U];
        Slot s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            s[u] = find_slot<T>(a, slot + u * step, slots0, row);
            x[u].load((const T*)s[u].src + ia, (const T*)s[u].src + ib);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            turn(x[u]);
            x[u].store((T*)s[u].dst + ia, (T*)s[u].dst + ib);
        }
    }
    for (; slot < slots; slot += step) {
        const Slot s = find_slot<T>(a, slot, slots0, row);
        Unit16<T> x;
        x.load((const T*)s.src + ia, (const T*)s.src + ib);
        turn(x);
        x.store((T*)s.dst + ia, (T*)s.dst + ib);
    }
}

int log2_floor(long long x) {
    int l = 0;
    while ((x >> (l + 1)) > 0) ++l;
    return l;
}

}  // namespace

void launch_rope_rows(int dtype, const RopeArgs& a, cudaStream_t s) {
    const int units_log2 = a.head_dim == 128 ? 3 : 2;
    const int slots0 = a.part[0].heads * a.part[0].n_layers;
    const int slots = slots0 + (a.n_parts > 1 ? a.part[1].heads * a.part[1].n_layers : 0);
    // Slots side by side: as many as fill the GPU (152 SMs of 1024 threads), not more, since every thread
    // computes its eight angles before it starts; a power of two, at most the slots.  (4099 rows x 48 heads: 20.8 us; each
    // thread over all heads of its row 31, one head a thread 31; 16064 rows x 64 slots: 87, 91 and 198.)
    const long long per_row = (long long)a.max_n << units_log2;
    int want = 0;
    while (want < log2_floor(slots) && (per_row << want) < 152ll * 1024) ++want;
    if ((1 << want) < slots && (per_row << want) < 152ll * 1024) ++want;
    const long long threads = per_row << want;
    const unsigned grid = (unsigned)((threads + ROPE_THREADS - 1) / ROPE_THREADS);
#define GO(T, P) k_rope_rows<T, P><<<grid, ROPE_THREADS, 0, s>>>(a, units_log2, want, slots, slots0)
    if (dtype == BLEND_BF16) {
        if (a.pairs) GO(bf16, true);
        else GO(bf16, false);
    } else {
        if (a.pairs) GO(float, true);
        else GO(float, false);
    }
#undef GO
    note_launch();
}

}  // namespace blend

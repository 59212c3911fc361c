// What the kernels of products with 4-bit weights share (layout in blend.h at blend_w4).
#pragma once
#include <atomic>
#include <mutex>

#include "attn_tc.cuh"
#include "paged.cuh"
#include "tokens.cuh"

namespace blend {
namespace {  // every translation unit uses a part of them

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// Scales of one row's chunk: 128 / G bf16.
template <int G> struct Scales;
template <> struct Scales<32> {
    uint2 v;
    __device__ __forceinline__ void load(const bf16* p) { v = __ldg((const uint2*)p); }
    __device__ __forceinline__ void load_shared(const char* p, int) { v = *(const uint2*)p; }
    __device__ __forceinline__ float get(int i) const {
        const uint32_t w = i < 2 ? v.x : v.y;
        return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
    }
};
template <> struct Scales<64> {
    uint32_t v;
    __device__ __forceinline__ void load(const bf16* p) { v = __ldg((const uint32_t*)p); }
    __device__ __forceinline__ void load_shared(const char* p, int) { v = *(const uint32_t*)p; }
    __device__ __forceinline__ float get(int i) const { return __uint_as_float(i & 1 ? v & 0xffff0000u : v << 16); }
};
template <> struct Scales<128> {
    unsigned short v;
    __device__ __forceinline__ void load(const bf16* p) { v = __ldg((const unsigned short*)p); }
    __device__ __forceinline__ void load_shared(const char* p, int odd) { v = *(const unsigned short*)(p + 2 * odd); }
    __device__ __forceinline__ float get(int) const { return __uint_as_float((uint32_t)v << 16); }
};

constexpr int WAIT_LIMIT = 1 << 24;

// shared::cluster address of this CTA's variable in CTA `rank` of the cluster, and a load from one
__device__ __forceinline__ uint32_t peer_addr(const void* p, int rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(su32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ float ld_peer(uint32_t at) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_peer4(uint32_t at) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
    return v;
}
// A warp's wait for a phase that other CTAs' arrivals end, and its arrival on a barrier in n CTAs of the
// cluster.  (They are looked at without blocking: a blocking look resumes late after an arrival from outside.)
__device__ __forceinline__ bool cluster_phase(uint64_t* b, uint32_t par, volatile int* abort_flag) {
    bool done = false;
#pragma unroll 1
    for (int i = 0; i < WAIT_LIMIT && !done; ++i) {
        uint32_t p;
        asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}\n"
                     : "=r"(p)
                     : "r"(su32(b)), "r"(par)
                     : "memory");
        done = p != 0;
        if (!done && *abort_flag) break;
    }
    return __all_sync(0xffffffffu, done);
}
__device__ __forceinline__ void meet(uint64_t* b, int first, int n) {
    __syncwarp();
    const int lane = threadIdx.x & 31;
    if (lane < n)
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(peer_addr(b, first + lane)) : "memory");
    __syncwarp();
}
// One lane of a converged warp, in a form that the compiler knows to be one.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
    return p != 0;
}

}  // namespace

// What launches of a kernel need once on every device: a kernel's limits belong to a device's context.  `make` fills a T
// (with a bool `ok`) on the current device; only what succeeded is kept.  NULL where it did not.
template <typename T> class PerDevice {
    static constexpr int MAX = 64;
    std::mutex lock;
    std::atomic<bool> made[MAX] = {};
    T of[MAX];

public:
    template <typename Make> const T* get(Make make) {
        int d = -1;
        if (cudaGetDevice(&d) != cudaSuccess || d < 0 || d >= MAX) return nullptr;
        if (made[d].load(std::memory_order_acquire)) return &of[d];
        std::lock_guard<std::mutex> hold(lock);
        if (!made[d].load(std::memory_order_relaxed)) {
            of[d] = make();
            if (!of[d].ok) return nullptr;
            made[d].store(true, std::memory_order_release);
        }
        return &of[d];
    }
};

// A tensor map of the codes: boxes of `rows` weight rows by one chunk, 64-byte swizzle; of the inputs: boxes of `rows` rows by
// 64 bf16, 128-byte swizzle.  False where they cannot be described.
bool w4_encode_codes(CUtensorMap* map, const W4View& w, int rows);
bool w4_encode_inputs(CUtensorMap* map, const W4Linear& a, int rows);

// Many rows of bf16 inputs on tcgen05 (w4_tile.cu): k of 64 and n of 128 at least.  BLEND_EUNSUPPORTED where it
// cannot run.
int launch_w4_tile(const W4Linear& a, cudaStream_t s);

}  // namespace blend

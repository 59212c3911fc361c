// What the kernels of products with 4-bit weights share (layout in blend.h at blend_w4).
#pragma once
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
    __device__ __forceinline__ float get(int i) const {
        const uint32_t w = i < 2 ? v.x : v.y;
        return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
    }
};
template <> struct Scales<64> {
    uint32_t v;
    __device__ __forceinline__ void load(const bf16* p) { v = __ldg((const uint32_t*)p); }
    __device__ __forceinline__ float get(int i) const { return __uint_as_float(i & 1 ? v & 0xffff0000u : v << 16); }
};
template <> struct Scales<128> {
    unsigned short v;
    __device__ __forceinline__ void load(const bf16* p) { v = __ldg((const unsigned short*)p); }
    __device__ __forceinline__ float get(int) const { return __uint_as_float((uint32_t)v << 16); }
};

}  // namespace

// Many rows of bf16 inputs on tcgen05 (w4_tile.cu): k of 64 and n of 128 at least.  BLEND_EUNSUPPORTED where it
// cannot run.
int launch_w4_tile(const W4Linear& a, cudaStream_t s);

}  // namespace blend

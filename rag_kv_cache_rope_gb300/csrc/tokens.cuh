// What follows the finished cache, per generated token: products with 4-bit weights, log
// probabilities, rotary positions.  Launch interfaces.
#pragma once
#include "common.cuh"

namespace blend {

// Do rows [layers][n][width] at pa and pb meet?  (Bytes.)  Exact where both step alike, so that rows which lie side by side in one
// buffer do not, although their ranges do; rows that step differently count as meeting where their ranges meet.  A
// step that a tensor does not take (one row, one layer) does not matter.
inline bool rows_meet(const void* pa, long long row_a, long long layer_a, long long layers_a, long long wa, const void* pb,
                      long long row_b, long long layer_b, long long layers_b, long long wb, long long n) {
    const long long d = (long long)((intptr_t)pb - (intptr_t)pa);  // b's place from a's
    const long long end_a = (layers_a - 1) * (layers_a > 1 ? layer_a : 0) + (n - 1) * row_a + wa;
    const long long end_b = (layers_b - 1) * (layers_b > 1 ? layer_b : 0) + (n - 1) * row_b + wb;
    if (d >= end_a || -d >= end_b) return false;
    if ((n > 1 && row_a != row_b) || (layers_a > 1 && layers_b > 1 && layer_a != layer_b)) return true;
    const long long layer = layers_a > 1 ? layer_a : layers_b > 1 ? layer_b : 0;
    // a row of b and one of a, l layers and i rows apart: b's begins at + i row_a behind a's
    for (long long l = 1 - layers_a; l < layers_b; ++l) {
        const long long at = d + l * layer, end = -wb - at;
        long long i = 0;  // the first step with which b's row ends behind a's start
        if (n > 1) {
            i = end / row_a - (end % row_a < 0) + 1;
            if (i < 1 - n) i = 1 - n;
        }
        if (i < n && at + i * row_a < wa && at + i * row_a > -wb) return true;
    }
    return false;
}

// Do `bytes` bytes at p meet rows [layers][n][width] at pa?  (Exact.)
inline bool bytes_meet_rows(const void* p, long long bytes, const void* pa, long long row, long long layer, long long layers,
                            long long width, long long n) {
    const long long d = (long long)((intptr_t)p - (intptr_t)pa);
    if (d >= (layers - 1) * (layers > 1 ? layer : 0) + (n - 1) * row + width || d + bytes <= 0) return false;
    for (long long l = 0; l < layers; ++l) {
        const long long at = d - (layers > 1 ? l * layer : 0), end = at - width;
        // the first row that ends behind p
        long long i = end / row - (end % row < 0) + 1;
        if (i < 0) i = 0;
        if (i < n && i * row < at + bytes) return true;
    }
    return false;
}

// ---- 4-bit weights (w4.cu); layout in blend.h at blend_w4
struct W4View {
    const uint4* codes;  // [n][4 chunks] sixteen-byte pieces
    const bf16* scale;   // [n][chunks * 128 / group]
    int n, k, group, chunks;
};
void launch_w4_pack(int dtype, const W4View& w, const void* src, long long ld, cudaStream_t s);
void launch_w4_unpack(int dtype, const W4View& w, void* out, long long ld, cudaStream_t s);
struct W4Linear {
    W4View w;
    const void* x;
    long long ld_x;
    int rows;
    void* y;
    long long ld_y;
    int y_f32, epi;
    bool tc;  // tcgen05 may be used
    int32_t* err;
};
// x of `dtype`.  Returns BLEND_OK or the code of a failed launch set-up.
int launch_w4_linear(int dtype, const W4Linear& a, cudaStream_t s);

// ---- log probabilities (logprobs.cu)
struct Logprobs {
    const void* logits;
    long long ld;
    int rows, vocab;
    float scale;
    const int32_t* ids;
    int n_ids;
    float* logp;
    float* entropy;
    int top;
    int32_t* top_id;
    float* top_logp;
    int32_t* err;
};
int launch_logprobs(int dtype, const Logprobs& a, cudaStream_t s);

// ---- rotary positions (rope_rows.cu)
constexpr int ROPE_MAX_SHIFT = 1 << 24;
struct RopeArgs {
    blend_rope_rows part[2];
    int n_parts, max_n, rot_dim, head_dim;
    int pairs;        // BLEND_ROPE_PAIRS
    float magnitude;
    const int32_t* rot;
    const int32_t* n;
    int32_t* err;
    uint64_t freq[64];  // each pair's turn per position, in 2^-64 of a turn
};
void launch_rope_rows(int dtype, const RopeArgs& a, cudaStream_t s);

}  // namespace blend

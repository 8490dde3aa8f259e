// Launchers of the block-scaled FP8 operators: E4M3 codes with one fp32 scale
// per 128 values along K (activations) or per 128 x 128 block (weights).
#pragma once

#include "common.hpp"

namespace fp8q {

constexpr int kBlock = 128;              // values per scale along K, weight rows per scale
inline int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }

// x[rows, cols] -> codes and scale[K blocks, rows], one per 1 x 128 block.
hipError_t launch_quantize_blocks(const void* x, int dtype, int64_t rows, int64_t cols, uint8_t* q,
                                  float* scale, hipStream_t stream);
// w[batch, rows, cols] -> codes and scale[batch, row blocks, K blocks].
hipError_t launch_quantize_weight_blocks(const void* w, int dtype, int64_t batch, int64_t rows,
                                         int64_t cols, uint8_t* q, float* scale,
                                         hipStream_t stream);

// The product of block-scaled codes, sa[K blocks, M] and sw[N blocks, K
// blocks], on the kernel that product_block_kernel names: weight streaming up
// to kDecodeBlockMaxM tokens and for few outputs, LDS tiles else.
constexpr int kDecodeBlockMaxM = 16;
hipError_t launch_product_block(const uint8_t* qa, const float* sa, const uint8_t* qw,
                                const float* sw, uint16_t* y, int M, int N, int K,
                                hipStream_t stream);
const char* product_block_kernel(int M, int N, int K);
// Quantizer and product in one launch, taken where linear_block_fused_pays.
constexpr int kFusedBlockMaxCells = 256; // 1 x 128 blocks of the activation
bool linear_block_fused_pays(int64_t M, int64_t N, int64_t K);
hipError_t launch_linear_block_fused(const void* x, int dtype, const uint8_t* qw, const float* sw,
                                     uint16_t* y, uint8_t* q, float* sa, int M, int N, int K,
                                     hipStream_t stream);

// A mixture-of-experts layer for a few tokens (see moe.hip).
constexpr int kMoeMaxTokens = 64;
constexpr int kMoeMaxExperts = 512;
constexpr int kMoeMaxTopK = 16;
constexpr int64_t kMoeMaxDim = 1 << 16;  // H and I
struct MoeArgs {
    const void* x;           // [T, H]
    const float* logits;     // [T, E]
    const uint8_t* w13;      // [E, 2, I, H]
    const float* s13;        // [E, 2, I blocks, H blocks]
    const uint8_t* w2;       // [E, H, I]
    const float* s2;         // [E, H blocks, I blocks]
    uint16_t* y;             // [T, H]
    int* ids;                // [T, top_k]
    float* weights;          // [T, top_k]
    void* work;              // moe_work_bytes
    int T, H, I, E, top_k, renormalize;
};
int64_t moe_work_bytes(int64_t T, int64_t I, int64_t top_k);
hipError_t launch_moe(const MoeArgs& a, int dtype, hipStream_t stream);

}  // namespace fp8q

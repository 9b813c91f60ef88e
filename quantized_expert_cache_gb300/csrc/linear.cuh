// Weight layout of the dense 4-bit layers, shared by their kernels.
#pragma once
#include "common.cuh"
#include "kernels.h"

namespace moe {

constexpr int kKB = 8;            // blocks of a group
constexpr int kARec = 16 * 18;    // bytes of 16 rows of a Q4_0 block

// bytes of a group of n blocks of 16 rows, and of all nb blocks of 16 rows
__host__ __device__ constexpr int group_bytes(int fmt, int n) { return n * kARec + (fmt == kFmtQ4K ? 64 : 0); }
__host__ __device__ inline size_t tile_bytes(int fmt, int nb) {
    return (size_t)nb * kARec + (fmt == kFmtQ4K ? (size_t)(nb / kKB) * 64 : 0);
}

// Q4_K: the rows' powers of two (kernels_linear_gemm.cu), fp32, whole tiles of
// 128 rows, stand after the blocks.
__host__ __device__ inline size_t row_scale_offset(int fmt, int rows, int nb) {
    return (size_t)((rows + 15) / 16) * tile_bytes(fmt, nb);
}
constexpr int kScaleRows = 128;

}  // namespace moe

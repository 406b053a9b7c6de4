// The table of tensors that one launch of the gradient-norm kernels works on, passed by
// value in the kernel's parameters.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace flce {

constexpr int kTableTensors = 112;   // 29 bytes each: within the 4 KB of plain parameters

struct ClipTable {
  const void* src[kTableTensors];
  void* dst[kTableTensors];        // null: the norm only
  int64_t numel[kTableTensors];
  int first[kTableTensors];        // piece index of the tensor's first piece
  uint8_t bf16[kTableTensors];
  int count;
  int pieces;                      // of all tensors of the table
  float density;                   // count / pieces
};

int clip_piece_bytes();

// part[b] = sum of squares of the pieces of CTA b.
cudaError_t launch_grad_squares(const ClipTable& tab, double* part, int grid, cudaStream_t stream);

// Sums the `parts` partials of all tables, writes the norm (norm not null) and scales
// the table's pieces.
cudaError_t launch_grad_scale(const ClipTable& tab, const double* part, int parts, float max_norm,
                              float* norm, int grid, cudaStream_t stream);

}  // namespace flce

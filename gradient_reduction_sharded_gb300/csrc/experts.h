// The experts' products between kernels_experts.cu (calls, any size and type)
// and kernels_experts_mma.cu (bf16 on the tensor cores).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"

namespace grs {

// Every product is O[c][f] = sum over k of A[f][k] B[c][k] for each expert:
//   kForward  f an output feature of w,  c a row, k an input feature
//   kRows     f an input feature of w,   c a row, k an output feature
//   kWeights  f an input feature of xs,  c an output feature of dys, k a row
// so that f is what lies next to one another in the result and the expert's
// rows, of which only the device knows how many, are c or k.
enum class Product { kForward, kRows, kWeights };

struct ExpLd {
  int64_t x, y, w;  // elements from one row to the next of xs and dxs, of ys and dys, of w
};

// One product in bf16; xs, w and dys 16-byte aligned, the row distances of
// those that it reads multiples of 8.  o_ld: of the result's rows.
cudaError_t experts_mma(Product p, const grs_experts* s, const ExpLd& ld, const void* xs, const void* w, const void* dys,
                        const int32_t* offsets, void* o, int64_t o_ld, void* stream);

}  // namespace grs

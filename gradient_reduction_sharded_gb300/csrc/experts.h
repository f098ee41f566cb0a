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

// The self-test has the loads of block `quitter` give up at its `tile`th tile.
struct ExpQuit {
  int32_t quitter = -1, tile = 0;
};

// Where a product has few tiles with a long k, k is cut into slices whose
// results (fp32) are added up afterwards.
struct ExpSlices {
  int n = 1;
  float* parts = nullptr;       // [n][rows of the result][ld]
  int64_t ld = 0, distance = 0;  // of its rows, of the slices
};

// k of a slice: in 512s on the tensor cores and 64s elsewhere, so that the sections of an fp32 sum are whole ones.
template <int kSection>
__host__ __device__ inline int64_t slice_length(int64_t k, int32_t slices) {
  return ((k + slices - 1) / slices + kSection - 1) / kSection * kSection;
}

// Tiles that a product in bf16 has at most, how many columns they have, and how long k is (in the mean).
struct ExpTiles {
  int columns;
  int64_t n, k;
};
ExpTiles experts_mma_tiles(Product p, const grs_experts* s);

// One product in bf16; xs, w and dys 16-byte aligned, the row distances of
// those that it reads multiples of 8.  o_ld: of the result's rows.
cudaError_t experts_mma(Product p, const grs_experts* s, const ExpLd& ld, const void* xs, const void* w, const void* dys,
                        const int32_t* offsets, void* o, int64_t o_ld, const ExpSlices& slices, const ExpQuit& quit, void* stream);

}  // namespace grs

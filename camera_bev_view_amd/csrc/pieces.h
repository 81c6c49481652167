// Pieces of neighbouring channels that a lane moves at a time.
#pragma once

#include <hip/hip_runtime.h>

namespace fbev {

template <typename T, int V>
struct alignas(sizeof(T) * V) Piece {
  T e[V];
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__bf16 x) { return (float)x; }

}  // namespace fbev

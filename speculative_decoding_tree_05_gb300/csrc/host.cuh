// host.cuh -- host-side checks and set-up shared by the C entry points.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>
#include "../../include/ddtree.h"

namespace ddt {

constexpr size_t kStatusBytes = 256;

// Return codes of include/ddtree.h.
int check_dims(const ddt_dims* d);
struct BlockClusters;  // cache_ops.cuh
// The current device: DDT_OK and its SM count if it is an sm_103 GPU on which the cache-size and block
// kernels are set up; also how many clusters of block attention it runs at once, if asked.
int current_device(int* sm_count, BlockClusters* clusters = nullptr);

struct AcceptClusters;  // accept.cuh
void current_accept_clusters(AcceptClusters* clusters);  // of a device that current_device() has found fit

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + bn && y < x + an;
}

// Rows of 576 bf16 values as a 2-D tensor, box of box_cols columns (64: 128-byte
// swizzle, 32: 64-byte) x box_rows rows; rows past the tensor read as zero.
bool encode_pool_map(CUtensorMap* m, const void* pool, int64_t rows, uint32_t box_cols, uint32_t box_rows);
// Rows of 640 bytes, box of 128 bytes x one row, 128-byte swizzle.
bool encode_kv8_map(CUtensorMap* m, const void* pool, int64_t rows);

}  // namespace ddt

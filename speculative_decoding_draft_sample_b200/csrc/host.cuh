// Host-side helpers shared by the C ABI's translation units.
#pragma once

#include <atomic>

#include "common.cuh"

namespace dspark {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA; }

// Sizes of a [B, K, V] logit tensor that the calls take.
inline bool shape_ok(int B, int K, int V, int dtype) {
  if (dtype != DSPARK_F32 && dtype != DSPARK_BF16) return false;
  if (B < 1 || B > 65535 || K < 1 || K > 64) return false;
  if (V < 8 || V >= (1 << 24) || V % 8 != 0) return false;
  return true;
}

// Sizes of a [M, H] norm (a row stays in its CTA's registers).
inline bool norm_shape_ok(int M, int H) { return M >= 1 && H >= 8 && H <= 16384 && H % 8 == 0; }

// Sizes of an [M, K] x [N, K] product: rows of K entries are whole 16-byte units.
inline bool linear_shape_ok(int M, int N, int K, int in_type) {
  if (in_type != DSPARK_BF16 && in_type != DSPARK_E4M3) return false;
  if (M < 1 || M >= (1 << 24) || N < 1 || N >= (1 << 24) || K < 1 || K >= (1 << 20)) return false;
  return K % (in_type == DSPARK_E4M3 ? 16 : 8) == 0;
}

// DSPARK_OK on a device of compute capability 10.0 (the fatbin carries sm_100a
// code only), and its SM count. Both are fixed for the life of the process, so
// each device is asked once (a query costs a call about 1 us of host time).
inline int device_check(int* num_sms) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];  // 0 unknown, -1 unsupported, else the SM count
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DSPARK_ERR_CUDA;
  int sms = dev < kDevices ? known[dev].load(std::memory_order_relaxed) : 0;
  if (sms == 0) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return DSPARK_ERR_CUDA;
    if (major != 10 || minor != 0) sms = -1;
    if (dev < kDevices) known[dev].store(sms, std::memory_order_relaxed);
  }
  if (sms < 0) return DSPARK_ERR_UNSUPPORTED;
  if (num_sms) *num_sms = sms;
  return DSPARK_OK;
}

}  // namespace dspark

// probe_adamw.hip - test-only kernels that hold the AdamW step's square root and
// quotient (precision_state_amd/csrc/dev_adamw.h) against the library's over
// whole ranges, for tests/test_gpu_adamw_exact.py. Part of libps_probe.so.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../precision_state_amd/csrc/dev_adamw.h"

namespace {

constexpr int kThreads = 256;
constexpr uint32_t kGrid = 16384;

__device__ void count(uint32_t n, unsigned long long* out) {
  if (n) atomicAdd(out, (unsigned long long)n);
}

// Fp32 bit patterns first .. first + n - 1 whose sqrt_fast differs from the root.
__global__ __launch_bounds__(kThreads) void k_root_diff(uint32_t first, uint32_t n, unsigned long long* out) {
  uint32_t bad = 0;
  for (uint64_t i = blockIdx.x * kThreads + threadIdx.x; i < n; i += kGrid * kThreads) {
    const float v = __uint_as_float(first + (uint32_t)i);
    bad += __float_as_uint(ps::sqrt_fast(v)) != __float_as_uint(__builtin_sqrtf(v));
  }
  count(bad, out);
}

// Every mantissa of d with `rounds` numerators each: random ones, and ones next
// to d times a point half way between two floats, where a quotient's rounding
// is hardest. ea, ed: exponents.
__global__ __launch_bounds__(kThreads) void k_quotient_diff(int ea, int ed, uint32_t rounds, uint32_t seed,
                                                            unsigned long long* out) {
  uint32_t bad = 0;
  for (uint32_t i = blockIdx.x * kThreads + threadIdx.x; i < (1u << 23); i += kGrid * kThreads) {
    const float d = __uint_as_float(((uint32_t)(ed + 127) << 23) | i);
    for (uint32_t k = 0; k < rounds; ++k) {
      const uint64_t z = ps::splitmix64_mix(((uint64_t)seed << 40) + ((uint64_t)i << 16) + k);
      float a;
      if (k & 1) {
        const double half = 1.0 + ((double)(z & 0x7FFFFF) + 0.5) * 0x1p-23;
        const float near = (float)((double)__uint_as_float(0x3F800000u | i) * half);   // in [1, 4)
        const int step = (int)((z >> 32) % 3) - 1;
        a = __builtin_ldexpf(__uint_as_float(__float_as_uint(near) + step), ea);
      } else {
        a = __uint_as_float(((uint32_t)(ea + 127) << 23) | (uint32_t)(z & 0x7FFFFF));
      }
      if (z >> 63) a = -a;
      bad += __float_as_uint(ps::div_fast(a, d)) != __float_as_uint(a / d);
    }
  }
  count(bad, out);
}

}  // namespace

extern "C" {

int probe_root_diff(uint32_t first, uint32_t n, unsigned long long* out, hipStream_t s) {
  hipLaunchKernelGGL(k_root_diff, dim3(kGrid), dim3(kThreads), 0, s, first, n, out);
  return (int)hipGetLastError();
}

int probe_quotient_diff(int ea, int ed, uint32_t rounds, uint32_t seed, unsigned long long* out, hipStream_t s) {
  if (ea < -60 || ea > 57 || ed < -60 || ed > 59) return -1;
  hipLaunchKernelGGL(k_quotient_diff, dim3(kGrid), dim3(kThreads), 0, s, ea, ed, rounds, seed, out);
  return (int)hipGetLastError();
}

}  // extern "C"

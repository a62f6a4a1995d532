// Host-side helpers shared by the C ABI's translation units: scratch rounding,
// alignment, the tensor-map encoder and the rotary angles.
#pragma once

#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cmath>
#include <mutex>

#include "jl_kernels.cuh"

namespace jl {

constexpr size_t kAlign = 256;
inline size_t round_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

inline int device_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
  return n;
}

inline void fill_theta(double* theta, int D, double base) {
  for (int t = 0; t < D / 2; ++t) theta[t] = std::pow(base, -2.0 * t / D);
}

// theta_t / (2 pi) as u_hi + u_lo, u_hi rounded to 22 significant bits (so that
// n * u_hi is exact in fp64 for |n| < 2^31; see sincos_int_angle).
inline void fill_turns(double* u_hi, double* u_lo, const double* theta, int D) {
  for (int t = 0; t < D / 2; ++t) {
    const double u = theta[t] / 6.283185307179586;
    int e = 0;
    const double m = std::frexp(u, &e);
    u_hi[t] = std::ldexp(std::nearbyint(std::ldexp(m, 22)), e - 22);
    u_lo[t] = u - u_hi[t];
  }
}

inline float resolve_scale(float s, int D) { return s == 0.f ? 1.0f / std::sqrt((float)D) : s; }

// theta_t / (2 pi) of one (head_dim, rope_base), as fill_turns splits it and its
// fraction in 64-bit fixed point.
struct TurnTable {
  double hi[kMaxHalfDim], lo[kMaxHalfDim];
  uint64_t fixed[kMaxHalfDim];
};

// The table for (D, base).  Each thread keeps the last one it formed (64 pow and
// frexp calls, about 3 us, against a launch's 2 us): a model has one base.
inline const TurnTable& turn_table(int D, double base) {
  struct Last {
    int D = 0;
    double base = 0.0;
    TurnTable t;
  };
  static thread_local Last last;
  if (last.D != D || last.base != base) {
    double theta[kMaxHalfDim];
    fill_theta(theta, D, base);
    fill_turns(last.t.hi, last.t.lo, theta, D);
    for (int t = 0; t < D / 2; ++t) {
      const double u = theta[t] / 6.283185307179586;  // whole turns of theta itself change no integer multiple
      last.t.fixed[t] = (uint64_t)std::ldexp(u - std::floor(u), 64);
    }
    last.D = D;
    last.base = base;
  }
  return last.t;
}

}  // namespace jl

// vq_turn.cuh -- sine and cosine of a 64-bit fraction of a turn, in 64 bits.  Compiles for the host too.
#pragma once

#include <cuda_runtime.h>

namespace vqk {

// By the series of sine and cosine around the nearest quarter turn: |x| <= pi / 4, where the terms left out are under
// x^17 / 17! = 4.7e-17 and x^18 / 18! = 2.1e-18.  The fraction is taken apart as whole numbers, so what is off is the rounding
// of x (2^-52 relative) and of the sums.
__host__ __device__ inline void turn_sincos(unsigned long long turn, double& si, double& co) {
  const unsigned quarter = static_cast<unsigned>((turn + (1ULL << 61)) >> 62);  // (of a turn; 4: none)
  const double x = static_cast<double>(static_cast<long long>(turn - (static_cast<unsigned long long>(quarter) << 62))) * 3.4061215800865545e-19;  // 2 pi / 2^64
  const double x2 = x * x;
  double s = -1.0 / 1307674368000.0, c = 1.0 / 20922789888000.0;  // 15!, 16!
  s = s * x2 + 1.0 / 6227020800.0;
  c = c * x2 - 1.0 / 87178291200.0;
  s = s * x2 - 1.0 / 39916800.0;
  c = c * x2 + 1.0 / 479001600.0;
  s = s * x2 + 1.0 / 362880.0;
  c = c * x2 - 1.0 / 3628800.0;
  s = s * x2 - 1.0 / 5040.0;
  c = c * x2 + 1.0 / 40320.0;
  s = s * x2 + 1.0 / 120.0;
  c = c * x2 - 1.0 / 720.0;
  s = s * x2 - 1.0 / 6.0;
  c = c * x2 + 1.0 / 24.0;
  s = s * x2 * x + x;
  c = (c * x2 - 0.5) * x2 + 1.0;
  const bool swapped = quarter & 1u;
  si = swapped ? c : s;
  co = swapped ? s : c;
  if (quarter & 2u) si = -si;
  if ((quarter + 1u) & 2u) co = -co;
}

}  // namespace vqk

// csrc/vq_turn.cuh, run on the host.
#include "../bit_vector_quantized_gb300/csrc/vq_turn.cuh"

extern "C" void turn_sincos_host(const unsigned long long* turn, long long n, double* si, double* co) {
  for (long long i = 0; i < n; ++i) vqk::turn_sincos(turn[i], si[i], co[i]);
}

// vq_rotary.cu -- rotary positions of queries and keys before they are cached (sm_103a).
//
// Pair i of a head's first `rotary_dim` elements turns by the angle
// x = position * f_i:  (a, b) -> m (a cos x - b sin x, b cos x + a sin x),
// the pairs being (2i, 2i + 1) or (i, i + rotary_dim / 2); the other elements
// pass through.  The values of a fused projection are carried along, so one
// call turns the projection's rows into the contiguous fp16 rows that
// vq_encode_kv and the attention calls read.
//
// Angle.  position * f_i in fp32 is off by 0.01 rad at 200 000 positions, so
// the host passes f_i / 2 pi as a 64-bit fraction of a turn and the kernel
// forms position * fraction modulo 2^64: an exact reduction to one turn (off
// by position * 2^-53 turns from the host's double), whose upper 32 bits go
// to sincospi as fp32 (2^-25 of a half turn).
//
// Work split.  The kernel is bound by the bytes it moves: 2 bytes in and 2
// out per element.  Eight threads serve a token, each two 16-byte pieces (8
// pairs) of every head, so a pair's sine and cosine are formed once and used
// for all heads of the thread's share, and every access is 16 bytes.  Few
// tokens: the heads are spread over more threads (blockIdx.y), which form the
// angles again, until every SM has about 1000 threads.  Four heads' loads go
// out before the first use.  The arithmetic is fp32, rounded once to fp16.
// Measured: 32 768 tokens of 48 heads (805 MB) in 127.6 us, 6.31 TB/s, 0.93 of
// the measured copy rate (the whole call 133 us); 4099 tokens of 56 bf16 heads
// in 21.6 us (floor 17).
#include "vq_rotary.cuh"

namespace vqk {
namespace {

template <bool kBf16, bool kWhole>
__global__ void __launch_bounds__(kRotThreads) vq_rotary_kernel(const RotaryParams p) {
  rotary_share<kBf16, kWhole>(p, blockIdx.x, blockIdx.y);
}

}  // namespace

cudaError_t launch_rotary(RotaryParams p, bool bf16, int sms, cudaStream_t stream) {
  const dim3 grid = rotary_grid(p, sms);
  const bool whole = p.interleaved || p.rotary_dim % 16 == 0;
  auto kern = bf16 ? (whole ? vq_rotary_kernel<true, true> : vq_rotary_kernel<true, false>)
                   : (whole ? vq_rotary_kernel<false, true> : vq_rotary_kernel<false, false>);
  kern<<<grid, kRotThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace vqk

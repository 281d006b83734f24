// vq_chunk_common.cuh -- what the chunk-attention kernels share beside the plan (vq_chunk_plan.cuh): the
// sequences' estimated lengths summed by a CTA, the records of cut tiles, and the split of fp32 pairs.
#pragma once

#include "vq_chunk_plan.cuh"
#include "vq_device.cuh"
#include "vq_kernels.h"

namespace vqk {
namespace {

// fp32 pair -> fp16 pairs of the high and low parts, hi + lo == x to about 2^-22 relative
// (split_half2's values, by packed conversions: half the instructions).
__device__ __forceinline__ void split_pair(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x0, x1);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(x0 - f.x, x1 - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

// pre[b] for all sequences (all threads of the CTA; scratch: 32 long longs).
__device__ __forceinline__ void chunk_plan(const ChunkParams& p, long long* pre, long long* scratch) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthr = blockDim.x;
  const int per = (p.batch + nthr - 1) / nthr;
  const int b0 = min(tid * per, p.batch), b1 = min(b0 + per, p.batch);
  long long sum = 0;
  for (int b = b0; b < b1; ++b) {
    bool bad = false;
    const ChunkSeq s = chunk_seq(p, b, bad);
    if (bad && blockIdx.x == 0) report(p.status, kDevBadLength);
    const long long w = p.hkv * chunk_sum(p, s, (s.n + p.tile_tok - 1) / p.tile_tok);
    pre[b] = w;
    sum += w;
  }
  long long in = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, in, o);
    if (lane >= o) in += v;
  }
  if (lane == 31) scratch[warp] = in;
  __syncthreads();
  long long run = in - sum;
  for (int w = 0; w < warp; ++w) run += scratch[w];
  for (int b = b0; b < b1; ++b) {
    const long long w = pre[b];
    pre[b] = run;
    run += w;
  }
  if (tid == nthr - 1) pre[p.batch] = run;
  __syncthreads();
}

// The record of the tile that a worker begins and does not end (or none).
__device__ __forceinline__ void write_record(const ChunkParams& p, int worker, const ChunkPiece* q) {
  ChunkRecord r = {};
  if (q) {
    r.tokens = min(p.tile_tok, q->s.n - q->tile * p.tile_tok);
    r.row0 = q->s.row0 + q->tile * p.tile_tok;
    r.kvh = q->kvh;
    r.last = q->last;
  }
  *reinterpret_cast<int4*>(p.records + worker) = *reinterpret_cast<const int4*>(&r);
}

}  // namespace
}  // namespace vqk

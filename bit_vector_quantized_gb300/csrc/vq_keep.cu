// vq_keep.cu -- the accepted ones of a step's drafted tokens, moved together in all layers' pools (sm_103a).
//
// Sequence b's n drafted tokens sit at places base .. base + n - 1 (base = len - n); token keep[i] moves to
// place base + i, i = 0 .. kept - 1, keep ascending.  So keep[i] >= i: a row is never moved over one that a
// later row still needs, and a warp that moves the rows in order, in pieces of which it has loaded
// all before it stores any, needs no second buffer.
//
// Two launches: the moves (a warp per layer, tensor, KV head and sequence; a CTA stays with one sequence and checks
// it first; loads and stores are one round trip each, so many CTAs), then the lengths and the pages that are left
// empty (one CTA, prefix sums over the sequences), which may overwrite the lengths that the moves read.  Both find the
// same sequences out of range.  6 us for one sequence's path in 32 layers, bound by latency; 15 us for 48 sequences' (7.7 MB),
// of which the moves issue in 54 % of the cycles: a word a lane, with two divisions for its row on either side (two CTAs an SM
// for the moves instead of eight: 19 us).
#include "vq_device.cuh"
#include "vq_kernels.h"

namespace vqk {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kMoveThreads = 256, kBookThreads = 1024;
constexpr int kMoveWords = 8;  // words of a lane under way

struct KeepSeq {
  int base, len, kept;  // kept: -1 where the sequence is left as it is
  int bad;              // the status that says why
};

// The sequence's lengths (not its indices and pages).
__device__ __forceinline__ KeepSeq keep_seq(const KeepParams& p, int b) {
  KeepSeq s;
  s.len = __ldcg(p.seq_lens + b);
  const int c0 = __ldg(p.cu + b), c1 = __ldg(p.cu + b + 1);
  const long long n = static_cast<long long>(c1) - c0;
  s.kept = __ldg(p.keep_lens + b);
  s.bad = kDevOk;
  if (s.len < 0 || s.len > static_cast<long long>(p.max_pages) * p.page_size || n < 0 || n > s.len || s.kept < 0 || s.kept > p.max_keep || s.kept > n) {
    s.kept = -1;
    s.bad = kDevBadLength;
    s.base = s.len;
  } else {
    s.base = static_cast<int>(s.len - n);
  }
  return s;
}

// Index i and the one before it are in order.
__device__ __forceinline__ bool keep_in_order(const KeepParams& p, const KeepSeq& s, int b, int i) {
  const int32_t* const keep = p.keep + static_cast<long long>(b) * p.max_keep;
  const int at = __ldg(keep + i);
  return at >= 0 && at < s.len - s.base && (i == 0 || __ldg(keep + i - 1) < at);
}

__device__ __forceinline__ bool keep_has_page(const KeepParams& p, int b, int page) {
  const int x = __ldg(p.page_table + static_cast<long long>(b) * p.max_pages + page);
  return x >= 0 && x < p.num_pages;
}

__global__ void __launch_bounds__(kMoveThreads) vq_keep_move_kernel(const __grid_constant__ KeepParams p) {
  __shared__ long long from[kKeepMaxTokens], to[kKeepMaxTokens];  // rows of the pool, as KV head 0 has them
  pdl_trigger();
  const int b = blockIdx.x, tid = threadIdx.x, P = p.page_size;
  const KeepSeq s = keep_seq(p, b);
  if (s.kept <= 0) return;
  bool ok = true;
  for (int i = tid; i < s.kept; i += kMoveThreads) ok &= keep_in_order(p, s, b, i);
  for (int page = s.base / P + tid; page <= (s.len - 1) / P; page += kMoveThreads) ok &= keep_has_page(p, b, page);
  if (!__syncthreads_and(ok)) return;
  for (int i = tid; i < s.kept; i += kMoveThreads) {
    const int32_t* const pages = p.page_table + static_cast<long long>(b) * p.max_pages;
    const int src = s.base + __ldg(p.keep + static_cast<long long>(b) * p.max_keep + i), dst = s.base + i;
    from[i] = static_cast<long long>(__ldg(pages + src / P)) * p.hkv * P + src % P;
    to[i] = static_cast<long long>(__ldg(pages + dst / P)) * p.hkv * P + dst % P;
  }
  __syncthreads();
  int first = 0;  // the rows before it stay where they are
  while (first < s.kept && from[first] == to[first]) ++first;
  const int lane = tid & 31, warps = gridDim.y * (kMoveThreads / 32);
  for (int task = blockIdx.y * (kMoveThreads / 32) + (tid >> 5); task < 2 * p.layers * p.hkv; task += warps) {
    const int h = task % p.hkv, which = task / p.hkv & 1, layer = task / p.hkv >> 1;
    const int rb = p.row_bytes[which], rw = rb / 4, words = s.kept * rw;
    uint8_t* const pool = p.pool[which][layer] + static_cast<long long>(h) * P * rb;
    for (int w0 = first * rw; w0 < words; w0 += 32 * kMoveWords) {
      uint32_t x[kMoveWords];
#pragma unroll
      for (int u = 0; u < kMoveWords; ++u) {
        const int w = w0 + 32 * u + lane;
        if (w < words) x[u] = reinterpret_cast<const uint32_t*>(pool + from[w / rw] * rb)[w % rw];
      }
      __syncwarp();
#pragma unroll
      for (int u = 0; u < kMoveWords; ++u) {
        const int w = w0 + 32 * u + lane;
        if (w < words) reinterpret_cast<uint32_t*>(pool + to[w / rw] * rb)[w % rw] = x[u];
      }
      __syncwarp();
    }
  }
}

__global__ void __launch_bounds__(kBookThreads) vq_keep_book_kernel(const __grid_constant__ KeepParams p) {
  __shared__ long long warp_sum[kBookThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, P = p.page_size;
  const int num_free = __ldcg(p.num_free);
  // this thread's run of sequences, checked twice: for the sum, and where the results are written
  auto check = [&](int b) {
    KeepSeq s = keep_seq(p, b);
    if (s.kept < 0) return s;
    for (int i = 0; i < s.kept; ++i)
      if (!keep_in_order(p, s, b, i)) s.bad = kDevBadLength;
    // (nothing kept: only the pages that are given back count, and those are among these)
    for (int page = s.base / P; s.bad == kDevOk && s.base < s.len && page <= (s.len - 1) / P; ++page)
      if (!keep_has_page(p, b, page)) s.bad = kDevBadPage;
    if (s.bad != kDevOk) s.kept = -1;
    return s;
  };
  auto pages = [&](int tokens) { return static_cast<int>((static_cast<unsigned>(tokens) + P - 1u) / P); };
  auto gone = [&](const KeepSeq& s) { return s.kept < 0 ? 0 : pages(s.len) - pages(s.base + s.kept); };
  const int per = (p.batch + kBookThreads - 1) / kBookThreads;
  const int b0 = min(tid * per, p.batch), b1 = min(b0 + per, p.batch);
  long long sum = 0;
  KeepSeq s = {};  // (of one sequence a thread, what it found serves twice)
  for (int b = b0; b < b1; ++b) {
    s = check(b);
    if (s.bad != kDevOk) report(p.status, s.bad);
    sum += gone(s);
  }
  long long in = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(kAll, in, o);
    if (lane >= o) in += x;
  }
  if (lane == 31) warp_sum[tid >> 5] = in;
  __syncthreads();
  long long at = in - sum, all = 0;
  for (int w = 0; w < kBookThreads / 32; ++w) {
    if (w < tid >> 5) at += warp_sum[w];
    all += warp_sum[w];
  }
  const bool fits = num_free >= 0 && num_free <= p.free_capacity && all <= p.free_capacity - num_free;
  pdl_wait();  // the moves have read the lengths
  for (int b = b0; b < b1; ++b) {
    if (per > 1) s = check(b);
    const int n = gone(s), last = pages(s.len) - 1;
    if (fits)
      for (int i = 0; i < n; ++i) p.free_pages[num_free + at + i] = __ldg(p.page_table + static_cast<long long>(b) * p.max_pages + last - i);
    at += n;
    p.seq_lens_out[b] = s.kept < 0 ? s.len : s.base + s.kept;
  }
  if (tid == 0) {
    if (!fits) report(p.status, kDevBadLength);
    p.num_free_out[0] = fits ? num_free + static_cast<int>(all) : num_free;
  }
}

}  // namespace

cudaError_t launch_keep(const KeepParams& p, int sms, cudaStream_t stream) {
  // CTAs per sequence: enough for eight per SM (its loads and stores are one round trip each), at most one per eight tasks
  const int tasks = (2 * p.layers * p.hkv + kMoveThreads / 32 - 1) / (kMoveThreads / 32);
  const int want = (8 * sms + p.batch - 1) / p.batch;
  const int y = want < tasks ? want : tasks;
  cudaError_t e = launch_pdl(vq_keep_move_kernel, dim3(p.batch, y), dim3(kMoveThreads), 0, stream, p, false);
  if (e != cudaSuccess) return e;
  return launch_pdl(vq_keep_book_kernel, dim3(1), dim3(kBookThreads), 0, stream, p, true);
}

}  // namespace vqk

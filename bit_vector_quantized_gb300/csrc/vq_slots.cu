// vq_slots.cu -- page tables, slot map, positions and row offsets from request lengths (sm_103a).
//
// Sequence b has len_b cached tokens and brings n_b new ones.  With pages of
// P tokens it has ceil(len_b / P) pages and needs ceil((len_b + n_b) / P);
// the difference comes off the top of the free stack, sequences in order:
// with A_b the pages taken by the sequences before b,
//   page_table[b][have_b + j] = free_pages[num_free - 1 - (A_b + j)],
// token i of the step's cu_b .. cu_{b+1} (cu: exclusive sums of n) stands at
// position len_b + i and in slot page_table[b][pos / P] P + pos % P.
//
// One cluster of up to 8 CTAs does it in one launch.  Every CTA reads all
// lengths and forms both prefix sums in shared memory (a few KB; instead of a
// second launch, which was not tried), checks everything the step takes, and only after the
// cluster's barrier writes its share, so seq_lens and num_free may be updated
// in place and a step that cannot be served changes nothing.  A thread
// finds its tokens' sequence by binary search in shared memory, four tokens
// at a time (48 bytes of slots and positions).  Bound by latency: three
// dependent global loads and two barriers.  Measured from a cold L2: 10 us for
// 256 decode tokens, 19 us for 120 000 tokens of 48 sequences (8 CTAs).
#include "vq_device.cuh"
#include "vq_kernels.h"

namespace vqk {
namespace {

constexpr int kSlotThreads = 512;

__device__ __forceinline__ int pages_of(int tokens, int page_size) {
  return static_cast<int>((static_cast<unsigned>(tokens) + page_size - 1u) / page_size);
}

// Last index i in [0, n) with x[i] <= v (x ascending, x[0] <= v).
__device__ __forceinline__ int last_at_most(const int* x, int n, int v) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (x[mid] <= v) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kSlotThreads) vq_slots_kernel(const SlotsParams p) {
  extern __shared__ int sm[];
  const int B = p.batch, P = p.page_size, tid = threadIdx.x;
  int* const cu = sm;              // [B + 1] new tokens before b
  int* const first = cu + B + 1;   // [B + 1] pages taken before b
  int* const len = first + B + 1;  // [B]
  __shared__ long long warp_new[kSlotThreads / 32], warp_take[kSlotThreads / 32];
  __shared__ int bad;
  if (tid == 0) bad = kDevOk;
  __syncthreads();
  // Of several faults the same one is reported in every run: lengths, then too few pages, then pages.
  static_assert(kDevOk < kDevBadPage && kDevBadPage < kDevBadLength && kDevBadLength < kDevNoPages, "the larger wins");
  auto fail = [&](int code) { atomicMax(&bad, code); };

  // ---- lengths and their checks, this thread's run of sequences ----------------
  const int num_free = __ldg(p.num_free);
  if (tid == 0 && (num_free < 0 || num_free > p.free_capacity)) fail(kDevBadLength);
  const int per = (B + kSlotThreads - 1) / kSlotThreads;
  const int b0 = min(tid * per, B), b1 = min(b0 + per, B);
  long long sum_new = 0, sum_take = 0;
  for (int b = b0; b < b1; ++b) {
    int l = p.seq_lens[b], n = p.new_lens[b];
    const long long end = static_cast<long long>(l) + n;
    if (l < 0 || n < 0 || end > 0x7fffffffLL || end > static_cast<long long>(p.max_pages) * P) {
      fail(kDevBadLength);
      l = n = 0;
    }
    const int have = pages_of(l, P), need = pages_of(l + n, P);
    if (n > 0 && l % P) {  // the first new token joins a page that is there already
      const int pg = p.page_table[static_cast<long long>(b) * p.max_pages + l / P];
      if (pg < 0 || pg >= p.num_pages) fail(kDevBadPage);
    }
    len[b] = l;
    cu[b] = n;
    first[b] = need - have;
    sum_new += n;
    sum_take += need - have;
  }
  // ---- exclusive sums over the CTA ---------------------------------------------
  const int lane = tid & 31, warp = tid >> 5;
  long long in = sum_new, it = sum_take;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, in, o), y = __shfl_up_sync(0xffffffffu, it, o);
    if (lane >= o) {
      in += x;
      it += y;
    }
  }
  if (lane == 31) {
    warp_new[warp] = in;
    warp_take[warp] = it;
  }
  __syncthreads();
  long long base_new = in - sum_new, base_take = it - sum_take, all_new = 0, all_take = 0;
  for (int w = 0; w < kSlotThreads / 32; ++w) {
    if (w < warp) {
      base_new += warp_new[w];
      base_take += warp_take[w];
    }
    all_new += warp_new[w];
    all_take += warp_take[w];
  }
  if (tid == 0) {
    if (all_new > p.max_tokens) fail(kDevBadLength);
    else if (bad != kDevBadLength && all_take > num_free) fail(kDevNoPages);
  }
  for (int b = b0; b < b1; ++b) {  // (sums past int32 are never used: the step is refused)
    const int n = cu[b], k = first[b];
    cu[b] = static_cast<int>(base_new);
    first[b] = static_cast<int>(base_take);
    base_new += n;
    base_take += k;
  }
  if (tid == 0) {
    cu[B] = static_cast<int>(all_new);
    first[B] = static_cast<int>(all_take);
  }
  __syncthreads();
  const int takes = bad == kDevOk ? first[B] : 0;
  for (int i = tid; i < takes; i += kSlotThreads) {  // every page that is taken is a page
    const int pg = __ldg(p.free_pages + (num_free - 1 - i));
    if (pg < 0 || pg >= p.num_pages) fail(kDevBadPage);
  }
  __syncthreads();
  const bool ok = bad == kDevOk;
  cluster_sync();  // every CTA has read what the step may overwrite

  // ---- this CTA's share of the outputs ------------------------------------------
  const int nthreads = gridDim.x * kSlotThreads, gtid = blockIdx.x * kSlotThreads + tid;
  if (!ok && gtid == 0) report(p.status, bad);
  for (int b = gtid; b <= B; b += nthreads) p.cu_new_lens[b] = ok ? cu[b] : 0;
  if (gtid == 0) p.num_free_out[0] = ok ? num_free - first[B] : num_free;
  if (ok) {
    for (int b = gtid; b < B; b += nthreads) p.seq_lens_out[b] = len[b] + (cu[b + 1] - cu[b]);
    for (int i = gtid; i < takes; i += nthreads) {
      const int b = last_at_most(first, B + 1, i);  // the last such b takes pages: first[b + 1] > i
      const int have = pages_of(len[b], P);
      p.page_table[static_cast<long long>(b) * p.max_pages + have + (i - first[b])] =
          __ldg(p.free_pages + (num_free - 1 - i));
    }
  } else if (p.seq_lens_out != p.seq_lens) {
    for (int b = gtid; b < B; b += nthreads) p.seq_lens_out[b] = p.seq_lens[b];
  }
  const int total = ok ? cu[B] : 0;
  for (int q = gtid; q < (p.max_tokens + 3) / 4; q += nthreads) {
    long long slot[4];
    int pos[4];
    int b = 0, end = -1, have = 0, page_of = -1;
    long long page = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = 4 * q + e;
      slot[e] = -1;
      pos[e] = -1;
      if (i >= total) continue;
      if (i >= end) {
        b = last_at_most(cu, B + 1, i);
        end = cu[b + 1];
        have = pages_of(len[b], P);
        page_of = -1;
      }
      const int at = len[b] + (i - cu[b]);
      const int lp = at / P;
      if (lp != page_of) {
        page_of = lp;
        page = lp < have ? p.page_table[static_cast<long long>(b) * p.max_pages + lp]
                         : __ldg(p.free_pages + (num_free - 1 - (first[b] + lp - have)));
      }
      pos[e] = at;
      slot[e] = page * P + (at - lp * P);
    }
    if (4 * q + 3 < p.max_tokens) {
      longlong2* s = reinterpret_cast<longlong2*>(p.slot_mapping + 4 * q);
      s[0] = make_longlong2(slot[0], slot[1]);
      s[1] = make_longlong2(slot[2], slot[3]);
      *reinterpret_cast<int4*>(p.positions + 4 * q) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (4 * q + e < p.max_tokens) {
          p.slot_mapping[4 * q + e] = slot[e];
          p.positions[4 * q + e] = pos[e];
        }
    }
  }
}

SmemOptIn g_slots_smem;

}  // namespace

cudaError_t launch_slots(const SlotsParams& p, cudaStream_t stream) {
  const size_t smem = (3 * static_cast<size_t>(p.batch) + 2) * sizeof(int);
  cudaError_t e = cudaSuccess;
  if (smem > 40 * 1024) e = ensure_smem(vq_slots_kernel, smem, g_slots_smem);
  if (e != cudaSuccess) return e;
  // one CTA per 2048 tokens (a thread's four), at most a portable cluster
  const int ctas = static_cast<int>((static_cast<long long>(p.max_tokens) + 4 * kSlotThreads - 1) / (4 * kSlotThreads));
  const int c = ctas < 1 ? 1 : ctas > 4 ? 8 : ctas > 2 ? 4 : ctas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(c);
  cfg.blockDim = dim3(kSlotThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = c;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, vq_slots_kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace vqk

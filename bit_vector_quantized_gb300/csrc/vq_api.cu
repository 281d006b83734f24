// vq_api.cu -- the extern "C" boundary (include/vqattn.h): argument checks,
// launch-shape choice and kernel launches.  No allocation, no synchronisation.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <string>

#include "../../include/vqattn.h"
#include "vq_kernels.h"

namespace {

thread_local std::string g_last_error;

vq_status fail(vq_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return st;
}

vq_status cuda_fail(cudaError_t e, const char* what) {
  return fail(VQ_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool is_pow2(int x) { return x > 0 && (x & (x - 1)) == 0; }

// Device attributes the launch choices need, read once per device.
struct DeviceAttrs {
  std::atomic<int> sms[vqk::kMaxDevices] = {};
  std::atomic<int> smem_optin[vqk::kMaxDevices] = {};
};
DeviceAttrs g_attrs;

int device_attr(std::atomic<int>* cache, cudaDeviceAttr attr) {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= vqk::kMaxDevices) return 0;
  n = cache[dev].load(std::memory_order_relaxed);
  if (n > 0) return n;
  if (cudaDeviceGetAttribute(&n, attr, dev) != cudaSuccess) return 0;
  cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

int device_sms() { return device_attr(g_attrs.sms, cudaDevAttrMultiProcessorCount); }

int device_smem_optin() {
  return device_attr(g_attrs.smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin);
}

bool decode_formats_supported(const vq_layout& L) {
  const bool k_ok = (L.k_sub == 2 || L.k_sub == 4) && L.k_bits == 8;
  const bool v_ok = (L.v_sub == 4 && (L.v_bits == 8 || L.v_bits == 9)) ||
                    (L.v_sub == 2 && L.v_bits == 8);
  const bool wide = L.k_sub == 8 && L.k_bits == 12 && L.v_sub == 8 && L.v_bits == 12;
  return (k_ok && v_ok) || wide;
}

constexpr int kMaxSplits = 4096;
constexpr int kMaxResidual = 4096;  // residual window capacity (tokens)

// Largest value the length-balanced kernel's slot term of W,
// ceil(longest pair's blocks / (splits - 1)), can take: the pairs' blocks
// are at most ceil(max_seq_len / 32).
int balance_wmin(int max_seq_len, int splits) {
  const int nsl = (max_seq_len + vqk::kUnitTok - 1) / vqk::kUnitTok;
  return (nsl + splits - 2) / (splits - 1);
}

// Length-balanced units (decode kernel, DecodeParams::balanced) for batches
// of two or more sequences: the grid (one CTA per SM) splits the pairs' blocks
// evenly whatever the lengths.  Needs two or more partial slots per pair and
// at most kMaxUnitsPerCta units per CTA, which holds with at most that many
// pairs or with a per-CTA range W <= (kMaxUnitsPerCta - 2) (1 + kBalanceGap)
// (pairs after a CTA's first start inside its range, 1 + kBalanceGap
// positions apart at least); the kernel's W is at most the bound taken here
// from max_seq_len.
bool balanced_units(const vq_layout& L, int batch, int max_seq_len, int splits, int sms) {
  if (batch < 2 || batch > vqk::kBalanceMaxBatch || splits < 2 || sms <= 0 || max_seq_len < 1) return false;
  const long long pairs = static_cast<long long>(batch) * L.num_kv_heads;
  const long long nsl = (static_cast<long long>(max_seq_len) + vqk::kUnitTok - 1) / vqk::kUnitTok;
  const long long total = pairs * (nsl + vqk::kBalanceGap);  // the largest total the kernel can see
  if (total >= (1LL << 30)) return false;
  const long long w = std::max<long long>((total + sms - 1) / sms, balance_wmin(max_seq_len, splits));
  return pairs <= vqk::kMaxUnitsPerCta ||
         w <= static_cast<long long>(vqk::kMaxUnitsPerCta - 2) * (1 + vqk::kBalanceGap);
}

// Split count.  Batches of two or more sequences: length-balanced units with
// 1 + ceil(2 SMs / pairs) slots per pair (a pair may be twice the average
// length before the slot term, rather than the total, sets the CTA range).
// Otherwise the count minimising an estimate of the persistent grid's
// makespan: waves(units) * (tokens per unit + fixed per-unit cost).
int pick_splits(const vq_layout& L, int batch, int max_seq_len, int sms) {
  const long long pairs = static_cast<long long>(batch) * L.num_kv_heads;
  const long long chunks = (static_cast<long long>(max_seq_len) + 15) / 16;
  if (pairs <= 0 || chunks <= 0 || sms <= 0) return 1;
  if (batch >= 2) {
    const int sb = static_cast<int>(std::min<long long>(1 + (2LL * sms + pairs - 1) / pairs, kMaxSplits));
    if (balanced_units(L, batch, max_seq_len, sb, sms)) return sb;
  }
  const double kUnitOverhead = 384.0;  // tokens-equivalent per unit (q~, merge, pipeline fill)
  int best = 1;
  double best_cost = 1e300;
  const long long smax = std::min<long long>(kMaxSplits, chunks);
  for (long long s = 1; s <= smax; ++s) {
    const long long units = pairs * s;
    if ((units + sms - 1) / sms > vqk::kMaxUnitsPerCta) break;
    const double waves = static_cast<double>((units + sms - 1) / sms);
    const double per_unit = std::ceil(static_cast<double>(chunks) / s) * 16.0 + kUnitOverhead;
    const double cost = waves * per_unit + 8.0 * s;  // combine reads grow with s
    if (cost < best_cost * 0.999) {
      best_cost = cost;
      best = static_cast<int>(s);
    }
  }
  return best;
}

// Codebooks of 1024 centroids or more: the decode step's append is spread
// over kAppendSlices CTAs per vector.
bool sliced_append(const vq_layout& L) { return L.k_bits >= 10 || L.v_bits >= 10; }

struct WsLayout {
  size_t o_off, ml_off, cnt_off, cand_off, total;
};

// Split partials, the units per (sequence, KV head) of length-balanced
// units, then (large codebooks) the sliced append's candidates.
WsLayout ws_layout(const vq_layout& L, int batch, int splits) {
  WsLayout w;
  const size_t rows = static_cast<size_t>(batch) * L.num_q_heads * splits;
  w.o_off = 0;
  w.ml_off = (rows * L.head_dim * sizeof(float) + 255) & ~size_t(255);
  w.cnt_off = w.ml_off + ((rows * 2 * sizeof(float) + 255) & ~size_t(255));
  w.cand_off = w.cnt_off + ((static_cast<size_t>(batch) * L.num_kv_heads * sizeof(int) + 255) & ~size_t(255));
  const size_t cand = sliced_append(L) ? static_cast<size_t>(batch) * L.num_kv_heads * 2 *
                                             vqk::kAppendSlices * 32 * 4 * sizeof(int2)
                                       : 0;
  w.total = w.cand_off + cand;
  return w;
}

vq_status check_layout_impl(const vq_layout* L, int for_decode) {
  if (!L) return fail(VQ_ERR_INVALID_ARG, "layout is NULL");
  if (!is_pow2(L->head_dim)) return fail(VQ_ERR_INVALID_ARG, "head_dim %d is not a power of two", L->head_dim);
  if (L->head_dim != 128)
    return fail(VQ_ERR_UNSUPPORTED, "head_dim %d: this build implements head_dim 128", L->head_dim);
  if (L->num_q_heads < 1 || L->num_kv_heads < 1 || L->num_q_heads % L->num_kv_heads)
    return fail(VQ_ERR_INVALID_ARG, "num_q_heads %d must be a positive multiple of num_kv_heads %d",
                L->num_q_heads, L->num_kv_heads);
  if (L->num_q_heads / L->num_kv_heads > 8)
    return fail(VQ_ERR_UNSUPPORTED, "query group %d > 8", L->num_q_heads / L->num_kv_heads);
  const int subs[2] = {L->k_sub, L->v_sub}, bits[2] = {L->k_bits, L->v_bits};
  for (int i = 0; i < 2; ++i) {
    if (!(subs[i] == 1 || subs[i] == 2 || subs[i] == 4 || subs[i] == 8))
      return fail(VQ_ERR_INVALID_ARG, "%s_sub %d not in {1, 2, 4, 8}", i ? "v" : "k", subs[i]);
    if (bits[i] < 1 || bits[i] > 12)
      return fail(VQ_ERR_INVALID_ARG, "%s_bits %d not in 1..12", i ? "v" : "k", bits[i]);
  }
  if (L->page_size < 16 || L->page_size % 16)
    return fail(VQ_ERR_INVALID_ARG, "page_size %d must be a positive multiple of 16", L->page_size);
  if (for_decode && !decode_formats_supported(*L))
    return fail(VQ_ERR_UNSUPPORTED,
                "decode attention implements (k_sub,k_bits) in {(2,8),(4,8)} with (v_sub,v_bits) "
                "in {(2,8),(4,8),(4,9)}, and (8,12) with (8,12); got (%d,%d) and (%d,%d)",
                L->k_sub, L->k_bits, L->v_sub, L->v_bits);
  return VQ_OK;
}

}  // namespace

extern "C" {

size_t vq_code_row_bytes(int32_t head_dim, int32_t sub, int32_t bits) {
  if (head_dim <= 0 || sub <= 0 || head_dim % sub || bits < 1 || bits > 16) return 0;
  const size_t n = static_cast<size_t>(head_dim / sub) * bits;
  return ((n + 7) / 8 + 3) / 4 * 4;
}

vq_status vq_check_layout(const vq_layout* layout, int32_t for_decode) {
  return check_layout_impl(layout, for_decode);
}

// Launches the encode of num_tokens tokens: the caller has set the sources,
// codebooks, pools, lambda, the slot source and the status word; the launch
// shape follows from the number of vectors.
vq_status launch_encode_impl(const vq_layout& L, vqk::EncodeParams& p, int32_t num_tokens,
                             bool has_k, bool has_v, void* stream, const char* what,
                             bool overlap, int2* cand = nullptr, bool merge_kernel = true) {
  p.sub[0] = L.k_sub;
  p.sub[1] = L.v_sub;
  p.bits[0] = L.k_bits;
  p.bits[1] = L.v_bits;
  p.row_bytes[0] = static_cast<int>(vq_code_row_bytes(L.head_dim, L.k_sub, L.k_bits));
  p.row_bytes[1] = static_cast<int>(vq_code_row_bytes(L.head_dim, L.v_sub, L.v_bits));
  p.num_tokens = num_tokens;
  p.hkv = L.num_kv_heads;
  p.page_size = L.page_size;
  const long long vectors = static_cast<long long>(num_tokens) * L.num_kv_heads;
  const int sms = device_sms();
  // few vectors (a decode-step append): spread each codebook scan over 8 warps
  p.split = vectors * 2 < static_cast<long long>(sms > 0 ? sms : 148) * 8 ? 8 : 1;
  // many vectors with sub-vector lengths 2 / 4: several vectors per warp
  const bool multi_ok = (!has_k || L.k_sub == 2 || L.k_sub == 4) && (!has_v || L.v_sub == 2 || L.v_sub == 4);
  p.vec_per_warp = (p.split == 1 && multi_ok) ? vqk::kMultiVec : 1;
  const int per_cta = 8 * p.vec_per_warp / p.split;
  // a few vectors of a large codebook (with candidate space): several CTAs each
  p.slices = (cand && p.split > 1 && sliced_append(L)) ? vqk::kAppendSlices : 1;
  p.cand = cand;
  const long long grid_x = (vectors + per_cta - 1) / per_cta * p.slices;
  if (grid_x > 0x7fffffffLL) return fail(VQ_ERR_INVALID_ARG, "too many tokens (%d)", num_tokens);
  p.which_base = has_k ? 0 : 1;
  const int grid_y = (has_k && has_v) ? 2 : 1;
  size_t smem = 0;
  if (has_k) smem = std::max(smem, vqk::encode_smem_bytes(L.k_sub, L.k_bits));
  if (has_v) smem = std::max(smem, vqk::encode_smem_bytes(L.v_sub, L.v_bits));
  const int optin = device_smem_optin();
  if (optin > 0 && smem > static_cast<size_t>(optin))
    return fail(VQ_ERR_UNSUPPORTED, "encode needs %zu bytes of shared memory, device has %d", smem, optin);
  cudaError_t e = vqk::launch_encode(p, static_cast<int>(grid_x), grid_y, smem,
                                     static_cast<cudaStream_t>(stream), overlap);
  if (e != cudaSuccess) return cuda_fail(e, what);
  if (p.slices > 1 && merge_kernel) {
    e = vqk::launch_encode_merge(p, static_cast<int>(vectors), grid_y, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, what);
  }
  return VQ_OK;
}

vq_status vq_encode_kv(const vq_layout* layout, int32_t num_tokens, const void* k, const void* v,
                       const int64_t* slot_mapping, const float* lambda, const void* codebook_k,
                       const void* codebook_v, void* k_pool, void* v_pool, int64_t num_pages,
                       int32_t* status, void* stream) {
  vq_status st = check_layout_impl(layout, 0);
  if (st != VQ_OK) return st;
  const vq_layout& L = *layout;
  if (num_tokens < 0) return fail(VQ_ERR_INVALID_ARG, "num_tokens %d < 0", num_tokens);
  if (!k && !v) return fail(VQ_ERR_INVALID_ARG, "k and v are both NULL");
  if (!slot_mapping) return fail(VQ_ERR_INVALID_ARG, "slot_mapping is NULL");
  if (num_pages < 1) return fail(VQ_ERR_INVALID_ARG, "num_pages %lld < 1", (long long)num_pages);
  if (k && (!lambda || !codebook_k || !k_pool))
    return fail(VQ_ERR_INVALID_ARG, "k given but lambda, codebook_k or k_pool is NULL");
  if (v && (!codebook_v || !v_pool))
    return fail(VQ_ERR_INVALID_ARG, "v given but codebook_v or v_pool is NULL");
  const void* ptrs[] = {k, v, lambda, codebook_k, codebook_v, k_pool, v_pool, slot_mapping};
  for (const void* ptr : ptrs)
    if (ptr && !aligned16(ptr)) return fail(VQ_ERR_INVALID_ARG, "device buffer %p is not 16-byte aligned", ptr);
  if (num_tokens == 0) return VQ_OK;

  vqk::EncodeParams p{};
  p.src[0] = k;
  p.src[1] = v;
  p.cb[0] = codebook_k;
  p.cb[1] = codebook_v;
  p.pool[0] = static_cast<uint8_t*>(k_pool);
  p.pool[1] = static_cast<uint8_t*>(v_pool);
  p.lambda = lambda;
  p.slots = slot_mapping;
  p.status = status;
  p.num_slots = static_cast<long long>(num_pages) * L.page_size;
  return launch_encode_impl(L, p, num_tokens, k != nullptr, v != nullptr, stream,
                            "vq_encode_kv launch", false);
}

vq_status vq_dequantize_kv(const vq_layout* layout, int32_t num_tokens,
                           const int64_t* slot_mapping, const float* lambda,
                           const void* codebook_k, const void* codebook_v, const void* k_pool,
                           const void* v_pool, int64_t num_pages, void* k_out, void* v_out,
                           int32_t* status, void* stream) {
  vq_status st = check_layout_impl(layout, 0);
  if (st != VQ_OK) return st;
  const vq_layout& L = *layout;
  if (num_tokens < 0) return fail(VQ_ERR_INVALID_ARG, "num_tokens %d < 0", num_tokens);
  if (num_tokens == 0) return VQ_OK;  // empty tensors may come with NULL pointers
  if (!k_out && !v_out) return fail(VQ_ERR_INVALID_ARG, "k_out and v_out are both NULL");
  if (!slot_mapping) return fail(VQ_ERR_INVALID_ARG, "slot_mapping is NULL");
  if (num_pages < 1) return fail(VQ_ERR_INVALID_ARG, "num_pages %lld < 1", (long long)num_pages);
  if (k_out && (!lambda || !codebook_k || !k_pool))
    return fail(VQ_ERR_INVALID_ARG, "k_out given but lambda, codebook_k or k_pool is NULL");
  if (v_out && (!codebook_v || !v_pool))
    return fail(VQ_ERR_INVALID_ARG, "v_out given but codebook_v or v_pool is NULL");
  const void* ptrs[] = {k_out, v_out, lambda, codebook_k, codebook_v, k_pool, v_pool, slot_mapping};
  for (const void* ptr : ptrs)
    if (ptr && !aligned16(ptr)) return fail(VQ_ERR_INVALID_ARG, "device buffer %p is not 16-byte aligned", ptr);

  vqk::DequantParams p{};
  p.k_pool = static_cast<const uint8_t*>(k_pool);
  p.v_pool = static_cast<const uint8_t*>(v_pool);
  p.cb_k = codebook_k;
  p.cb_v = codebook_v;
  p.out_k = k_out;
  p.out_v = v_out;
  p.k_sub = L.k_sub;
  p.k_bits = L.k_bits;
  p.k_row = static_cast<int>(vq_code_row_bytes(L.head_dim, L.k_sub, L.k_bits));
  p.v_sub = L.v_sub;
  p.v_bits = L.v_bits;
  p.v_row = static_cast<int>(vq_code_row_bytes(L.head_dim, L.v_sub, L.v_bits));
  p.lambda = lambda;
  p.slots = slot_mapping;
  p.status = status;
  p.num_slots = static_cast<long long>(num_pages) * L.page_size;
  p.num_tokens = num_tokens;
  p.hkv = L.num_kv_heads;
  p.page_size = L.page_size;
  p.which_base = k_out ? 0 : 1;
  p.which_last = v_out ? 1 : 0;
  const int per_cta = vqk::dequant_tokens_per_cta();
  const int grid_x = (num_tokens + per_cta - 1) / per_cta;
  cudaError_t e = vqk::launch_dequant(p, grid_x, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "vq_dequantize_kv launch");
  return VQ_OK;
}

int32_t vq_default_num_splits(const vq_layout* layout, int32_t batch, int32_t max_seq_len,
                              int32_t num_sms) {
  if (!layout || batch < 0 || max_seq_len < 0 || layout->num_kv_heads < 1) return 0;
  const int sms = num_sms > 0 ? num_sms : device_sms();
  if (sms <= 0) return 0;
  return pick_splits(*layout, batch, max_seq_len, sms);
}

int32_t vq_decode_units_balanced(const vq_layout* layout, int32_t batch, int32_t max_seq_len,
                                 int32_t num_splits, int32_t num_sms) {
  if (!layout || batch < 0 || max_seq_len < 0 || layout->num_kv_heads < 1) return -1;
  if (num_splits > kMaxSplits) return -1;
  const int sms = num_sms > 0 ? num_sms : device_sms();
  if (sms <= 0) return -1;
  const int splits = num_splits > 0 ? num_splits : pick_splits(*layout, batch, max_seq_len, sms);
  return balanced_units(*layout, batch, max_seq_len, splits, sms) ? 1 : 0;
}

size_t vq_decode_workspace_bytes(const vq_layout* layout, int32_t batch, int32_t max_seq_len,
                                 int32_t num_splits, int32_t num_sms) {
  if (!layout || batch < 0 || max_seq_len < 0 || layout->num_q_heads < 1) return 0;
  int splits = num_splits;
  if (splits <= 0) splits = vq_default_num_splits(layout, batch, max_seq_len, num_sms);
  if (splits <= 0 || splits > kMaxSplits) return 0;
  return ws_layout(*layout, batch, splits).total;
}

}  // extern "C"

namespace {

// Validates the decode arguments and fills the split kernel's parameters.
vq_status prepare_decode(const vq_layout* layout, int32_t batch, const void* q, const float* lambda,
                         const void* codebook_k, const void* codebook_v, const void* k_pool,
                         const void* v_pool, int64_t num_pages, const int32_t* page_table,
                         int32_t max_pages_per_seq, const int32_t* seq_lens, int32_t max_seq_len,
                         float softmax_scale, int32_t num_splits, const void* workspace,
                         size_t workspace_bytes, int32_t* status, vqk::DecodeParams& p,
                         int& grid, size_t& smem, bool* append = nullptr,
                         int method = vqk::kMethodGather, int res_capacity = 0) {
  const vq_layout& L = *layout;
  const void* ptrs[] = {q, lambda, codebook_k, codebook_v, k_pool, v_pool, page_table, seq_lens, workspace};
  const char* names[] = {"q", "lambda", "codebook_k", "codebook_v", "k_pool", "v_pool",
                         "page_table", "seq_lens", "workspace"};
  for (int i = 0; i < 9; ++i) {
    if (!ptrs[i]) return fail(VQ_ERR_INVALID_ARG, "%s is NULL", names[i]);
    if (!aligned16(ptrs[i])) return fail(VQ_ERR_INVALID_ARG, "%s is not 16-byte aligned", names[i]);
  }
  if (num_pages < 1) return fail(VQ_ERR_INVALID_ARG, "num_pages %lld < 1", (long long)num_pages);
  if (max_pages_per_seq < 1) return fail(VQ_ERR_INVALID_ARG, "max_pages_per_seq %d < 1", max_pages_per_seq);
  if (max_seq_len < 0) return fail(VQ_ERR_INVALID_ARG, "max_seq_len %d < 0", max_seq_len);
  if (static_cast<long long>(max_seq_len) > static_cast<long long>(max_pages_per_seq) * L.page_size)
    return fail(VQ_ERR_INVALID_ARG, "max_seq_len %d exceeds max_pages_per_seq * page_size", max_seq_len);
  if (!std::isfinite(softmax_scale)) return fail(VQ_ERR_INVALID_ARG, "softmax_scale is not finite");
  if (num_splits > kMaxSplits) return fail(VQ_ERR_INVALID_ARG, "num_splits %d > %d", num_splits, kMaxSplits);

  const int sms = device_sms();
  if (sms <= 0) return fail(VQ_ERR_CUDA, "no CUDA device");
  const int splits = num_splits > 0 ? num_splits : pick_splits(L, batch, max_seq_len, sms);
  const WsLayout ws = ws_layout(L, batch, splits);
  if (workspace_bytes < ws.total)
    return fail(VQ_ERR_WORKSPACE, "workspace %zu bytes < %zu required", workspace_bytes, ws.total);
  const long long units = static_cast<long long>(batch) * L.num_kv_heads * splits;
  if (units > 0x7fffffffLL) return fail(VQ_ERR_INVALID_ARG, "too many work units");
  const bool balanced = balanced_units(L, batch, max_seq_len, splits, sms);
  long long g = std::min<long long>(units, sms);
  g = std::max<long long>(g, (units + vqk::kMaxUnitsPerCta - 1) / vqk::kMaxUnitsPerCta);
  grid = static_cast<int>(balanced ? sms : g);

  p = vqk::DecodeParams{};
  p.q = q;
  p.lambda = lambda;
  p.cb_k = codebook_k;
  p.cb_v = codebook_v;
  p.k_pool = static_cast<const uint8_t*>(k_pool);
  p.v_pool = static_cast<const uint8_t*>(v_pool);
  p.page_table = page_table;
  p.seq_lens = seq_lens;
  uint8_t* wsb = static_cast<uint8_t*>(const_cast<void*>(workspace));
  p.ws_o = reinterpret_cast<float*>(wsb + ws.o_off);
  p.ws_ml = reinterpret_cast<float2*>(wsb + ws.ml_off);
  p.status = status;
  p.num_pages = num_pages;
  p.timeout_ns = 2000000000ULL;
  p.batch = batch;
  p.hq = L.num_q_heads;
  p.hkv = L.num_kv_heads;
  p.group = L.num_q_heads / L.num_kv_heads;
  p.page_size = L.page_size;
  p.max_pages = max_pages_per_seq;
  p.max_seq_len = max_seq_len;
  p.splits = splits;
  p.num_units = static_cast<int>(units);
  const int nsl = (max_seq_len + vqk::kUnitTok - 1) / vqk::kUnitTok;
  p.split_q = nsl / splits;
  p.split_r = nsl % splits;
  p.balanced = balanced ? 1 : 0;
  p.ws_cnt = balanced ? reinterpret_cast<int*>(wsb + ws.cnt_off) : nullptr;
  p.k_row = static_cast<int>(vq_code_row_bytes(L.head_dim, L.k_sub, L.k_bits));
  p.v_row = static_cast<int>(vq_code_row_bytes(L.head_dim, L.v_sub, L.v_bits));
  const float scale = softmax_scale == 0.f ? 1.f / std::sqrt(static_cast<float>(L.head_dim)) : softmax_scale;
  p.qscale = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634 / std::sqrt(128.0));
  // residual window: a unit's slice is at most ceil(capacity / splits)
  // tokens (length-balanced units: the whole window), staged in shared
  // memory up to kMaxResTok at a time
  const int res_slice = balanced ? res_capacity : (res_capacity + splits - 1) / splits;
  const int res_tok = res_capacity > 0 ? std::min(res_slice, vqk::kMaxResTok) : 0;
  p.res_tok = res_tok;

  const int optin = device_smem_optin();
  // Pipeline stages: the most (up to kMaxStages) that fit, and never fewer
  // than the producer warps.  A producer waits for its slot to be released by
  // the parity of the slot's "empty" barrier, which tells adjacent phases
  // apart only; with at least as many stages as producer warps, the
  // producer's own previous stage guarantees the barrier is at most one phase
  // behind.
  bool with_append = false;
  auto stages_for = [&](const vqk::DecodeShape& sh, size_t& bytes) {
    int ns = vqk::kMaxStages;
    for (; ns >= vqk::kProducerWarps; --ns) {
      bytes = vqk::decode_smem(L.k_bits, L.v_bits, p.group, p.k_row, p.v_row, ns, sh.warps,
                               sh.stage_tok(),
                               with_append && !sliced_append(L)
                                   ? vqk::append_enc_bytes(L.k_bits, L.v_bits, L.k_sub, L.v_sub) : 0,
                               method, res_tok)
                  .total;
      if (optin <= 0 || bytes <= static_cast<size_t>(optin)) return ns;
    }
    return 0;
  };
  // Consumer shape: 12 warps for G <= 4, 8 warps for G > 4 (register
  // budget), and 8 wherever 12 leaves room for fewer than kProducerWarps
  // stages; VQ_DECODE_SHAPE=8x1|12x1 selects a shape explicitly (a tuning
  // switch for profiling; an explicit shape that does not fit is an error).
  // (the 1.5-bit format: 8, its whole-centroid gathers need the registers)
  vqk::DecodeShape shape = (p.group > 4 || L.k_bits == 12) ? vqk::DecodeShape{8} : vqk::DecodeShape{12};
  bool explicit_shape = false;
  if (const char* env = std::getenv("VQ_DECODE_SHAPE")) {
    if (std::strcmp(env, "8x1") == 0) shape = vqk::DecodeShape{8}, explicit_shape = true;
    if (std::strcmp(env, "12x1") == 0) shape = vqk::DecodeShape{12}, explicit_shape = true;
  }
  if (method != vqk::kMethodGather) {
    if (!(L.k_sub == 4 && L.k_bits == 8 && L.v_sub == 4 && L.v_bits == 8 && p.group <= 4))
      return fail(VQ_ERR_UNSUPPORTED,
                  "the LUT and bins methods are built for k_sub = v_sub = 4, 8-bit codes and "
                  "num_q_heads / num_kv_heads <= 4");
    shape = vqk::DecodeShape{12};
    explicit_shape = true;
  }
  int nstage = stages_for(shape, smem);
  if (nstage == 0 && !explicit_shape && shape.warps != 8) {
    shape = vqk::DecodeShape{8};
    nstage = stages_for(shape, smem);
  }
  if (nstage == 0)
    return fail(VQ_ERR_UNSUPPORTED,
                "decode pipeline does not fit: %d consumer warps need %zu bytes of shared memory "
                "for %d stages",
                shape.warps, smem, vqk::kProducerWarps);
  // The decode-step append inside the attention kernel needs a little more
  // shared memory; it runs only with the same consumer shape (so the results
  // equal the separate append and attention bit for bit) and enough stages.
  if (append && *append) {
    with_append = true;
    size_t bytes_app = 0;
    const int ns_app = stages_for(shape, bytes_app);
    if (ns_app >= vqk::kProducerWarps) {
      nstage = ns_app;
      smem = bytes_app;
    } else {
      *append = false;
    }
  }
  p.warps = shape.warps;
  p.nstage = nstage;
  return VQ_OK;
}

// CTAs of the decode step's append encode: one warp per (sequence, KV head)
// vector, 8 per CTA, keys and values.
vq_status launch_partial(const vq_layout& L, const vqk::DecodeParams& p, int grid, size_t smem,
                         void* stream, bool overlap, int method = vqk::kMethodGather) {
  cudaError_t e = vqk::launch_decode(p, L.k_sub, L.k_bits, L.v_sub, L.v_bits, grid, smem,
                                     static_cast<cudaStream_t>(stream), overlap, method);
  if (e != cudaSuccess) return cuda_fail(e, "decode split kernel");
  return VQ_OK;
}

vq_status combine_impl(const vq_layout* layout, int32_t batch, int32_t max_seq_len,
                       int32_t num_splits, const void* workspace, size_t workspace_bytes,
                       void* out, void* stream, bool overlap) {
  const vq_layout& L = *layout;
  if (!workspace || !out) return fail(VQ_ERR_INVALID_ARG, "workspace or out is NULL");
  if (!aligned16(workspace) || !aligned16(out))
    return fail(VQ_ERR_INVALID_ARG, "workspace or out is not 16-byte aligned");
  if (num_splits > kMaxSplits) return fail(VQ_ERR_INVALID_ARG, "num_splits %d > %d", num_splits, kMaxSplits);
  int splits = num_splits;
  int sms = 0;
  if (splits <= 0 || batch >= 2) {  // the split choice, or whether the units were length-balanced
    sms = device_sms();
    if (sms <= 0) return fail(VQ_ERR_CUDA, "no CUDA device");
  }
  if (splits <= 0) splits = pick_splits(L, batch, max_seq_len, sms);
  const WsLayout ws = ws_layout(L, batch, splits);
  if (workspace_bytes < ws.total)
    return fail(VQ_ERR_WORKSPACE, "workspace %zu bytes < %zu required", workspace_bytes, ws.total);
  vqk::CombineParams cp{};
  const uint8_t* wsb = static_cast<const uint8_t*>(workspace);
  cp.ws_o = reinterpret_cast<const float*>(wsb + ws.o_off);
  cp.ws_ml = reinterpret_cast<const float2*>(wsb + ws.ml_off);
  cp.out = out;
  cp.rows = batch * L.num_q_heads;
  cp.splits = splits;
  cp.cnt = balanced_units(L, batch, max_seq_len, splits, sms) ? reinterpret_cast<const int*>(wsb + ws.cnt_off)
                                                               : nullptr;
  cp.group = L.num_q_heads / L.num_kv_heads;
  cudaError_t e = vqk::launch_combine(cp, static_cast<cudaStream_t>(stream), overlap);
  if (e != cudaSuccess) return cuda_fail(e, "decode combine kernel");
  return VQ_OK;
}

}  // namespace

extern "C" {

vq_status vq_decode_partial(const vq_layout* layout, int32_t batch, const void* q,
                            const float* lambda, const void* codebook_k, const void* codebook_v,
                            const void* k_pool, const void* v_pool, int64_t num_pages,
                            const int32_t* page_table, int32_t max_pages_per_seq,
                            const int32_t* seq_lens, int32_t max_seq_len, float softmax_scale,
                            int32_t num_splits, void* workspace, size_t workspace_bytes,
                            int32_t* status, void* stream) {
  vq_status st = check_layout_impl(layout, 1);
  if (st != VQ_OK) return st;
  if (batch < 0) return fail(VQ_ERR_INVALID_ARG, "batch %d < 0", batch);
  if (batch == 0) return VQ_OK;
  vqk::DecodeParams p;
  int grid = 0;
  size_t smem = 0;
  st = prepare_decode(layout, batch, q, lambda, codebook_k, codebook_v, k_pool, v_pool, num_pages,
                      page_table, max_pages_per_seq, seq_lens, max_seq_len, softmax_scale,
                      num_splits, workspace, workspace_bytes, status, p, grid, smem);
  if (st != VQ_OK) return st;
  return launch_partial(*layout, p, grid, smem, stream, false);
}

vq_status vq_decode_partial_method(const vq_layout* layout, int32_t batch, const void* q,
                                   const float* lambda, const void* codebook_k,
                                   const void* codebook_v, const void* k_pool, const void* v_pool,
                                   int64_t num_pages, const int32_t* page_table,
                                   int32_t max_pages_per_seq, const int32_t* seq_lens,
                                   int32_t max_seq_len, float softmax_scale, int32_t num_splits,
                                   int32_t method, void* workspace, size_t workspace_bytes,
                                   int32_t* status, void* stream) {
  vq_status st = check_layout_impl(layout, 1);
  if (st != VQ_OK) return st;
  if (method < VQ_METHOD_GATHER || method > VQ_METHOD_BINS)
    return fail(VQ_ERR_INVALID_ARG, "method %d is not a vq_decode_method", method);
  if (batch < 0) return fail(VQ_ERR_INVALID_ARG, "batch %d < 0", batch);
  if (batch == 0) return VQ_OK;
  vqk::DecodeParams p;
  int grid = 0;
  size_t smem = 0;
  st = prepare_decode(layout, batch, q, lambda, codebook_k, codebook_v, k_pool, v_pool, num_pages,
                      page_table, max_pages_per_seq, seq_lens, max_seq_len, softmax_scale,
                      num_splits, workspace, workspace_bytes, status, p, grid, smem, nullptr, method);
  if (st != VQ_OK) return st;
  return launch_partial(*layout, p, grid, smem, stream, false, method);
}

vq_status vq_decode_combine(const vq_layout* layout, int32_t batch, int32_t max_seq_len,
                            int32_t num_splits, const void* workspace, size_t workspace_bytes,
                            void* out, void* stream) {
  vq_status st = check_layout_impl(layout, 1);
  if (st != VQ_OK) return st;
  if (batch < 0 || max_seq_len < 0) return fail(VQ_ERR_INVALID_ARG, "batch or max_seq_len < 0");
  if (batch == 0) return VQ_OK;
  return combine_impl(layout, batch, max_seq_len, num_splits, workspace, workspace_bytes, out, stream,
                      false);
}

vq_status vq_decode_step(const vq_layout* layout, int32_t batch, const void* q, const void* k_new,
                         const void* v_new, const float* lambda, const void* codebook_k,
                         const void* codebook_v, void* k_pool, void* v_pool, int64_t num_pages,
                         const int32_t* page_table, int32_t max_pages_per_seq,
                         const int32_t* seq_lens, int32_t max_seq_len, float softmax_scale,
                         int32_t num_splits, void* out, void* workspace, size_t workspace_bytes,
                         int32_t* status, void* stream) {
  vq_status st = check_layout_impl(layout, 1);
  if (st != VQ_OK) return st;
  const vq_layout& L = *layout;
  if (batch < 0) return fail(VQ_ERR_INVALID_ARG, "batch %d < 0", batch);
  if (batch == 0) return VQ_OK;
  const void* ptrs[] = {k_new, v_new, out};
  const char* names[] = {"k_new", "v_new", "out"};
  for (int i = 0; i < 3; ++i) {
    if (!ptrs[i]) return fail(VQ_ERR_INVALID_ARG, "%s is NULL", names[i]);
    if (!aligned16(ptrs[i])) return fail(VQ_ERR_INVALID_ARG, "%s is not 16-byte aligned", names[i]);
  }
  vqk::DecodeParams p;
  int grid = 0;
  size_t smem = 0;
  // With at most one (sequence, KV head) pair per SM the new tokens are
  // appended inside the attention kernel: the producer warps of the CTA whose
  // split holds a new token encode it while their first copies are in flight
  // (codes of at most 9 bits), or merge the candidates that the encode
  // kernel's sliced scan left in the workspace (the 1.5-bit format, whose
  // 4096-centroid scan needs more than one CTA).  With more pairs than SMs the
  // separate append kernel spreads the appends over the GPU sooner (measured:
  // 32K, ragged batch-16 and 196K steps faster fused, batch 64 no faster).
  const int sms_now = device_sms();
  const bool wide = sliced_append(L);
  const bool wide_ok = L.k_sub == 8 && L.k_bits == 12 && L.v_sub == 8 && L.v_bits == 12;
  bool fused = ((L.k_bits <= 9 && L.v_bits <= 9) || wide_ok) &&
               static_cast<long long>(batch) * L.num_kv_heads <= (sms_now > 0 ? sms_now : 0);
  st = prepare_decode(layout, batch, q, lambda, codebook_k, codebook_v, k_pool, v_pool, num_pages,
                      page_table, max_pages_per_seq, seq_lens, max_seq_len, softmax_scale,
                      num_splits, workspace, workspace_bytes, status, p, grid, smem, &fused);
  if (st != VQ_OK) return st;

  vqk::EncodeParams ep{};
  ep.src[0] = k_new;
  ep.src[1] = v_new;
  ep.cb[0] = codebook_k;
  ep.cb[1] = codebook_v;
  ep.pool[0] = static_cast<uint8_t*>(k_pool);
  ep.pool[1] = static_cast<uint8_t*>(v_pool);
  ep.lambda = lambda;
  ep.slots = nullptr;
  ep.page_table = page_table;
  ep.seq_lens = seq_lens;
  ep.max_pages = max_pages_per_seq;
  ep.status = status;
  ep.num_slots = static_cast<long long>(num_pages) * L.page_size;
  // a large codebook's append goes over several CTAs per vector, its
  // candidates in the workspace after the split partials
  const WsLayout wsl = ws_layout(L, batch, p.splits);
  int2* cand = wide ? reinterpret_cast<int2*>(static_cast<uint8_t*>(workspace) + wsl.cand_off) : nullptr;

  if (fused) {
    p.append = 1;
    p.k_new = k_new;
    p.v_new = v_new;
    p.k_pool_w = static_cast<uint8_t*>(k_pool);
    p.v_pool_w = static_cast<uint8_t*>(v_pool);
    bool overlap = false;
    if (wide) {  // the sliced scan first; the attention kernel merges its candidates
      st = launch_encode_impl(L, ep, batch, true, true, stream, "vq_decode_step append scan", false, cand,
                              false);
      if (st != VQ_OK) return st;
      if (ep.slices <= 1) return fail(VQ_ERR_UNSUPPORTED, "vq_decode_step: the append scan was not sliced");
      p.app_cand = cand;
      p.app_slices = ep.slices;
      overlap = true;
    }
    st = launch_partial(L, p, grid, smem, stream, overlap);
    if (st != VQ_OK) return st;
    return combine_impl(layout, batch, max_seq_len, p.splits, workspace, workspace_bytes, out, stream,
                        true);
  }

  // 1. append: token seq_lens[b] - 1 of every sequence, slot from the page table
  st = launch_encode_impl(L, ep, batch, true, true, stream, "vq_decode_step append encode", false, cand);
  if (st != VQ_OK) return st;
  // 2. split attention (its copies wait for the append), 3. merge of the splits
  st = launch_partial(L, p, grid, smem, stream, true);
  if (st != VQ_OK) return st;
  return combine_impl(layout, batch, max_seq_len, p.splits, workspace, workspace_bytes, out, stream,
                      true);
}

vq_status vq_decode_attention(const vq_layout* layout, int32_t batch, const void* q,
                              const float* lambda, const void* codebook_k, const void* codebook_v,
                              const void* k_pool, const void* v_pool, int64_t num_pages,
                              const int32_t* page_table, int32_t max_pages_per_seq,
                              const int32_t* seq_lens, int32_t max_seq_len, float softmax_scale,
                              int32_t num_splits, void* out, void* workspace,
                              size_t workspace_bytes, int32_t* status, void* stream) {
  vq_status st = check_layout_impl(layout, 1);
  if (st != VQ_OK) return st;
  if (batch < 0) return fail(VQ_ERR_INVALID_ARG, "batch %d < 0", batch);
  if (batch == 0) return VQ_OK;
  if (!out) return fail(VQ_ERR_INVALID_ARG, "out is NULL");
  if (!aligned16(out)) return fail(VQ_ERR_INVALID_ARG, "out is not 16-byte aligned");
  vqk::DecodeParams p;
  int grid = 0;
  size_t smem = 0;
  st = prepare_decode(layout, batch, q, lambda, codebook_k, codebook_v, k_pool, v_pool, num_pages,
                      page_table, max_pages_per_seq, seq_lens, max_seq_len, softmax_scale,
                      num_splits, workspace, workspace_bytes, status, p, grid, smem);
  if (st != VQ_OK) return st;
  st = launch_partial(*layout, p, grid, smem, stream, false);
  if (st != VQ_OK) return st;
  return combine_impl(layout, batch, max_seq_len, p.splits, workspace, workspace_bytes, out, stream,
                      true);
}

}  // extern "C"

// ---- decode attention without a caller workspace ----------------------------
// Some callers cannot allocate device memory at the point where they run
// attention: code that executes inside a region where allocation is forbidden
// or would synchronise the device, embedders whose memory is owned by a
// foreign allocator they cannot call, or plug-ins that are handed only the
// tensors of one call.  For them the split partials live in this fixed,
// file-scope device array instead of a workspace.  Every GPU that loads the
// library holds the array until the process exits.
namespace {

constexpr size_t kStaticScratchBytes = size_t(4) << 20;  // 4 MiB
static __device__ __align__(256) unsigned char g_static_scratch[kStaticScratchBytes];

std::mutex g_scratch_mu;
struct ScratchAddr {
  unsigned long long ctx_id;  // the context the address belongs to (0: not looked up)
  void* ptr;
};
ScratchAddr g_scratch[vqk::kMaxDevices] = {};

// Identity of the current context, so that an address looked up in a context
// that has since been destroyed (cudaDeviceReset) is looked up again.  The
// driver entry points come through the runtime, so no driver library is linked.
unsigned long long current_context_id() {
  using GetCurrent = int (*)(void**);
  using GetId = int (*)(void*, unsigned long long*);
  static GetCurrent get_current = nullptr;
  static GetId get_id = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &f, 12000, cudaEnableDefault, nullptr) ==
        cudaSuccess)
      get_current = reinterpret_cast<GetCurrent>(f);
    f = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &f, 12000, cudaEnableDefault, nullptr) ==
        cudaSuccess)
      get_id = reinterpret_cast<GetId>(f);
  });
  void* ctx = nullptr;
  unsigned long long id = 0;
  if (!get_current || !get_id || get_current(&ctx) != 0 || !ctx || get_id(ctx, &id) != 0) return 1;
  return id + 1;  // never 0
}

// Device address of the array in the current context (a host-side name of a
// __device__ variable is not a device address); looked up once per device and
// context.
vq_status static_scratch(void** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= vqk::kMaxDevices) return fail(VQ_ERR_UNSUPPORTED, "device %d out of range", dev);
  const unsigned long long ctx = current_context_id();
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (g_scratch[dev].ctx_id != ctx || !g_scratch[dev].ptr) {
    void* ptr = nullptr;
    e = cudaGetSymbolAddress(&ptr, g_static_scratch);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress(static scratch)");
    g_scratch[dev].ptr = ptr;
    g_scratch[dev].ctx_id = ctx;
  }
  *out = g_scratch[dev].ptr;
  return VQ_OK;
}

}  // namespace

extern "C" {

vq_status vq_decode_attention_static(const vq_layout* layout, int32_t batch, const void* q,
                                     const float* lambda, const void* codebook_k,
                                     const void* codebook_v, const void* k_pool,
                                     const void* v_pool, int64_t num_pages,
                                     const int32_t* page_table, int32_t max_pages_per_seq,
                                     const int32_t* seq_lens, int32_t max_seq_len,
                                     float softmax_scale, int32_t num_splits, void* out,
                                     int32_t* status, void* stream) {
  vq_status st = check_layout_impl(layout, 1);
  if (st != VQ_OK) return st;
  if (batch < 0) return fail(VQ_ERR_INVALID_ARG, "batch %d < 0", batch);
  if (batch == 0) return VQ_OK;
  if (!out) return fail(VQ_ERR_INVALID_ARG, "out is NULL");
  if (!aligned16(out)) return fail(VQ_ERR_INVALID_ARG, "out is not 16-byte aligned");
  if (max_seq_len < 0) return fail(VQ_ERR_INVALID_ARG, "max_seq_len %d < 0", max_seq_len);
  if (num_splits > kMaxSplits) return fail(VQ_ERR_INVALID_ARG, "num_splits %d > %d", num_splits, kMaxSplits);
  int splits = num_splits;
  if (splits <= 0) {
    // the library's split choice, lowered until the partials fit the array
    const int sms = device_sms();
    if (sms <= 0) return fail(VQ_ERR_CUDA, "no CUDA device");
    splits = pick_splits(*layout, batch, max_seq_len, sms);
    while (splits > 1 && ws_layout(*layout, batch, splits).total > kStaticScratchBytes) --splits;
  }
  const size_t need = ws_layout(*layout, batch, splits).total;
  if (need > kStaticScratchBytes)
    return fail(VQ_ERR_WORKSPACE,
                "batch %d x %d query heads x %d splits needs %zu bytes of split scratch; the static "
                "scratch holds %zu bytes (use vq_decode_attention with a workspace, or fewer splits)",
                batch, layout->num_q_heads, splits, need, kStaticScratchBytes);
  void* scratch = nullptr;
  st = static_scratch(&scratch);
  if (st != VQ_OK) return st;
  // The split kernel writes every partial it later merges, so nothing in the
  // scratch has to start at zero; stale contents of an earlier call are never read.
  vqk::DecodeParams p;
  int grid = 0;
  size_t smem = 0;
  st = prepare_decode(layout, batch, q, lambda, codebook_k, codebook_v, k_pool, v_pool, num_pages,
                      page_table, max_pages_per_seq, seq_lens, max_seq_len, softmax_scale, splits,
                      scratch, kStaticScratchBytes, status, p, grid, smem);
  if (st != VQ_OK) return st;
  st = launch_partial(*layout, p, grid, smem, stream, false);
  if (st != VQ_OK) return st;
  return combine_impl(layout, batch, max_seq_len, splits, scratch, kStaticScratchBytes, out, stream,
                      true);
}

size_t vq_static_scratch_bytes(void) { return kStaticScratchBytes; }

const char* vq_last_error(void) { return g_last_error.c_str(); }

const char* vq_version(void) { return "vqattn 0.1.0 sm_103a"; }

size_t vq_decode_residual_workspace_bytes(const vq_layout* layout, int32_t batch,
                                          int32_t max_seq_len, int32_t num_splits,
                                          int32_t num_sms) {
  if (!layout || batch < 0 || max_seq_len < 0 || layout->num_q_heads < 1) return 0;
  int splits = num_splits;
  if (splits <= 0) splits = vq_default_num_splits(layout, batch, max_seq_len, num_sms);
  if (splits <= 0 || splits > kMaxSplits) return 0;
  return ws_layout(*layout, batch, splits).total;
}

vq_status vq_decode_attention_residual(const vq_layout* layout, int32_t batch, const void* q,
                                       const float* lambda, const void* codebook_k,
                                       const void* codebook_v, const void* k_pool,
                                       const void* v_pool, int64_t num_pages,
                                       const int32_t* page_table, int32_t max_pages_per_seq,
                                       const int32_t* seq_lens, int32_t max_seq_len,
                                       const void* k_res, const void* v_res,
                                       const int32_t* res_lens, int32_t res_capacity,
                                       float softmax_scale, int32_t num_splits, void* out,
                                       void* workspace, size_t workspace_bytes, int32_t* status,
                                       void* stream) {
  vq_status st = check_layout_impl(layout, 1);
  if (st != VQ_OK) return st;
  const vq_layout& L = *layout;
  if (batch < 0) return fail(VQ_ERR_INVALID_ARG, "batch %d < 0", batch);
  if (batch == 0) return VQ_OK;
  if (res_capacity < 1 || res_capacity > kMaxResidual)
    return fail(VQ_ERR_INVALID_ARG, "res_capacity %d not in 1..%d", res_capacity, kMaxResidual);
  const void* ptrs[] = {out, k_res, v_res, res_lens};
  const char* names[] = {"out", "k_res", "v_res", "res_lens"};
  for (int i = 0; i < 4; ++i) {
    if (!ptrs[i]) return fail(VQ_ERR_INVALID_ARG, "%s is NULL", names[i]);
    if (!aligned16(ptrs[i])) return fail(VQ_ERR_INVALID_ARG, "%s is not 16-byte aligned", names[i]);
  }
  vqk::DecodeParams p;
  int grid = 0;
  size_t smem = 0;
  st = prepare_decode(layout, batch, q, lambda, codebook_k, codebook_v, k_pool, v_pool, num_pages,
                      page_table, max_pages_per_seq, seq_lens, max_seq_len, softmax_scale,
                      num_splits, workspace, workspace_bytes, status, p, grid, smem, nullptr,
                      vqk::kMethodGather, res_capacity);
  if (st != VQ_OK) return st;

  // 1. split attention over the codes, every unit merging its slice of the
  // residual window into its own partial, 2. merge of the splits
  p.residual = 1;
  p.k_res = k_res;
  p.v_res = v_res;
  p.res_lens = res_lens;
  p.res_capacity = res_capacity;
  const float scale = softmax_scale == 0.f ? 1.f / std::sqrt(static_cast<float>(L.head_dim)) : softmax_scale;
  p.res_scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  st = launch_partial(L, p, grid, smem, stream, false);
  if (st != VQ_OK) return st;
  return combine_impl(layout, batch, max_seq_len, p.splits, workspace, workspace_bytes, out, stream,
                      true);
}

}  // extern "C"

// ---- page tables, slot maps and rotary positions -------------------------------
namespace {

// The frequencies of a rotary configuration as 64-bit fractions of a turn
// per position; false when they are not finite.
bool rotary_frequencies(const vq_rotary_config& c, unsigned long long (&freq)[64]) {
  const double kTwoPi = 6.283185307179586;
  const double r = c.rotary_dim;
  double base = c.base;
  if (c.scaling == VQ_ROTARY_BASE && c.rotary_dim > 2) base *= std::pow(c.factor, r / (r - 2.0));
  double lo = 0, hi = 0;
  if (c.scaling == VQ_ROTARY_PARTS) {
    auto at = [&](double turns) { return r * std::log(c.original_len / (turns * kTwoPi)) / (2.0 * std::log(base)); };
    lo = std::max(std::floor(at(c.high_turns)), 0.0);
    hi = std::min(std::ceil(at(c.low_turns)), r - 1.0);
  }
  for (int i = 0; i < 64; ++i) freq[i] = 0;
  for (int i = 0; i < c.rotary_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / r);
    if (c.scaling == VQ_ROTARY_LINEAR) {
      f /= c.factor;
    } else if (c.scaling == VQ_ROTARY_PARTS) {
      const double ramp = std::min(std::max((i - lo) / std::max(hi - lo, 1e-3), 0.0), 1.0);
      f = f * (1.0 - ramp) + f / c.factor * ramp;
    } else if (c.scaling == VQ_ROTARY_WAVELENGTH) {
      const double w = std::min(std::max((c.original_len * f / kTwoPi - c.low_turns) / (c.high_turns - c.low_turns), 0.0), 1.0);
      f = w * f + (1.0 - w) * f / c.factor;
    }
    double turns = f / kTwoPi;
    if (!std::isfinite(turns)) return false;
    turns -= std::floor(turns);
    const double scaled = turns * 18446744073709551616.0;  // 2^64
    freq[i] = scaled >= 18446744073709551615.0 ? 0ULL : static_cast<unsigned long long>(scaled);
  }
  return true;
}

vq_status check_rotary_config(const vq_rotary_config* config, int32_t dtype) {
  if (!config) return fail(VQ_ERR_INVALID_ARG, "config is NULL");
  const vq_rotary_config& c = *config;
  if (c.head_dim != 128)
    return fail(VQ_ERR_UNSUPPORTED, "head_dim %d: this build implements head_dim 128", c.head_dim);
  if (c.rotary_dim < 2 || c.rotary_dim > c.head_dim || c.rotary_dim % 2)
    return fail(VQ_ERR_INVALID_ARG, "rotary_dim %d must be even and in 2..%d", c.rotary_dim, c.head_dim);
  if (c.scaling < VQ_ROTARY_NONE || c.scaling > VQ_ROTARY_WAVELENGTH)
    return fail(VQ_ERR_INVALID_ARG, "scaling %d is not a vq_rotary_scaling", c.scaling);
  if (!(c.base >= 1.0) || !std::isfinite(c.base)) return fail(VQ_ERR_INVALID_ARG, "base must be finite and >= 1");
  if (!(c.attention_factor > 0.0) || !std::isfinite(c.attention_factor))
    return fail(VQ_ERR_INVALID_ARG, "attention_factor must be finite and > 0");
  if (c.scaling != VQ_ROTARY_NONE && (!(c.factor > 0.0) || !std::isfinite(c.factor)))
    return fail(VQ_ERR_INVALID_ARG, "factor must be finite and > 0");
  if (c.scaling == VQ_ROTARY_PARTS || c.scaling == VQ_ROTARY_WAVELENGTH) {
    if (!(c.original_len > 0.0) || !std::isfinite(c.original_len) || !(c.low_turns > 0.0) ||
        !(c.high_turns > c.low_turns) || !std::isfinite(c.high_turns))
      return fail(VQ_ERR_INVALID_ARG, "original_len > 0 and 0 < low_turns < high_turns are needed");
    if (c.scaling == VQ_ROTARY_PARTS && !(c.base > 1.0))
      return fail(VQ_ERR_INVALID_ARG, "scaling by parts needs a base > 1");
  }
  if (dtype != VQ_FP16 && dtype != VQ_BF16) return fail(VQ_ERR_INVALID_ARG, "dtype %d is not a vq_dtype", dtype);
  return VQ_OK;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

}  // namespace

extern "C" {

vq_status vq_append_slots(int32_t batch, const int32_t* seq_lens, const int32_t* new_lens,
                          int32_t* page_table, int32_t max_pages_per_seq,
                          const int32_t* free_pages, int32_t free_capacity,
                          const int32_t* num_free, int32_t page_size, int64_t num_pages,
                          int32_t max_tokens, int32_t* seq_lens_out, int32_t* num_free_out,
                          int32_t* cu_new_lens, int64_t* slot_mapping, int32_t* positions,
                          int32_t* status, void* stream) {
  if (batch < 0) return fail(VQ_ERR_INVALID_ARG, "batch %d < 0", batch);
  if (batch > vqk::kSlotsMaxBatch)
    return fail(VQ_ERR_UNSUPPORTED, "batch %d > %d", batch, vqk::kSlotsMaxBatch);
  if (page_size < 16 || page_size % 16)
    return fail(VQ_ERR_INVALID_ARG, "page_size %d must be a positive multiple of 16", page_size);
  if (num_pages < 1) return fail(VQ_ERR_INVALID_ARG, "num_pages %lld < 1", (long long)num_pages);
  if (max_pages_per_seq < 1) return fail(VQ_ERR_INVALID_ARG, "max_pages_per_seq %d < 1", max_pages_per_seq);
  if (free_capacity < 0) return fail(VQ_ERR_INVALID_ARG, "free_capacity %d < 0", free_capacity);
  if (max_tokens < 0 || max_tokens > (1 << 30))
    return fail(VQ_ERR_INVALID_ARG, "max_tokens %d not in 0..2^30", max_tokens);
  // an empty batch, free list or row list may come with NULL pointers
  const void* ptrs[] = {seq_lens, new_lens, page_table, seq_lens_out, free_pages, num_free,
                        num_free_out, cu_new_lens, slot_mapping, positions};
  const char* names[] = {"seq_lens", "new_lens", "page_table", "seq_lens_out", "free_pages", "num_free",
                         "num_free_out", "cu_new_lens", "slot_mapping", "positions"};
  for (int i = 0; i < 10; ++i) {
    const bool may_be_null = i < 4 ? batch == 0 : i == 4 ? free_capacity == 0 : i >= 8 && max_tokens == 0;
    if (!ptrs[i] && !may_be_null) return fail(VQ_ERR_INVALID_ARG, "%s is NULL", names[i]);
    if (!aligned16(ptrs[i])) return fail(VQ_ERR_INVALID_ARG, "%s is not 16-byte aligned", names[i]);
  }
  vqk::SlotsParams p{};
  p.seq_lens = seq_lens;
  p.new_lens = new_lens;
  p.free_pages = free_pages;
  p.num_free = num_free;
  p.page_table = page_table;
  p.seq_lens_out = seq_lens_out;
  p.num_free_out = num_free_out;
  p.cu_new_lens = cu_new_lens;
  p.slot_mapping = slot_mapping;
  p.positions = positions;
  p.status = status;
  p.num_pages = num_pages;
  p.batch = batch;
  p.max_pages = max_pages_per_seq;
  p.free_capacity = free_capacity;
  p.page_size = page_size;
  p.max_tokens = max_tokens;
  cudaError_t e = vqk::launch_slots(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "vq_append_slots launch");
  return VQ_OK;
}

vq_status vq_rotary(const vq_rotary_config* config, int32_t num_tokens, const int32_t* positions,
                    int32_t dtype, const void* q, int64_t q_stride, int32_t num_q_heads,
                    void* q_out, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                    int32_t num_kv_heads, void* k_out, void* v_out, void* stream) {
  vq_status checked = check_rotary_config(config, dtype);
  if (checked != VQ_OK) return checked;
  const vq_rotary_config& c = *config;
  if (num_tokens < 0) return fail(VQ_ERR_INVALID_ARG, "num_tokens %d < 0", num_tokens);
  if (num_tokens == 0) return VQ_OK;  // empty tensors may come with NULL pointers
  if (!positions || !aligned16(positions))
    return fail(VQ_ERR_INVALID_ARG, "positions is NULL or not 16-byte aligned");
  const void* src[] = {q, k, v};
  void* dst[] = {q_out, k_out, v_out};
  const int64_t stride[] = {q_stride, k_stride, v_stride};
  const int32_t heads[] = {num_q_heads, num_kv_heads, num_kv_heads};
  const char* names[] = {"q", "k", "v"};
  vqk::RotaryParams p{};
  size_t in_bytes[3] = {}, out_bytes[3] = {};
  bool any = false;
  for (int i = 0; i < 3; ++i) {
    if (!src[i] != !dst[i]) return fail(VQ_ERR_INVALID_ARG, "%s and %s_out go together", names[i], names[i]);
    if (!src[i]) continue;
    any = true;
    if (!aligned16(src[i]) || !aligned16(dst[i]))
      return fail(VQ_ERR_INVALID_ARG, "%s or %s_out is not 16-byte aligned", names[i], names[i]);
    if (heads[i] < 1 || heads[i] > 4096) return fail(VQ_ERR_INVALID_ARG, "%d heads of %s: 1..4096", heads[i], names[i]);
    const int64_t row = static_cast<int64_t>(heads[i]) * c.head_dim;
    if (stride[i] < row || stride[i] % 8 || stride[i] > (1LL << 31))
      return fail(VQ_ERR_INVALID_ARG, "%s_stride %lld must be a multiple of 8, at least %lld and at most 2^31", names[i],
                  (long long)stride[i], (long long)row);
    p.src[i] = src[i];
    p.dst[i] = dst[i];
    p.stride[i] = stride[i];
    p.heads[i] = heads[i];
    in_bytes[i] = 2 * (static_cast<size_t>(num_tokens - 1) * stride[i] + row);
    out_bytes[i] = 2 * static_cast<size_t>(num_tokens) * row;
  }
  if (!any) return fail(VQ_ERR_INVALID_ARG, "q, k and v are all NULL");
  for (int o = 0; o < 3; ++o) {
    if (!dst[o]) continue;
    for (int i = 0; i < 3; ++i) {
      if (!src[i]) continue;
      const bool in_place = i == o && dst[o] == src[i] && dtype == VQ_FP16 && in_bytes[i] == out_bytes[o];
      if (!in_place && overlap(dst[o], out_bytes[o], src[i], in_bytes[i]))
        return fail(VQ_ERR_INVALID_ARG, "%s_out overlaps %s", names[o], names[i]);
      if (i > o && dst[i] && overlap(dst[o], out_bytes[o], dst[i], out_bytes[i]))
        return fail(VQ_ERR_INVALID_ARG, "%s_out overlaps %s_out", names[o], names[i]);
    }
    if (overlap(dst[o], out_bytes[o], positions, 4 * static_cast<size_t>(num_tokens)))
      return fail(VQ_ERR_INVALID_ARG, "%s_out overlaps positions", names[o]);
  }
  if (!rotary_frequencies(c, p.freq)) return fail(VQ_ERR_INVALID_ARG, "the frequencies are not finite");
  p.positions = positions;
  p.factor = static_cast<float>(c.attention_factor);
  p.rotary_dim = c.rotary_dim;
  p.interleaved = c.interleaved != 0;
  p.num_tokens = num_tokens;
  const int sms = device_sms();
  if (sms <= 0) return fail(VQ_ERR_CUDA, "no CUDA device");
  cudaError_t e = vqk::launch_rotary(p, dtype == VQ_BF16, sms, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "vq_rotary launch");
  return VQ_OK;
}

}  // extern "C"

// ---- attention of several new tokens per sequence --------------------------------
namespace {

// Tile height of a call, by the rows of its longest (sequence, KV head): all
// of them where 8 or 16 hold them (warp mma), else 128 (tcgen05) or 256 (a
// pair of CTAs on one product).  Where three tiles of 128 hold the rows, the
// pair's second tile is mostly empty and one CTA is faster, but for the 1.5-bit
// format.  Measured on the device, merge included, from a cold L2 (4 heads per
// KV head, (4,8) codes; batch 8: contexts of 4000 to 8000; batch 16: (2,8)
// keys, 3000 to 6000):
//   5 rows (5 heads), 64 windows of 4096: 99 us at height 8, 221 at 16
//   12 to 16 rows, batch 8: 48 us at 16, 60 at 128
//   20 to 32 rows, batch 8: 70 to 72 us at 16, 60 to 62 at 128; 32 rows 78 at 256
//   128 rows, batch 8: 65 us at 128, 80 at 256; 192 rows: 89 and 83
//   260 to 384 rows, batch 8: 116 to 121 us at 128, 127 to 130 at 256; one
//     sequence of 32K: 83 to 84 and 91; batch 16: 182 to 188 and 185 to 188;
//     1.5 bit, one sequence of 8K: 56 and 52 to 55
//   512 rows, batch 8: 146 us at 128, 131 at 256; 640 rows: 170 and 178, but
//     batch 16: 290 and 266 (left to 256); ragged chunks of 1 to 100 tokens
//     (400 rows), batch 16 of 4096 to 8192: 158 and 168 (left to 256 too)
//   2048 rows, one chunk of 512 tokens in 8K: 103 us at 128, 97 at 256
// The height is the whole call's, from the bound of its longest chunk: many
// single tokens beside one chunk pay for rows that they have not.  63 single
// tokens (4000 to 16 000) and a chunk of 512: 668 us in one call, 144 and 97 in
// two; 32 (4000 to 10 000) and a chunk of 5: 166, or 67 and 43.
// VQ_CHUNK_ROWS=16|128|256 selects a height explicitly (a tuning switch for
// profiling).
int chunk_tile_rows(const vq_layout& L, int max_new_len) {
  const long long rows = static_cast<long long>(max_new_len) * (L.num_q_heads / L.num_kv_heads);
  if (const char* env = std::getenv("VQ_CHUNK_ROWS")) {
    if (std::strcmp(env, "16") == 0) return 16;
    if (std::strcmp(env, "128") == 0) return 128;
    if (std::strcmp(env, "256") == 0) return 256;
  }
  const int per_tile = 128 / (L.num_q_heads / L.num_kv_heads);  // tokens of 128 rows
  const bool three = max_new_len > 2 * per_tile && max_new_len <= 3 * per_tile && L.k_bits != 12;
  return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 128 || three ? 128 : 256;
}

struct ChunkWs {
  size_t o_off, ml_off, rec_off, total;
};

// Workers of a launch over `grid` CTAs.
int chunk_workers(int tile_rows, int grid) {
  return tile_rows == 8 ? vqk::kFewGroups * grid : tile_rows == 256 ? grid / 2 : grid;
}

// Two partials and a record per worker.
ChunkWs chunk_ws(int tile_rows, int grid) {
  ChunkWs w;
  const size_t workers = chunk_workers(tile_rows, grid), rows = 2 * workers * tile_rows;
  w.o_off = 0;
  w.ml_off = rows * 128 * sizeof(float);
  w.rec_off = (w.ml_off + rows * sizeof(float2) + 255) & ~size_t(255);
  w.total = (w.rec_off + workers * sizeof(vqk::ChunkRecord) + 255) & ~size_t(255);
  return w;
}

// Tile height of a call over trees of drafted tokens, by the rows of its longest (sequence, KV head): 16 or (but for the 1.5-bit
// format) 32 of vq_tree.cu where they hold them, else 128 (or what three of these hold, but for the 1.5-bit format) or 256
// of vq_chunk_wide.cu.  Measured (us a call of many, merge included, inputs that change; contexts of 4000 to 8000, 4 heads
// per KV head, (4,8) where nothing else is said):
//   16 rows, batch 8: 41 at 16, 49 at 32, 55 at 128; 20 to 32 rows: 59 at 16, 49 at 32, 56 at 128
//   1.5 bit, contexts of 3000 to 6000, batch 48: 16 rows 153 at 16, 185 at 128; 28 rows 288 at 16, 186 at 128
//   64 rows, batch 8: 74 at 32, 57 at 128, 84 at 256
//   192 rows, batch 8: 92 at 128, 89 at 256; batch 16 at (2,8): 161 and 154; 250 rows at (2,8), (4,9): 175 and 161;
//     256 rows, 1.5 bit: 110 and 96
//   320 rows, batch 8: 124 at 128, 146 at 256; 384 rows, batch 16 at (2,8): 239 and 284
// Trees of different sizes under a bound of two tiles of 128 rows: one such tile takes about 0.7 of the time of a tile of
// 256, two of them 1.1, so 128 wins where a third of the sequences need one only.  For sizes spread evenly that is a mean
// of at most 96 rows and a quarter of the bound.  (Sequences without drafted tokens lower the mean too.)  At 128 | 256, batch
// 24, contexts of 0 to 9001:
//   1 to 61 tokens at (2,8) 144 | 168, 1 to 50 of 5 heads at (2,8), (4,9) 153 | 172, 1 to 64 at 1.5 bit 162 | 169
//   above that mean: 20 to 50 of 5 heads 178 | 175
// The mean is that of num_tokens, the rows of the tensors: where a captured graph has rows for the bound of every sequence, the
// mean is the bound and the height 256.
// VQ_TREE_ROWS=16|32|128|256 selects one explicitly (a tuning switch for profiling).
int tree_tile_rows(const vq_layout& L, int batch, int num_tokens, int max_new_len) {
  const int group = L.num_q_heads / L.num_kv_heads;
  const int narrow = L.k_bits == 12 ? 16 : 32;  // the most of vq_tree.cu
  if (const char* env = std::getenv("VQ_TREE_ROWS"))
    for (int rows : {16, 32, 128, 256})
      if (std::atoi(env) == rows && (rows <= narrow || rows >= 128)) return rows;
  const long long rows = static_cast<long long>(max_new_len) * group;
  const int per_tile = 128 / group;  // tokens of 128 rows
  const bool three = max_new_len > 2 * per_tile && max_new_len <= 3 * per_tile && L.k_bits != 12;
  const bool ragged = max_new_len <= 2 * per_tile && static_cast<long long>(num_tokens) * group <= (96 + rows / 4) * batch;
  return rows <= 16 ? 16 : rows <= narrow ? 32 : rows <= 128 || three || ragged ? 128 : 256;
}

struct TreeArgs {
  const uint64_t* masks;
  int32_t mask_words;
  const int32_t* positions;
};

// vq_chunk_attention, or with `tree` vq_tree_attention.
vq_status attention_of_rows(const vq_layout* layout, int32_t batch, int32_t num_tokens,
                            const void* q, const float* lambda, const void* codebook_k,
                            const void* codebook_v, const void* k_pool, const void* v_pool,
                            int64_t num_pages, const int32_t* page_table,
                            int32_t max_pages_per_seq, const int32_t* seq_lens,
                            int32_t max_seq_len, const int32_t* cu_new_lens, int32_t max_new_len,
                            int32_t window, int32_t num_sinks, float softmax_scale, void* out,
                            void* workspace, size_t workspace_bytes, int32_t* status,
                            void* stream, const TreeArgs* tree) {
  vq_status st = check_layout_impl(layout, 1);
  if (st != VQ_OK) return st;
  const vq_layout& L = *layout;
  if (batch < 0) return fail(VQ_ERR_INVALID_ARG, "batch %d < 0", batch);
  if (batch > vqk::kChunkMaxBatch) return fail(VQ_ERR_UNSUPPORTED, "batch %d > %d", batch, vqk::kChunkMaxBatch);
  if (num_tokens < 0) return fail(VQ_ERR_INVALID_ARG, "num_tokens %d < 0", num_tokens);
  if (max_new_len < 0) return fail(VQ_ERR_INVALID_ARG, "max_new_len %d < 0", max_new_len);
  if (window < 0 || num_sinks < 0) return fail(VQ_ERR_INVALID_ARG, "window %d or num_sinks %d < 0", window, num_sinks);
  if (num_sinks > 0 && window == 0) return fail(VQ_ERR_INVALID_ARG, "num_sinks %d without a window", num_sinks);
  if (!std::isfinite(softmax_scale)) return fail(VQ_ERR_INVALID_ARG, "softmax_scale is not finite");
  if (batch == 0 || num_tokens == 0 || max_new_len == 0) return VQ_OK;
  if (!cu_new_lens && num_tokens < batch)
    return fail(VQ_ERR_INVALID_ARG, "num_tokens %d < batch %d without cu_new_lens", num_tokens, batch);
  const void* ptrs[] = {q, lambda, codebook_k, codebook_v, k_pool, v_pool, page_table, seq_lens, out, workspace, cu_new_lens};
  const char* names[] = {"q", "lambda", "codebook_k", "codebook_v", "k_pool", "v_pool", "page_table",
                         "seq_lens", "out", "workspace", "cu_new_lens"};
  for (int i = 0; i < 11; ++i) {
    if (!ptrs[i] && i < 10) return fail(VQ_ERR_INVALID_ARG, "%s is NULL", names[i]);
    if (!aligned16(ptrs[i])) return fail(VQ_ERR_INVALID_ARG, "%s is not 16-byte aligned", names[i]);
  }
  if (num_pages < 1) return fail(VQ_ERR_INVALID_ARG, "num_pages %lld < 1", (long long)num_pages);
  if (max_pages_per_seq < 1) return fail(VQ_ERR_INVALID_ARG, "max_pages_per_seq %d < 1", max_pages_per_seq);
  if (max_seq_len < 0 || max_seq_len > (1 << 30))
    return fail(VQ_ERR_INVALID_ARG, "max_seq_len %d not in 0..2^30", max_seq_len);
  if (static_cast<long long>(max_seq_len) > static_cast<long long>(max_pages_per_seq) * L.page_size)
    return fail(VQ_ERR_INVALID_ARG, "max_seq_len %d exceeds max_pages_per_seq * page_size", max_seq_len);
  const size_t row_bytes = 2 * static_cast<size_t>(L.num_q_heads) * L.head_dim;
  if (overlap(q, num_tokens * row_bytes, out, num_tokens * row_bytes))
    return fail(VQ_ERR_INVALID_ARG, "out overlaps q");
  if (tree) {
    if (max_new_len > vqk::kTreeMaxTokens)
      return fail(VQ_ERR_UNSUPPORTED, "max_new_len %d > %d drafted tokens", max_new_len, vqk::kTreeMaxTokens);
    if (!cu_new_lens) return fail(VQ_ERR_INVALID_ARG, "cu_new_lens is NULL");
    if (!tree->masks || !aligned16(tree->masks)) return fail(VQ_ERR_INVALID_ARG, "tree_masks is NULL or not 16-byte aligned");
    if (tree->mask_words < (max_new_len + 63) / 64 || tree->mask_words > 64)
      return fail(VQ_ERR_INVALID_ARG, "mask_words %d not in %d..64", tree->mask_words, (max_new_len + 63) / 64);
    if (!tree->positions && window > 0) return fail(VQ_ERR_INVALID_ARG, "positions are needed with a window");
    if (!aligned16(tree->positions)) return fail(VQ_ERR_INVALID_ARG, "positions is not 16-byte aligned");
  }
  const int sms = device_sms();
  if (sms <= 0) return fail(VQ_ERR_CUDA, "no CUDA device");
  const int tile_rows = tree ? tree_tile_rows(L, batch, num_tokens, max_new_len) : chunk_tile_rows(L, max_new_len);
  const int grid = tile_rows == 256 ? std::max(sms & ~1, 2) : sms;
  const ChunkWs ws = chunk_ws(tile_rows, grid);
  if (workspace_bytes < ws.total)
    return fail(VQ_ERR_WORKSPACE, "workspace %zu bytes < %zu required", workspace_bytes, ws.total);

  vqk::ChunkParams p{};
  p.q = q;
  p.out = out;
  p.lambda = lambda;
  p.cb_k = codebook_k;
  p.cb_v = codebook_v;
  p.k_pool = static_cast<const uint8_t*>(k_pool);
  p.v_pool = static_cast<const uint8_t*>(v_pool);
  p.page_table = page_table;
  p.seq_lens = seq_lens;
  p.cu = cu_new_lens;
  uint8_t* wsb = static_cast<uint8_t*>(workspace);
  p.ws_o = reinterpret_cast<float*>(wsb + ws.o_off);
  p.ws_ml = reinterpret_cast<float2*>(wsb + ws.ml_off);
  p.records = reinterpret_cast<vqk::ChunkRecord*>(wsb + ws.rec_off);
  p.status = status;
  p.num_pages = num_pages;
  p.batch = batch;
  p.num_tokens = num_tokens;
  p.hq = L.num_q_heads;
  p.hkv = L.num_kv_heads;
  p.group = L.num_q_heads / L.num_kv_heads;
  p.page_size = L.page_size;
  p.page_shift = -1;
  for (int i = 4; i < 31; ++i)
    if (L.page_size == 1 << i) p.page_shift = i;
  p.max_pages = max_pages_per_seq;
  p.max_seq_len = max_seq_len;
  p.max_new_len = max_new_len;
  p.window = tree ? window : std::min(window, 1 << 30);  // (without a tree no position is further back: the same as none)
  p.sinks = tree ? num_sinks : std::min(num_sinks, 1 << 30);
  p.tile_rows = tile_rows;
  // (of 8 rows, 4 where they are enough: the kernel then holds high and low parts side by side)
  const bool few = p.tile_rows == 8 && static_cast<long long>(max_new_len) * p.group <= 4;
  p.tile_tok = p.tile_rows == 256 ? 2 * (128 / p.group) : (few ? 4 : p.tile_rows) / p.group;
  // A tile's fixed cost in tokens: a prompt of 8192 takes 648 us at 256, 585 at 640, 598 at 1024, 643 at 2304;
  // few rows are flat from 128 to 1024 (64 windows of 4096: 95 us at each).
  const bool wide = p.tile_rows >= 128;
  p.gap = wide ? 640 : 256;
  p.min_range = 512;
  // Two seconds, and time for one piece: some waits span a whole one, up to max_seq_len tokens (9 ns per
  // token measured in tiles of 128 and 256 rows; 40 leaves room for slower formats and clocks).
  p.timeout_ns = 2000000000ULL + 40ULL * max_seq_len;
  const float scale = softmax_scale == 0.f ? 1.f / std::sqrt(static_cast<float>(L.head_dim)) : softmax_scale;
  p.qscale = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634 / std::sqrt(128.0));
  if (tree) {
    p.masks = reinterpret_cast<const unsigned long long*>(tree->masks);
    p.mask_words = tree->mask_words;
    p.positions = tree->positions;
  }
  auto launch = tree && wide ? vqk::launch_tree_wide : tree ? vqk::launch_tree : wide ? vqk::launch_chunk_wide : vqk::launch_chunk_narrow;
  cudaError_t e = launch(p, L.k_sub, L.k_bits, L.v_sub, L.v_bits, grid, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, tree ? "vq_tree_attention launch" : "vq_chunk_attention launch");
  e = vqk::launch_chunk_merge(p, chunk_workers(tile_rows, grid), static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, tree ? "vq_tree_attention merge" : "vq_chunk_attention merge");
  return VQ_OK;
}

}  // namespace

extern "C" {

size_t vq_chunk_workspace_bytes(const vq_layout* layout, int32_t batch, int32_t num_tokens,
                                int32_t max_seq_len, int32_t max_new_len, int32_t num_sms) {
  if (check_layout_impl(layout, 1) != VQ_OK || batch < 0 || num_tokens < 0 || max_seq_len < 0 || max_new_len < 0)
    return 0;
  const int sms = num_sms > 0 ? num_sms : device_sms();
  if (sms <= 0) return 0;
  // a call with smaller bounds may take another tile (of 128 rows also 256), whose slots may be more
  size_t most = 0;
  const int need = chunk_tile_rows(*layout, max_new_len);
  for (int rows : {8, 16, 128, 256})
    if (rows <= need || need == 128) most = std::max(most, chunk_ws(rows, sms).total);
  return most;
}

vq_status vq_chunk_attention(const vq_layout* layout, int32_t batch, int32_t num_tokens,
                             const void* q, const float* lambda, const void* codebook_k,
                             const void* codebook_v, const void* k_pool, const void* v_pool,
                             int64_t num_pages, const int32_t* page_table,
                             int32_t max_pages_per_seq, const int32_t* seq_lens,
                             int32_t max_seq_len, const int32_t* cu_new_lens, int32_t max_new_len,
                             int32_t window, int32_t num_sinks, float softmax_scale, void* out,
                             void* workspace, size_t workspace_bytes, int32_t* status,
                             void* stream) {
  return attention_of_rows(layout, batch, num_tokens, q, lambda, codebook_k, codebook_v, k_pool, v_pool, num_pages, page_table,
                           max_pages_per_seq, seq_lens, max_seq_len, cu_new_lens, max_new_len, window, num_sinks, softmax_scale,
                           out, workspace, workspace_bytes, status, stream, nullptr);
}

size_t vq_tree_workspace_bytes(const vq_layout* layout, int32_t batch, int32_t num_tokens,
                               int32_t max_seq_len, int32_t max_new_len, int32_t num_sms) {
  if (check_layout_impl(layout, 1) != VQ_OK || batch < 0 || num_tokens < 0 || max_seq_len < 0 || max_new_len < 0)
    return 0;
  const int sms = num_sms > 0 ? num_sms : device_sms();
  if (sms <= 0) return 0;
  size_t most = 0;  // a call with smaller bounds may take another tile (of 128 rows also 256)
  const int need = tree_tile_rows(*layout, batch, num_tokens, max_new_len);
  for (int rows : {16, 32, 128, 256})
    if (rows <= need || need == 128) most = std::max(most, chunk_ws(rows, std::max(sms, 2)).total);
  return most;
}

vq_status vq_tree_attention(const vq_layout* layout, int32_t batch, int32_t num_tokens,
                            const void* q, const float* lambda, const void* codebook_k,
                            const void* codebook_v, const void* k_pool, const void* v_pool,
                            int64_t num_pages, const int32_t* page_table,
                            int32_t max_pages_per_seq, const int32_t* seq_lens,
                            int32_t max_seq_len, const int32_t* cu_new_lens, int32_t max_new_len,
                            const uint64_t* tree_masks, int32_t mask_words,
                            const int32_t* positions, int32_t window, int32_t num_sinks,
                            float softmax_scale, void* out, void* workspace,
                            size_t workspace_bytes, int32_t* status, void* stream) {
  const TreeArgs tree = {tree_masks, mask_words, positions};
  return attention_of_rows(layout, batch, num_tokens, q, lambda, codebook_k, codebook_v, k_pool, v_pool, num_pages, page_table,
                           max_pages_per_seq, seq_lens, max_seq_len, cu_new_lens, max_new_len, window, num_sinks, softmax_scale,
                           out, workspace, workspace_bytes, status, stream, &tree);
}

}  // extern "C"

// ---- keys and values from a projection's rows, and accepted tokens ----------------
extern "C" {

vq_status vq_append_kv(const vq_layout* layout, const vq_rotary_config* config,
                       int32_t num_tokens, const int32_t* positions,
                       const int64_t* slot_mapping, int32_t dtype, const void* q,
                       int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                       int64_t v_stride, const float* lambda, const void* codebook_k,
                       const void* codebook_v, void* q_out, void* k_pool, void* v_pool,
                       int64_t num_pages, int32_t* status, void* stream) {
  vq_status st = check_layout_impl(layout, 1);
  if (st != VQ_OK) return st;
  const vq_layout& L = *layout;
  st = check_rotary_config(config, dtype);
  if (st != VQ_OK) return st;
  const vq_rotary_config& c = *config;
  if (num_tokens < 0) return fail(VQ_ERR_INVALID_ARG, "num_tokens %d < 0", num_tokens);
  if (num_tokens == 0) return VQ_OK;  // empty tensors may come with NULL pointers
  if (!q != !q_out) return fail(VQ_ERR_INVALID_ARG, "q and q_out go together");
  const void* ptrs[] = {positions, slot_mapping, k, v, lambda, codebook_k, codebook_v, k_pool, v_pool, q, q_out};
  const char* names[] = {"positions", "slot_mapping", "k", "v", "lambda", "codebook_k", "codebook_v", "k_pool", "v_pool", "q", "q_out"};
  for (int i = 0; i < 11; ++i) {
    if (!ptrs[i] && i < 9) return fail(VQ_ERR_INVALID_ARG, "%s is NULL", names[i]);
    if (!aligned16(ptrs[i])) return fail(VQ_ERR_INVALID_ARG, "%s is not 16-byte aligned", names[i]);
  }
  if (num_pages < 1) return fail(VQ_ERR_INVALID_ARG, "num_pages %lld < 1", (long long)num_pages);
  if (L.num_q_heads > 4096) return fail(VQ_ERR_INVALID_ARG, "%d heads of q: 1..4096", L.num_q_heads);
  const void* src[] = {q, k, v};
  const int64_t stride[] = {q_stride, k_stride, v_stride};
  const int32_t heads[] = {L.num_q_heads, L.num_kv_heads, L.num_kv_heads};
  const char* row_names[] = {"q", "k", "v"};
  size_t in_bytes[3] = {};
  for (int i = 0; i < 3; ++i) {
    if (!src[i]) continue;
    const int64_t row = static_cast<int64_t>(heads[i]) * L.head_dim;
    if (stride[i] < row || stride[i] % 8 || stride[i] > (1LL << 31))
      return fail(VQ_ERR_INVALID_ARG, "%s_stride %lld must be a multiple of 8, at least %lld and at most 2^31", row_names[i],
                  (long long)stride[i], (long long)row);
    in_bytes[i] = 2 * (static_cast<size_t>(num_tokens - 1) * stride[i] + row);
  }
  vqk::AppendParams p{};
  const size_t q_bytes = 2 * static_cast<size_t>(num_tokens) * L.num_q_heads * L.head_dim;
  for (int i = 0; q && i < 3; ++i) {
    const bool in_place = i == 0 && q_out == q && dtype == VQ_FP16 && in_bytes[0] == q_bytes;
    if (!in_place && overlap(q_out, q_bytes, src[i], in_bytes[i])) return fail(VQ_ERR_INVALID_ARG, "q_out overlaps %s", row_names[i]);
  }
  if (q && (overlap(q_out, q_bytes, positions, 4 * static_cast<size_t>(num_tokens)) ||
            overlap(q_out, q_bytes, slot_mapping, 8 * static_cast<size_t>(num_tokens))))
    return fail(VQ_ERR_INVALID_ARG, "q_out overlaps positions or slot_mapping");
  if (!rotary_frequencies(c, p.freq)) return fail(VQ_ERR_INVALID_ARG, "the frequencies are not finite");
  const int sms = device_sms();
  if (sms <= 0) return fail(VQ_ERR_CUDA, "no CUDA device");
  p.positions = positions;
  p.slots = slot_mapping;
  p.lambda = lambda;
  p.status = status;
  p.num_slots = static_cast<long long>(num_pages) * L.page_size;
  p.factor = c.attention_factor;
  p.rotary_dim = c.rotary_dim;
  p.interleaved = c.interleaved != 0;
  p.bf16 = dtype == VQ_BF16;
  p.num_tokens = num_tokens;
  p.hkv = L.num_kv_heads;
  p.page_size = L.page_size;
  const void* cb[] = {codebook_k, codebook_v};
  void* pool[] = {k_pool, v_pool};
  const int32_t sub[] = {L.k_sub, L.v_sub}, bits[] = {L.k_bits, L.v_bits};
  for (int i = 0; i < 2; ++i) {
    p.src[i] = src[1 + i];
    p.stride[i] = stride[1 + i];
    p.cb[i] = cb[i];
    p.pool[i] = static_cast<uint8_t*>(pool[i]);
    p.sub[i] = sub[i];
    p.bits[i] = bits[i];
    p.row_bytes[i] = static_cast<int>(vq_code_row_bytes(L.head_dim, sub[i], bits[i]));
  }
  if (q) {
    p.q.positions = positions;
    p.q.src[0] = q;
    p.q.dst[0] = q_out;
    p.q.stride[0] = q_stride;
    p.q.heads[0] = L.num_q_heads;
    for (int i = 0; i < 64; ++i) p.q.freq[i] = p.freq[i];
    p.q.factor = static_cast<float>(c.attention_factor);
    p.q.rotary_dim = c.rotary_dim;
    p.q.interleaved = c.interleaved != 0;
    p.q.num_tokens = num_tokens;
  }
  cudaError_t e = vqk::launch_append(p, sms, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "vq_append_kv launch");
  return VQ_OK;
}

vq_status vq_keep_tokens(const vq_layout* layout, int32_t batch, const int32_t* seq_lens,
                         const int32_t* cu_new_lens, const int32_t* keep, int32_t max_keep,
                         const int32_t* keep_lens, const int32_t* page_table,
                         int32_t max_pages_per_seq, int64_t num_pages, int32_t num_layers,
                         void* const* k_pools, void* const* v_pools, int32_t* free_pages,
                         int32_t free_capacity, const int32_t* num_free, int32_t* seq_lens_out,
                         int32_t* num_free_out, int32_t* status, void* stream) {
  vq_status st = check_layout_impl(layout, 0);
  if (st != VQ_OK) return st;
  const vq_layout& L = *layout;
  if (batch < 0) return fail(VQ_ERR_INVALID_ARG, "batch %d < 0", batch);
  if (batch > vqk::kSlotsMaxBatch) return fail(VQ_ERR_UNSUPPORTED, "batch %d > %d", batch, vqk::kSlotsMaxBatch);
  if (max_keep < 0) return fail(VQ_ERR_INVALID_ARG, "max_keep %d < 0", max_keep);
  if (max_keep > vqk::kKeepMaxTokens) return fail(VQ_ERR_UNSUPPORTED, "max_keep %d > %d", max_keep, vqk::kKeepMaxTokens);
  if (num_layers < 1) return fail(VQ_ERR_INVALID_ARG, "num_layers %d < 1", num_layers);
  if (num_layers > vqk::kKeepMaxLayers) return fail(VQ_ERR_UNSUPPORTED, "num_layers %d > %d", num_layers, vqk::kKeepMaxLayers);
  if (max_pages_per_seq < 1) return fail(VQ_ERR_INVALID_ARG, "max_pages_per_seq %d < 1", max_pages_per_seq);
  if (num_pages < 1) return fail(VQ_ERR_INVALID_ARG, "num_pages %lld < 1", (long long)num_pages);
  if (free_capacity < 0) return fail(VQ_ERR_INVALID_ARG, "free_capacity %d < 0", free_capacity);
  if (batch == 0) return VQ_OK;
  const void* ptrs[] = {seq_lens, cu_new_lens, keep_lens, page_table, num_free, seq_lens_out, num_free_out, k_pools, v_pools, keep, free_pages};
  const char* names[] = {"seq_lens", "cu_new_lens", "keep_lens", "page_table", "num_free", "seq_lens_out", "num_free_out", "k_pools",
                         "v_pools", "keep", "free_pages"};
  for (int i = 0; i < 11; ++i) {
    const bool may_be_null = i == 9 ? max_keep == 0 : i == 10 && free_capacity == 0;
    if (!ptrs[i] && !may_be_null) return fail(VQ_ERR_INVALID_ARG, "%s is NULL", names[i]);
    if (i != 7 && i != 8 && !aligned16(ptrs[i])) return fail(VQ_ERR_INVALID_ARG, "%s is not 16-byte aligned", names[i]);
  }
  vqk::KeepParams p{};
  for (int i = 0; i < num_layers; ++i) {
    if (!k_pools[i] || !v_pools[i] || !aligned16(k_pools[i]) || !aligned16(v_pools[i]))
      return fail(VQ_ERR_INVALID_ARG, "a pool of layer %d is NULL or not 16-byte aligned", i);
    p.pool[0][i] = static_cast<uint8_t*>(k_pools[i]);
    p.pool[1][i] = static_cast<uint8_t*>(v_pools[i]);
  }
  p.seq_lens = seq_lens;
  p.cu = cu_new_lens;
  p.keep = keep;
  p.keep_lens = keep_lens;
  p.page_table = page_table;
  p.free_pages = free_pages;
  p.num_free = num_free;
  p.seq_lens_out = seq_lens_out;
  p.num_free_out = num_free_out;
  p.status = status;
  p.num_pages = num_pages;
  p.batch = batch;
  p.max_keep = max_keep;
  p.max_pages = max_pages_per_seq;
  p.free_capacity = free_capacity;
  p.page_size = L.page_size;
  p.hkv = L.num_kv_heads;
  p.layers = num_layers;
  p.row_bytes[0] = static_cast<int>(vq_code_row_bytes(L.head_dim, L.k_sub, L.k_bits));
  p.row_bytes[1] = static_cast<int>(vq_code_row_bytes(L.head_dim, L.v_sub, L.v_bits));
  const int sms = device_sms();
  if (sms <= 0) return fail(VQ_ERR_CUDA, "no CUDA device");
  cudaError_t e = vqk::launch_keep(p, sms, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "vq_keep_tokens launch");
  return VQ_OK;
}

}  // extern "C"

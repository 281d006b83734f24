// vq_gather.cuh -- codes and centroid gathers shared by the attention kernels.
//
// A kernel keeps its codebooks in a table at the start of its dynamic shared
// memory, and a lane turns a token's codes into table offsets, so a centroid
// is one shared-memory load.
#pragma once

#include "vq_device.cuh"
#include "vq_kernels.h"

namespace vqk {
namespace {

// The dynamic shared memory of the kernel; the codebook table sits at its
// start (offset 0), so a gather is one load at (code << 8) | lane byte.
extern __shared__ __align__(128) uint8_t g_smem[];

__device__ __forceinline__ uint2 tab64(uint32_t off) {
  return *reinterpret_cast<const uint2*>(g_smem + off);
}
__device__ __forceinline__ uint32_t tab32(uint32_t off) {
  return *reinterpret_cast<const uint32_t*>(g_smem + off);
}
__device__ __forceinline__ uint4 tab128(uint32_t off) {
  return *reinterpret_cast<const uint4*>(g_smem + off);
}
// Table offset of the 8-bit code in byte i of w: byte 1 of the result is the
// code (the 256-byte row), byte 0 the lane's byte inside the row (lw < 256).
__device__ __forceinline__ uint32_t row_addr(uint32_t w, uint32_t lw, int i) {
  return __byte_perm(w, lw, 0x5504 | (i << 4));
}

// The same with 128-byte table rows (one tensor per table, the table-based
// methods): (code << 7) | lane byte.
__device__ __forceinline__ uint32_t row7_addr(uint32_t w, uint32_t lw, int i) {
  return (__byte_perm(w, 0u, 0x4440 | i) << 7) | lw;
}

// K codes of one token for the lane's 8 (dk = 4) or 16 (dk = 2) sub-vectors.
template <int DK>
struct KCodes;
template <>
struct KCodes<4> {
  uint2 w;
  __device__ __forceinline__ void load(const uint8_t* row, int c) {
    w = *reinterpret_cast<const uint2*>(row + 8 * c);
  }
  __device__ __forceinline__ uint32_t off(int i, uint32_t lw) const {
    return row_addr(i < 4 ? w.x : w.y, lw, i & 3);
  }
  __device__ __forceinline__ uint32_t off7(int i, uint32_t lw) const {
    return row7_addr(i < 4 ? w.x : w.y, lw, i & 3);
  }
  __device__ __forceinline__ uint32_t code(int i) const {  // code of sub-vector 8c + i
    return __byte_perm(i < 4 ? w.x : w.y, 0u, 0x4440 | (i & 3));
  }
};
template <>
struct KCodes<2> {
  uint4 w;
  __device__ __forceinline__ void load(const uint8_t* row, int c) {
    w = *reinterpret_cast<const uint4*>(row + 16 * c);
  }
  __device__ __forceinline__ uint32_t off(int i, uint32_t lw) const {
    const uint32_t v = i < 4 ? w.x : i < 8 ? w.y : i < 12 ? w.z : w.w;
    return row_addr(v, lw, i & 3);
  }
};

// V codes of one token for the lane's sub-vectors: dv = 4 -> sub-vectors
// 4r .. 4r+3 (8- or 9-bit codes), dv = 2 -> sub-vectors 8r .. 8r+7 (8-bit).
template <int DV, int BV>
struct VCodes;
template <>
struct VCodes<4, 8> {
  uint32_t w;
  __device__ __forceinline__ void load(const uint8_t* row, int r) {
    w = *reinterpret_cast<const uint32_t*>(row + 4 * r);
  }
  __device__ __forceinline__ uint32_t off(int i, uint32_t lw) const { return row_addr(w, lw, i); }
  __device__ __forceinline__ uint32_t off7(int i, uint32_t lw) const { return row7_addr(w, lw, i); }
};
template <>
struct VCodes<4, 9> {
  uint32_t a, b;  // the lane's 36-bit code group: bits 0..31 in a, 32..35 in b
  __device__ __forceinline__ void load(const uint8_t* row, int r) {
    // codes 4r .. 4r+3 sit at bits 36r .. 36r+35: words r and r+1, shift 4r
    const uint32_t lo = *reinterpret_cast<const uint32_t*>(row + 4 * r);
    const uint32_t hi = *reinterpret_cast<const uint32_t*>(row + 4 * r + 4);
    a = __funnelshift_r(lo, hi, 4 * r);
    b = hi >> (4 * r);
  }
  __device__ __forceinline__ uint32_t off(int i, uint32_t lw) const {
    // code i = group bits 9i .. 9i+8, moved to bits 8..16 (the table row)
    const uint32_t x = i == 0 ? a << 8 : i == 1 ? a >> 1 : i == 2 ? a >> 10 : __funnelshift_r(a, b, 19);
    return (x & 0x1ff00u) | lw;
  }
};
template <>
struct VCodes<2, 8> {
  uint2 w;
  __device__ __forceinline__ void load(const uint8_t* row, int r) {
    w = *reinterpret_cast<const uint2*>(row + 8 * r);
  }
  __device__ __forceinline__ uint32_t off(int i, uint32_t lw) const {
    return row_addr(i < 4 ? w.x : w.y, lw, i & 3);
  }
};

// d = 8, 12-bit codes (the pages' 1.5-bit configuration): the table is not
// replicated (two 64 KiB tables, K at 0 and V at 64 KiB, one 16-byte row of
// fp16 elements per code).  A lane reads a whole centroid with one 16-byte
// load, which serves two k-steps (K) or two output steps (V): a quarter-warp
// phase of 8 random rows meets fewer bank conflicts than the half-warp phase
// of two 8-byte loads.
__device__ __forceinline__ uint32_t row16(uint32_t code, uint32_t lw) { return (code << 4) | lw; }
template <>
struct KCodes<8> {
  uint32_t a, b;  // the lane's 48-bit code group (sub-vectors 4c .. 4c+3), from bit 0
  __device__ __forceinline__ void load(const uint8_t* row, int c) {
    // codes 4c .. 4c+3 sit at bits 48c .. 48c+47: words w0, w0+1, shift 0 or 16
    const uint32_t* rw = reinterpret_cast<const uint32_t*>(row);
    const int w0 = (48 * c) >> 5;
    const uint32_t lo = rw[w0], hi = rw[w0 + 1];
    const uint32_t sh = (48 * c) & 31;
    a = __funnelshift_r(lo, hi, sh);
    b = hi >> sh;
  }
  // sub-vector 4c + j (0..3): k-steps 2j (elements 0..3) and 2j + 1 (4..7)
  __device__ __forceinline__ uint32_t off16(int j, uint32_t lw) const {
    const uint32_t code = j == 0 ? (a & 0xfffu) : j == 1 ? ((a >> 12) & 0xfffu)
                        : j == 2 ? (__funnelshift_r(a, b, 24) & 0xfffu) : ((b >> 4) & 0xfffu);
    return row16(code, lw);
  }
};
template <>
struct VCodes<8, 12> {
  uint32_t x;  // the lane's 24-bit code pair (sub-vectors 2r, 2r+1), from bit 0
  __device__ __forceinline__ void load(const uint8_t* row, int r) {
    // codes 2r, 2r+1 sit at bits 24r .. 24r+23 of the 24-byte row; the next
    // word is needed only when they cross a word boundary (never for r = 7)
    const uint32_t* rw = reinterpret_cast<const uint32_t*>(row);
    const int w0 = (24 * r) >> 5;
    const uint32_t sh = (24 * r) & 31;
    const uint32_t lo = rw[w0];
    const uint32_t hi = sh > 8 ? rw[w0 + 1] : 0u;
    x = __funnelshift_r(lo, hi, sh);
  }
  // sub-vector 2r + m (m = 0, 1): output steps 2m (elements 0..3) and 2m + 1 (4..7)
  __device__ __forceinline__ uint32_t off16(int m, uint32_t lw) const {
    return row16(m ? ((x >> 12) & 0xfffu) : (x & 0xfffu), lw);
  }
};

}  // namespace
}  // namespace vqk

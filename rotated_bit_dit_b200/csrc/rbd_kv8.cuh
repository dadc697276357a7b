// Shared pieces of the 8-bit paged key/value cache: the view of a cache that
// kernels receive, the layout of a page, the code conversions and the mapping
// of a launch's items to sequences.
//
// A page holds 64 consecutive tokens of one sequence.  codes is
// [pages][heads][2][64][128] bytes (side 0 keys, side 1 values): one (page,
// head) is 16 KB of contiguous memory, one bulk copy.  Inside a [64][128] tile
// the eight 16-byte chunks of token row t are permuted, chunk c standing at
// c ^ (t & 7): the fragment reads of the single-token kernel (eight lanes, two
// chunks of four token rows or the same chunk of four) then touch all 32 banks
// once, with no copy between the bulk load and the registers.  scales is
// [pages][heads][2] float32; value = code * scale.
#pragma once

#include <atomic>

#include <cuda_fp16.h>

#include "rbd_common.cuh"

namespace rbd {

// First refusal of device-side metadata (a page index outside the pool, offsets
// or lengths outside their buffers) since the last rbd_check.  Kept apart from
// g_device_status, which makes bounded waits give up.
__device__ int g_device_refusal = 0;
__device__ __forceinline__ void record_refusal() { atomicCAS(&g_device_refusal, 0, RBD_ERR_INVALID_ARG); }

// Raises a kernel's dynamic shared memory limit once per device (a driver call each time costs a call of these
// sizes a microsecond).  Setting it twice, from two threads, does no harm.
struct SmemAllowance {
  std::atomic<uint64_t> done{0};
  template <class Kernel>
  cudaError_t raise(Kernel* kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
  }
};

constexpr int kKv8Page = 64;                       // tokens per page
constexpr int kKv8Dim = 128;                       // channels per head
constexpr int kKv8Side = kKv8Page * kKv8Dim;       // bytes of one side of a (page, head)
constexpr float kKv8Floor = 7.888609052210118e-31f;   // 2^-100: smallest scale

struct Kv8View {
  uint8_t* codes;
  float* scales;
  const int32_t* table;   // [seqs][ldt]
  int64_t ldt;
  int pages, heads, max_pages, seqs;
};

// Byte offset of (token t, channel chunk c of 16) inside a [64][128] tile.
__host__ __device__ __forceinline__ constexpr int kv8_chunk(int t, int c) { return t * kKv8Dim + ((c ^ (t & 7)) << 4); }

__device__ __forceinline__ int64_t kv8_tile(const Kv8View& c, int page, int head, int side) {
  return ((((int64_t)page * c.heads + head) * 2) + side) * kKv8Side;
}
__device__ __forceinline__ int64_t kv8_scale(const Kv8View& c, int page, int head, int side) {
  return ((int64_t)page * c.heads + head) * 2 + side;
}

// Page p of sequence b, or -1 (recorded) when the table names none of the pool.
__device__ __forceinline__ int kv8_page(const Kv8View& c, int b, int p) {
  const int page = __ldg(c.table + (int64_t)b * c.ldt + p);
  if (page >= 0 && page < c.pages) return page;
  record_refusal();
  return -1;
}

// Rows [cu[b], cu[b+1]) of a packed tensor of `rows` rows; false (recorded) when they lie outside it.
__device__ __forceinline__ bool kv8_rows(const int32_t* cu, int b, int rows, int& r0, int& n) {
  const int a = __ldg(cu + b), z = __ldg(cu + b + 1);
  r0 = a;
  n = z - a;
  if (a >= 0 && z >= a && z <= rows) return true;
  record_refusal();
  n = 0;
  return false;
}

// What a block works on: sequence b, the item's index among the sequence's, and the
// sequence's rows of the packed tensors and length.
struct Kv8Item {
  int b, idx, r0, n, len;
};

// The item x of a launch, when sequence b has count(n, len) items in a row.  Every warp of the block finds out by
// itself (32 sequences per step, an inclusive scan of their counts; what the lanes have read is passed on, not read
// again); all 32 lanes call.  A sequence whose rows lie outside the packed tensors (recorded) has none.
template <class Count>
__device__ __forceinline__ bool kv8_find(const int32_t* cu, const int32_t* lens, int seqs, int rows, int x, Count count,
                                         Kv8Item& it) {
  const int lane = threadIdx.x & 31;
  int base = 0;
  for (int b0 = 0; b0 < seqs; b0 += 32) {
    int r0 = 0, n = 0, len = 0, c = 0;
    if (b0 + lane < seqs) {
      len = __ldg(lens + b0 + lane);
      if (kv8_rows(cu, b0 + lane, rows, r0, n) && n > 0) c = count(n, len);
    }
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, c, off);
      if (lane >= off) c += up;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, x < base + c);
    if (hit) {
      const int l = __ffs(hit) - 1;
      const int before = __shfl_sync(0xffffffffu, c, l > 0 ? l - 1 : 0);
      it.b = b0 + l;
      it.idx = x - base - (l > 0 ? before : 0);
      it.r0 = __shfl_sync(0xffffffffu, r0, l);
      it.n = __shfl_sync(0xffffffffu, n, l);
      it.len = __shfl_sync(0xffffffffu, len, l);
      return true;
    }
    base += __shfl_sync(0xffffffffu, c, 31);
  }
  return false;
}

template <int FMT>
__host__ __device__ __forceinline__ constexpr float kv8_inv_qmax() {
  return FMT == RBD_CODES_INT8 ? 1.f / 127.f : 1.f / 448.f;
}

// Code bytes of four values x under the inverse scale inv.  RAW: infinities and NaN may be among them (stored as the
// largest code and as zero); without, |x| is at most the scale's own qmax s (1 + 2^-22), which rounds to the largest
// code by itself.  INT8 rounds by adding 1.5 * 2^23, whose low byte is then the two's complement code (the conversion
// instruction runs at an eighth of the rate).
template <int FMT, bool RAW>
__device__ __forceinline__ uint32_t kv8_encode4(const float (&x)[4], float inv) {
  float y[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    y[j] = __fmul_rn(x[j], inv);
    if (RAW) y[j] = y[j] == y[j] ? y[j] : 0.f;
    if (RAW && FMT == RBD_CODES_INT8) y[j] = fminf(fmaxf(y[j], -127.f), 127.f);
  }
  if (FMT == RBD_CODES_INT8) {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = __float_as_uint(__fadd_rn(y[j], 12582912.f));
    return prmt(prmt(u[0], u[1], 0x0040u), prmt(u[2], u[3], 0x0040u), 0x5410u);
  }
  uint32_t d;
  asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
      : "=r"(d)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]));
  return d;
}

// Four code bytes -> two fp16 pairs.  INT8: (b0, b2) and (b1, b3); the byte with its sign bit flipped, under the
// exponent of 1024, is 1024 + 128 + b, from which one subtraction leaves b exactly.  E4M3: (b0, b1) and (b2, b3),
// every E4M3 value being an fp16 value.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t d;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(d) : "r"(two));
  return d;
}
template <int FMT>
__device__ __forceinline__ void kv8_to_f16(uint32_t w, uint32_t& p0, uint32_t& p1) {
  if (FMT == RBD_CODES_INT8) {
    // (and, then xor: function 0x6A of one logic instruction; left to the compiler it came out as two, and the
    // streaming kernel's integer pipe did 40% more)
    asm("{\n\t.reg .b32 a, b, c;\n\tmov.b32 c, 0x64806480;\n\t"
        "lop3.b32 a, %2, 0x00FF00FF, c, 0x6A;\n\tshr.u32 b, %2, 8;\n\tlop3.b32 b, b, 0x00FF00FF, c, 0x6A;\n\t"
        "sub.f16x2 %0, a, c;\n\tsub.f16x2 %1, b, c;\n\t}"
        : "=r"(p0), "=r"(p1)
        : "r"(w));
  } else {
    p0 = e4m3x2_to_f16x2(w & 0xFFFFu);
    p1 = e4m3x2_to_f16x2(w >> 16);
  }
}
// Four codes as float32, in order.
template <int FMT>
__device__ __forceinline__ void kv8_decode4(uint32_t w, float (&v)[4]) {
  uint32_t p0, p1;
  kv8_to_f16<FMT>(FMT == RBD_CODES_INT8 ? prmt(w, 0u, 0x3120u) : w, p0, p1);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&p0));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&p1));
  v[0] = a.x;
  v[1] = a.y;
  v[2] = b.x;
  v[3] = b.y;
}

}  // namespace rbd

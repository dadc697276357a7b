// 8-bit paged key/value cache: append (quantise), read, and eviction by
// accumulated attention weight.  The attention over it is in rbd_kv8_attn.cu.
//
// Quantisation of a page, per head and side, over its 64 x 128 values:
//   s = max(s_old, RN(amax * RN(1 / qmax)), 2^-100),  inv = RN(1 / s),
//   code = round(RN(x * inv))  (to the nearest whole number in [-127, 127], or E4M3 value, ties to even)
// with qmax = 127 (INT8) or 448 (E4M3), amax over the finite values that join
// the page, and s_old the page's scale while it already holds tokens.  When the
// scale grows, the older codes are formed again from the values they stand for,
// which adds at most half a step of the new scale; among 64 tokens drawn alike a
// running maximum moves H(64) = 4.7 times on average, so a page filled token by
// token is requantised a handful of times, mostly while it is nearly empty.
// The floor 2^-100 keeps 1 / s and the logarithms the attention takes finite; an
// all-zero page then still lets later tokens set its scale.
#include <algorithm>

#include "rbd_kv8.cuh"
#include "rbd_internal.cuh"

namespace rbd {

namespace {

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
// The larger |bf16| bit patterns of a word's two halves and m's, half by half.
__device__ __forceinline__ uint32_t amax2(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7FFF7FFFu); }
// The same with infinities and NaN counted as zero.
__device__ __forceinline__ uint32_t finite_amax2(uint32_t m, uint32_t w) {
  const uint32_t a = w & 0x7FFF7FFFu;
  return __vmaxu2(m, ((a & 0xFFFFu) < 0x7F80u ? a & 0xFFFFu : 0u) | ((a >> 16) < 0x7F80u ? a & 0xFFFF0000u : 0u));
}

template <int FMT, bool RAW>
__device__ __forceinline__ uint32_t encode_bf16x4(uint32_t w0, uint32_t w1, float inv) {
  const float x[4] = {bf16_lo(w0), bf16_hi(w0), bf16_lo(w1), bf16_hi(w1)};
  return kv8_encode4<FMT, RAW>(x, inv);
}

// Codes of four stored codes under a new scale: the values they stand for, quantised again.
template <int FMT>
__device__ __forceinline__ uint32_t requantise4(uint32_t w, float s_old, float inv) {
  float v[4];
  kv8_decode4<FMT>(w, v);
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = __fmul_rn(v[j], s_old);
  return kv8_encode4<FMT, false>(v, inv);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}

}  // namespace

// One block per (touched page, head): threads 0-127 the keys, 128-255 the values.
// Thread l of a side takes 8 channels (16 bytes of bf16) of rows l / 16, l / 16 +
// 8, ...: the page's new values stay in registers between the maximum and the
// codes, so they are read once.  Bound by memory: 2 bytes in, 1 byte out a value
// (24002 tokens x 12 heads: 40 us, 5.5 TB/s).
// Heads are the fastest index of the blocks: those that run together then read whole
// rows of k and v, not 256 bytes of each.
template <int FMT>
__global__ void __launch_bounds__(256, 4)
    kv8_append_kernel(const Kv8View c, const int32_t* __restrict__ lens, const int32_t* __restrict__ cu,
                      const uint16_t* __restrict__ k, int64_t ldk, const uint16_t* __restrict__ v, int64_t ldv,
                      int rows) {
  __shared__ uint32_t red[2][4];
  auto pages_of = [&](int n, int len) {
    if (len < 0 || (int64_t)len + n > (int64_t)c.max_pages * kKv8Page) {
      record_refusal();
      return 0;
    }
    return (len + n - 1) / kKv8Page - len / kKv8Page + 1;
  };
  Kv8Item it;
  if (!kv8_find(cu, lens, c.seqs, rows, blockIdx.x / c.heads, pages_of, it)) return;
  const int head = blockIdx.x % c.heads, b = it.b, idx = it.idx, len = it.len, r0 = it.r0, n = it.n;
  const int p = len / kKv8Page + idx;
  const int held = max(0, len - p * kKv8Page);                       // rows that already hold tokens
  const int end = min(kKv8Page, len + n - p * kKv8Page);             // rows held afterwards
  const int side = threadIdx.x >> 7, tid = threadIdx.x & 127;
  const uint16_t* src = side ? v : k;
  const int64_t ld = side ? ldv : ldk;
  const int chunk8 = tid & 15, row0 = tid >> 4;
  const int64_t first = (int64_t)r0 + (int64_t)p * kKv8Page - len;   // packed row of the page's row 0

  uint4 raw[8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int t = row0 + 8 * i;
    raw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (t >= held && t < end)
      raw[i] = __ldg(reinterpret_cast<const uint4*>(src + (first + t) * ld + head * kKv8Dim + 8 * chunk8));
    m = amax2(amax2(amax2(amax2(m, raw[i].x), raw[i].y), raw[i].z), raw[i].w);
  }
  const int page = kv8_page(c, b, p);            // (after the loads above: none waits for it)
  if (page < 0) return;
  float* scale = c.scales + kv8_scale(c, page, head, side);
  const float s_old = held > 0 ? *scale : kKv8Floor;
  auto block_max = [&](uint32_t v) {            // of either side, into red
    v = __reduce_max_sync(0xffffffffu, max(v & 0xFFFFu, v >> 16));
    if ((tid & 31) == 0) red[side][tid >> 5] = v;
    __syncthreads();
  };
  auto side_max = [&](int sd) { return max(max(red[sd][0], red[sd][1]), max(red[sd][2], red[sd][3])); };
  block_max(m);
  m = side_max(side);
  const bool clean = max(m, side_max(side ^ 1)) < 0x7F80u;
  if (!clean) {                                 // an infinity or NaN among the block's values: again, without them
    m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      m = finite_amax2(finite_amax2(finite_amax2(finite_amax2(m, raw[i].x), raw[i].y), raw[i].z), raw[i].w);
    __syncthreads();
    block_max(m);
    m = side_max(side);
  }
  const float amax = __uint_as_float(m << 16);
  const float s = fmaxf(fmaxf(s_old, __fmul_rn(amax, kv8_inv_qmax<FMT>())), kKv8Floor);
  const float inv = __frcp_rn(s);
  uint8_t* tile = c.codes + kv8_tile(c, page, head, side);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int t = row0 + 8 * i;
    uint2* dst = reinterpret_cast<uint2*>(tile + kv8_chunk(t, chunk8 >> 1) + 8 * (chunk8 & 1));
    if (t >= held && t < end) {
      *dst = clean ? make_uint2(encode_bf16x4<FMT, false>(raw[i].x, raw[i].y, inv),
                                encode_bf16x4<FMT, false>(raw[i].z, raw[i].w, inv))
                   : make_uint2(encode_bf16x4<FMT, true>(raw[i].x, raw[i].y, inv),
                                encode_bf16x4<FMT, true>(raw[i].z, raw[i].w, inv));
    } else if (t < held && s > s_old) {
      const uint2 w = *dst;
      *dst = make_uint2(requantise4<FMT>(w.x, s_old, inv), requantise4<FMT>(w.y, s_old, inv));
    }
  }
  if (tid == 0) *scale = s;
}

// The last `tokens` tokens of every sequence as bf16 rows [seqs * tokens].  A block
// takes 16 rows and up to 4 heads, a thread one side's 16-channel chunk of a row in
// each head: pages are read 2 KB at a time, all four loads in flight.  Bound by
// memory: 1 byte in, 2 out (16 x 4096 rows x 12 heads: 109 us, 5.4 TB/s).
constexpr int kRdRows = 16, kRdHeads = 4;
template <int FMT>
__global__ void __launch_bounds__(256)
    kv8_read_kernel(const Kv8View c, const int32_t* __restrict__ lens, int tokens, uint16_t* __restrict__ k,
                    int64_t ldk, uint16_t* __restrict__ v, int64_t ldv) {
  const int chunk = threadIdx.x & 7, side = (threadIdx.x >> 3) & 1;
  const int groups = (c.heads + kRdHeads - 1) / kRdHeads;
  const int head0 = (int)(blockIdx.x % groups) * kRdHeads;
  const int64_t block = blockIdx.x / groups;
  const int per = (tokens + kRdRows - 1) / kRdRows;
  const int b = (int)(block / per);
  const int i = (int)(block - (int64_t)b * per) * kRdRows + (threadIdx.x >> 4);
  if (i >= tokens) return;
  const int len = __ldg(lens + b);
  const int64_t t = (int64_t)len - tokens + i;
  int page = -1;
  if (len < 0 || len > c.max_pages * kKv8Page) record_refusal();
  else if (t >= 0) page = kv8_page(c, b, (int)(t / kKv8Page));
  uint4 w[kRdHeads];
  float s[kRdHeads];
#pragma unroll
  for (int h = 0; h < kRdHeads; ++h) {
    w[h] = make_uint4(0u, 0u, 0u, 0u);
    s[h] = 0.f;
    if (page >= 0 && head0 + h < c.heads) {
      w[h] = *reinterpret_cast<const uint4*>(c.codes + kv8_tile(c, page, head0 + h, side) +
                                             kv8_chunk((int)(t % kKv8Page), chunk));
      s[h] = c.scales[kv8_scale(c, page, head0 + h, side)];
    }
  }
  const int64_t row = (int64_t)b * tokens + i;
  uint16_t* dst = (side ? v + row * ldv : k + row * ldk) + 16 * chunk;
#pragma unroll
  for (int h = 0; h < kRdHeads; ++h) {
    if (head0 + h >= c.heads) break;
    const uint32_t ws[4] = {w[h].x, w[h].y, w[h].z, w[h].w};
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float x[4];
      kv8_decode4<FMT>(ws[j], x);
      o[2 * j] = pack_bf16(__fmul_rn(x[0], s[h]), __fmul_rn(x[1], s[h]));
      o[2 * j + 1] = pack_bf16(__fmul_rn(x[2], s[h]), __fmul_rn(x[3], s[h]));
    }
    uint4* out = reinterpret_cast<uint4*>(dst + (head0 + h) * kKv8Dim);
    out[0] = make_uint4(o[0], o[1], o[2], o[3]);
    out[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

// ---------------------------------------------------------------------------
// Eviction
// ---------------------------------------------------------------------------
// Selection, one block of 1024 threads per (sequence, head): the last `recent`
// tokens stay, and of the others the `keep - recent` of largest weight, equal
// weights by the lowest position.  The weights become unsigned keys of the same
// order, held in shared memory as far as they fit; three histogram passes (11, 11
// and 10 bits from the top) find the key of the last one to stay and how many of
// its equals stay with it; then every warp counts and emits its own run of
// positions, so the kept ones come out in ascending order with no atomics on the
// output and no dependence on timing.  Bound by its instructions (68% of the issue slots;
// 192 blocks of 32 warps, one or two an SM): 16 x 12 blocks over up to 16384 positions
// take 27 us.
constexpr int kSelThreads = 1024;
constexpr int kSelBins = 2048;
constexpr int kSelMaxKeys = 48 * 1024;    // 192 KB of keys; positions beyond are read from global memory

struct Kv8EvictArgs {
  const float* weights;                    // [seqs][heads][width]
  int64_t w_seq, w_head;
  int width;
  float* weights_out;                      // [seqs][heads][width_out], may be `weights`
  int64_t o_seq, o_head;
  int width_out;
  const int32_t* lens;
  int32_t* lens_out;
  int32_t* kept;                           // [seqs][heads][keep]
  int keep, recent;
};

__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0u;                                    // a NaN is the first to go
  const uint32_t u = __float_as_uint(w + 0.0f);             // -0 as +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kSelThreads) kv8_select_kernel(const Kv8View c, const Kv8EvictArgs a, int cap) {
  extern __shared__ uint32_t dyn[];
  uint32_t* hist = dyn;                     // [kSelBins]
  uint32_t* keys = dyn + kSelBins;          // [cap]
  __shared__ uint32_t warp_sum[32], warp_eq[32];
  __shared__ uint32_t sh_bin, sh_above;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.y, head = blockIdx.x;
  // sum of the warps' values in front of this warp's
  auto sum_before = [&](const uint32_t* v) { return __reduce_add_sync(0xffffffffu, lane < warp ? v[lane] : 0u); };
  int n = __ldg(a.lens + b);
  if (n < 0 || n > a.width || n > c.max_pages * kKv8Page) {
    if (tid == 0) record_refusal();
    n = 0;
  }
  const float* w = a.weights + b * a.w_seq + head * a.w_head;
  int32_t* kept = a.kept + ((int64_t)b * c.heads + head) * a.keep;
  const int m = min(n, a.keep);
  if (n <= a.keep) {
    for (int j = tid; j < a.keep; j += kSelThreads) kept[j] = j < n ? j : -1;
  } else {
    const int cand = n - a.recent;          // positions that compete
    int want = a.keep - a.recent;           // how many of them stay
    for (int j = tid; j < a.recent; j += kSelThreads) kept[want + j] = cand + j;
    const int cached = min(cand, cap);
    for (int i0 = tid; i0 < cached; i0 += 8 * kSelThreads) {        // eight loads in flight
      float x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) x[u] = i0 + u * kSelThreads < cached ? __ldg(w + i0 + u * kSelThreads) : 0.f;
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (i0 + u * kSelThreads < cached) keys[i0 + u * kSelThreads] = order_key(x[u]);
    }
    auto key = [&](int i) { return i < cap ? keys[i] : order_key(__ldg(w + i)); };
    uint32_t prefix = 0, mask = 0;
    uint32_t eq_want = (uint32_t)want;      // of the keys under the prefix, how many stay
    if (want > 0) {
      const int shifts[3] = {21, 10, 0}, bits[3] = {11, 11, 10};
#pragma unroll
      for (int pass = 0; pass < 3; ++pass) {
        for (int i = tid; i < kSelBins; i += kSelThreads) hist[i] = 0;
        __syncthreads();
        const uint32_t bin_mask = (1u << bits[pass]) - 1u;
        for (int i = tid; i < cand; i += kSelThreads) {
          const uint32_t u = key(i);
          if ((u & mask) == prefix) atomicAdd(&hist[(u >> shifts[pass]) & bin_mask], 1u);
        }
        __syncthreads();
        // bins from the top: thread t holds bins 2047 - 2t and 2046 - 2t
        const uint32_t h0 = hist[kSelBins - 1 - 2 * tid], h1 = hist[kSelBins - 2 - 2 * tid];
        uint32_t incl = h0 + h1;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const uint32_t up = __shfl_up_sync(0xffffffffu, incl, off);
          if (lane >= off) incl += up;
        }
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
        const uint32_t excl = sum_before(warp_sum) + incl - (h0 + h1);
        if (excl < eq_want && eq_want <= excl + h0 + h1) {
          const bool second = eq_want > excl + h0;
          sh_bin = (uint32_t)(kSelBins - 1 - 2 * tid - (second ? 1 : 0));
          sh_above = excl + (second ? h0 : 0u);
        }
        __syncthreads();
        prefix |= sh_bin << shifts[pass];
        mask |= bin_mask << shifts[pass];
        eq_want -= sh_above;
        __syncthreads();
      }
      // every warp takes a run of positions (a multiple of 32): counts, then the positions themselves
      const int run = ((cand + 31) / 32 + 31) / 32 * 32;
      const int i0 = warp * run, i1 = min(cand, i0 + run);
      uint32_t gt = 0, eq = 0;
      for (int i = i0; i < i1; i += 32) {
        const uint32_t u = i + lane < i1 ? key(i + lane) : 0u;
        gt += __popc(__ballot_sync(0xffffffffu, i + lane < i1 && u > prefix));
        eq += __popc(__ballot_sync(0xffffffffu, i + lane < i1 && u == prefix));
      }
      if (lane == 0) {
        warp_sum[warp] = gt;
        warp_eq[warp] = eq;
      }
      __syncthreads();
      uint32_t at_gt = sum_before(warp_sum), at_eq = sum_before(warp_eq);
      const uint32_t below = (1u << lane) - 1u;
      for (int i = i0; i < i1; i += 32) {
        const uint32_t u = i + lane < i1 ? key(i + lane) : 0u;
        const uint32_t bg = __ballot_sync(0xffffffffu, i + lane < i1 && u > prefix);
        const uint32_t be = __ballot_sync(0xffffffffu, i + lane < i1 && u == prefix);
        const uint32_t my_eq = at_eq + __popc(be & below);       // equals in front of this position
        const uint32_t pos = at_gt + __popc(bg & below) + min(my_eq, eq_want);
        if (i + lane < i1 && (u > prefix || (u == prefix && my_eq < eq_want))) kept[pos] = i + lane;
        at_gt += __popc(bg);
        at_eq += __popc(be);
      }
    }
  }
  __syncthreads();
  // weights of the kept tokens, ascending; safe in place, since position j never comes from below j and a
  // chunk is read before it is written
  float* wo = a.weights_out + b * a.o_seq + head * a.o_head;
  for (int j0 = tid; j0 - tid < m; j0 += 4 * kSelThreads) {
    float x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) x[u] = j0 + u * kSelThreads < m ? w[kept[j0 + u * kSelThreads]] : 0.f;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (j0 + u * kSelThreads < m) wo[j0 + u * kSelThreads] = x[u];
    __syncthreads();
  }
  for (int j = m + tid; j < a.width_out; j += kSelThreads) wo[j] = 0.f;
  if (head == 0 && tid == 0) a.lens_out[b] = m;
}

// The kept tokens into fresh pages, one block per (page, head, sequence): threads
// 0-127 the keys, 128-255 the values, 16 channels of 4 rows each, read once and
// kept in registers between the maximum and the new codes.  Bound by scattered 128-byte
// reads: a quarter of the tokens kept, 16 x 12 x up to 4096, in 87 us, 4.2 TB/s.
template <int FMT>
__global__ void __launch_bounds__(256, 4)
    kv8_gather_kernel(const Kv8View c, const int32_t* __restrict__ dst_table, int64_t ld_dst,
                      const int32_t* __restrict__ kept, int keep) {
  __shared__ uint32_t red[2][4];
  __shared__ int64_t row_at[kKv8Page];          // byte of the kept token's row of keys, -1 without a token, -2 without a page
  __shared__ float2 row_scale[kKv8Page];
  const int b = blockIdx.z, head = blockIdx.y, p = blockIdx.x;
  const int dst_page = __ldg(dst_table + b * ld_dst + p);
  // (kept is -1 behind the last token: how many there are need not be waited for)
  if (threadIdx.x < kKv8Page) {
    const int j = p * kKv8Page + threadIdx.x;
    const int src = j < keep ? __ldg(kept + ((int64_t)b * c.heads + head) * keep + j) : -1;
    int64_t at = -1;
    float2 sc = make_float2(0.f, 0.f);
    if (src >= 0) {
      const int page = kv8_page(c, b, src / kKv8Page);
      at = page >= 0 ? kv8_tile(c, page, head, 0) + src % kKv8Page * kKv8Dim : -2;
      if (page >= 0) sc = *reinterpret_cast<const float2*>(c.scales + kv8_scale(c, page, head, 0));
    }
    row_at[threadIdx.x] = at;
    row_scale[threadIdx.x] = sc;
  }
  __syncthreads();
  if (row_at[0] == -1) return;
  if (dst_page < 0 || dst_page >= c.pages) {
    if (threadIdx.x == 0) record_refusal();
    return;
  }
  const int side = threadIdx.x >> 7, tid = threadIdx.x & 127;
  const int chunk = tid & 7, row0 = tid >> 3;
  uint4 raw[4];
  float s_src[4];
  float am = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t at = row_at[row0 + 16 * i];
    raw[i] = make_uint4(0u, 0u, 0u, 0u);
    // (a row's chunks are permuted by its token's last three bits, which are the row address's bits 7 to 9)
    if (at >= 0)
      raw[i] = *reinterpret_cast<const uint4*>(c.codes + at + side * kKv8Side + ((chunk ^ ((int)(at >> 7) & 7)) << 4));
    const float2 sc = row_scale[row0 + 16 * i];
    s_src[i] = side ? sc.y : sc.x;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t ws[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
    float top;                                                  // largest |code| of the sixteen
    if (FMT == RBD_CODES_INT8) {
      __half2 t = __float2half2_rn(0.f);                        // codes are exact in fp16
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t p0, p1;
        kv8_to_f16<FMT>(ws[j], p0, p1);
        t = __hmax2(t, __hmax2(__habs2(*reinterpret_cast<__half2*>(&p0)), __habs2(*reinterpret_cast<__half2*>(&p1))));
      }
      const float2 t2 = __half22float2(t);
      top = fmaxf(t2.x, t2.y);
    } else {
      uint32_t t = 0;                                           // E4M3 magnitudes order like their bytes
#pragma unroll
      for (int j = 0; j < 4; ++j)
        t = __vmaxu2(t, __vmaxu2(ws[j] & 0x007F007Fu, (ws[j] >> 8) & 0x007F007Fu));
      float v[4];
      kv8_decode4<FMT>(max(t & 0xFFu, t >> 16), v);
      top = v[0];
    }
    am = fmaxf(am, __fmul_rn(top, s_src[i]));
  }
  const uint32_t m_bits = __reduce_max_sync(0xffffffffu, __float_as_uint(am));
  if ((tid & 31) == 0) red[side][tid >> 5] = m_bits;
  __syncthreads();
  am = __uint_as_float(max(max(red[side][0], red[side][1]), max(red[side][2], red[side][3])));
  const float s = fmaxf(__fmul_rn(am, kv8_inv_qmax<FMT>()), kKv8Floor);
  const float inv = __frcp_rn(s);
  uint8_t* tile = c.codes + kv8_tile(c, dst_page, head, side);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = row0 + 16 * i;
    if (row_at[t] != -1)
      *reinterpret_cast<uint4*>(tile + kv8_chunk(t, chunk)) =
          make_uint4(requantise4<FMT>(raw[i].x, s_src[i], inv), requantise4<FMT>(raw[i].y, s_src[i], inv),
                     requantise4<FMT>(raw[i].z, s_src[i], inv), requantise4<FMT>(raw[i].w, s_src[i], inv));
  }
  if (tid == 0) c.scales[kv8_scale(c, dst_page, head, side)] = s;
}

// ---------------------------------------------------------------------------
// Host launchers
// ---------------------------------------------------------------------------
cudaError_t launch_kv8_append(const Kv8View& c, bool e4m3, const int32_t* lens, const int32_t* cu, const uint16_t* k,
                              int64_t ldk, const uint16_t* v, int64_t ldv, int rows, cudaStream_t st) {
  // n tokens touch at most (n - 1) / 64 + 2 pages; never more than one page a token
  const int64_t items = std::min<int64_t>(rows, (int64_t)rows / kKv8Page + 2 * (int64_t)std::min(c.seqs, rows));
  const unsigned grid = (unsigned)(items * c.heads);
  if (e4m3) kv8_append_kernel<RBD_CODES_E4M3><<<grid, 256, 0, st>>>(c, lens, cu, k, ldk, v, ldv, rows);
  else kv8_append_kernel<RBD_CODES_INT8><<<grid, 256, 0, st>>>(c, lens, cu, k, ldk, v, ldv, rows);
  return cudaGetLastError();
}

cudaError_t launch_kv8_read(const Kv8View& c, bool e4m3, const int32_t* lens, int tokens, uint16_t* k, int64_t ldk,
                            uint16_t* v, int64_t ldv, cudaStream_t st) {
  const unsigned grid = (unsigned)((int64_t)c.seqs * ((tokens + kRdRows - 1) / kRdRows) *
                                   ((c.heads + kRdHeads - 1) / kRdHeads));
  if (e4m3) kv8_read_kernel<RBD_CODES_E4M3><<<grid, 256, 0, st>>>(c, lens, tokens, k, ldk, v, ldv);
  else kv8_read_kernel<RBD_CODES_INT8><<<grid, 256, 0, st>>>(c, lens, tokens, k, ldk, v, ldv);
  return cudaGetLastError();
}

cudaError_t launch_kv8_evict(const Kv8View& c, bool e4m3, const float* weights, int64_t w_seq, int64_t w_head,
                             int width, float* weights_out, int64_t o_seq, int64_t o_head, int width_out,
                             const int32_t* lens, int32_t* lens_out, int32_t* kept, int keep, int recent,
                             const int32_t* dst_table, int64_t ld_dst, cudaStream_t st) {
  const Kv8EvictArgs a{weights, w_seq, w_head, width, weights_out, o_seq, o_head, width_out,
                       lens,    lens_out, kept, keep,  recent};
  const int cap = std::min(std::min(width, c.max_pages * kKv8Page), kSelMaxKeys);
  const int smem = (kSelBins + cap) * 4;
  static SmemAllowance allowed;
  const cudaError_t e = allowed.raise(kv8_select_kernel, (kSelBins + kSelMaxKeys) * 4);
  if (e != cudaSuccess) return e;
  kv8_select_kernel<<<dim3(c.heads, c.seqs), kSelThreads, smem, st>>>(c, a, cap);
  const dim3 grid((keep + kKv8Page - 1) / kKv8Page, c.heads, c.seqs);
  if (e4m3) kv8_gather_kernel<RBD_CODES_E4M3><<<grid, 256, 0, st>>>(c, dst_table, ld_dst, kept, keep);
  else kv8_gather_kernel<RBD_CODES_INT8><<<grid, 256, 0, st>>>(c, dst_table, ld_dst, kept, keep);
  return cudaGetLastError();
}

}  // namespace rbd

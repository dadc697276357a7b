// Attention over the 8-bit paged cache (rbd_kv8.cuh): softmax(q k^T * scale) v per
// query head, grouped heads, causal or full, ragged batches, and the running sum
// of every key's attention weight.
//
// Keys and values are codes times a scale per (page, head, side).  INT8 and E4M3
// codes are exact in fp16; a query row is scaled by the power of two that brings
// its largest element to [2^14, 2^15), which makes its bf16 elements exact in fp16
// down to 2^-32 of that element (below, the rounding is 2^-40 of it).  So Q.K^T
// runs on fp16 operands with exact products and float32 sums, and the page scale
// multiplies whole 64-key blocks of scores.
// The value scale joins the exponent: with the score x_t (base 2) and the value
// scale s_v of key t's page,
//     e_t = x_t + log2 s_v,   m = running max of e_t,   p_t = 2^(e_t - m) in [0, 1],
//     O = sum p_t code_t,     L = sum over pages of (sum p_t) / s_v,   o = O / L,
// because 2^(x_t) code_t s_v = 2^(e_t) code_t and 2^(x_t) = 2^(e_t) / s_v.  The
// multiplication by s_v costs nothing per element, and p stays in fp16's best
// range whatever the pages' scales (up to 2^126 between them: a p below joins neither
// sum).  p is rounded to fp16 for the second product (a random half step of 2^-11
// each, and of 2^-24 below 2^-14); m, L, O and the scores are float32.
// The maximum moves only when a row exceeds it by 2^8 (p <= 256 then), which
// leaves most rescales of O out.
//
// Two kernels do the work, chosen by the rows (query tokens x heads of a group)
// that share a key/value head:
//   kv8_stream_kernel  up to kStreamRows a sequence on average: bound by reading
//                      the cache once.  Warps stream pages from memory.
//   kv8_tile_kernel    more: bound by the tensor cores (tcgen05).
// Both split the keys over several blocks when there are few items and write
// float32 partial results, which kv8_combine_kernel and kv8_tile_combine_kernel join.
#include <algorithm>

#include "rbd_kv8.cuh"
#include "rbd_internal.cuh"

namespace rbd {

struct Kv8AttnArgs {
  const uint16_t* q;
  int64_t ldq;
  uint16_t* o;
  int64_t ldo;
  const int32_t* cu;
  const int32_t* lens;
  int rows, q_heads, group, causal, max_len, nsplit, items, seqs;
  float scale_log2;
  int whole;           // tile kernel: (head, item) pairs in front whose keys are not split
  float* part_o;       // [slots][nsplit][128]: O of a split (null with one split); a slot is a (query token, head) in
                       // the streaming kernel, a row of a split (head, item) in the tile kernel
  float2* part_ml;     // [slots][nsplit]: (m, L)
  float2* stats;       // [rows * q_heads]: (m, 1 / L) of the whole row, or null
  float* logits;       // [rows * q_heads][logit_ld]: base-2 scores (stream kernel), or null
  int64_t logit_ld;
  uint8_t* q_image;    // [heads][items][2][32 KB]: the fp16 query tiles (tile kernel), or null
  float* q_rows;       // [heads][items][2][3][128]: score factor, softmax constant and keys seen of every row of them
  uint8_t* kv_image;   // [seqs][image_steps][heads][2][32 KB]: fp16 operands of every 128-key step, or null
  float4* kv_scale;    // [seqs][image_steps][heads][2]: their page scales (s_k, log2 s_v, 1 / s_v, least maximum)
  int image_steps;
};

namespace {

constexpr float kKv8Lazy = 8.0f;
// Largest magnitude of a row's maximum m.  A score enters as one fused x - m, with x unrounded and m rounded, so that
// the largest p is 2^8 at most but for the roundings of m and of log2 s_v - m: below 2^26 they are 2 and 4 at most, and
// p stays under fp16's 2^16.  A running maximum is not taken lower (p = 0 then, until a score says otherwise).
constexpr float kKv8Far = 67108864.0f;
// 1 / L of a row: 0 where it saw no key, NaN where its maximum lies beyond kKv8Far.
__device__ __forceinline__ float kv8_inverse(float m, float l) {
  if (m > -INFINITY && !(fabsf(m) < kKv8Far)) return __int_as_float(0x7FFFFFFF);
  return l == 0.f ? 0.f : 1.0f / l;
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// The power of two that brings a row whose largest |bf16| has bits `amax` to [2^14, 2^15), and its inverse.  A row
// with an infinite or NaN element has scores that are infinite or NaN, and by the definition a softmax of NaN: a NaN
// inverse, a factor of every score, says so (infinite scores by themselves vanish against an infinite maximum).
__device__ __forceinline__ void kv8_row_scale(uint32_t amax, float& f, float& inv) {
  const int e = (int)(amax >> 7);
  const int field = min(268 - e, 253);
  f = __uint_as_float((uint32_t)field << 23);
  inv = __uint_as_float(e == 255 ? 0x7FFFFFFFu : (uint32_t)(254 - field) << 23);
}

// A sequence's length, or 0 (recorded) when it exceeds what the call declared.
__device__ __forceinline__ int kv8_length(const Kv8View& c, const Kv8AttnArgs& a, int len) {
  if (len >= 0 && len <= a.max_len && len <= c.max_pages * kKv8Page) return len;
  record_refusal();
  return 0;
}
__device__ __forceinline__ int kv8_len(const Kv8View& c, const Kv8AttnArgs& a, int b) {
  return kv8_length(c, a, __ldg(a.lens + b));
}

// Keys query token i of n sees.
__device__ __forceinline__ int kv8_visible(int causal, int len, int n, int i) {
  return causal ? max(0, len - n + i + 1) : len;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

}  // namespace

// ---------------------------------------------------------------------------
// Few rows: warps stream pages
// ---------------------------------------------------------------------------
// A block takes 8 NQ rows of one (sequence, key/value head) and a run of its pages.
// Its warps take pages in turn, each with a buffer for a page's keys and one for its
// values (8 KB bulk copies, the next page's keys on their way as soon as the scores
// are formed), its own running maximum and its own O, and are joined through shared
// memory at the end: no warp waits for another in the loop.  The products are
// mma.sync m16n8k16 with keys (then channels) as the 16 and queries as the 8: a
// single token of a grouped head fills an 8 half or whole, where a 128-row tcgen05
// tile would be 1/32 full.  Fragments come straight from the bulk-copied bytes, since
// the order of a contraction is free:
//   scores^T = K Q^T   lane (g, l) holds channels 32 l .. 32 l + 31 of keys g and g + 8
//                      of every 16; the query fragments use the same order;
//   out^T = V^T P^T    lane (g, l) holds channels 16 g .. 16 g + 15 of keys 2 l, 2 l + 1,
//                      2 l + 8, 2 l + 9 of every 16: row g of product j is channel
//                      16 g + 2 j, row g + 8 the next; P^T is the transposed scores'
//                      fragment (one 8 x 8 transpose for 8 keys).
// What bounds it is reading the cache once, and close behind a warp's own time for a
// page (1260 instructions, 700 of them conversions, at three warps a scheduler), so
// what else a page needs (its index, the logarithm and inverse of its scale) is
// worked out 32 pages at a time, one a lane.  64 sequences of up to 8192 keys (292317
// in all), 12 heads, 4 query heads each: 167 us, 5.4 TB/s (when it took 174: without
// the products 158, without the loads 139).  24 sequences of up to 3000 keys, 8 heads, 1
// to 6 tokens of 5 query heads each: 47 us, of which reading takes 14; a block there
// has about four pages a warp, and the device less than two blocks an SM.
constexpr uint32_t kStPage = 2 * kKv8Side;                           // 16 KB: a warp's two buffers
constexpr int kStORow = kKv8Dim + 4;                                 // padded row of a warp's O in shared memory

template <int NQ>
struct StreamShape {
  // 16 rows want the registers of 8 warps: 12 spill (54 us against 51 for the 24 sequences above), and with the query
  // fragments read from shared memory for every page instead gain nothing (51)
  static constexpr int kWarps = NQ == 1 ? 12 : 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kRows = 8 * NQ;
  static constexpr uint32_t kRing = kWarps * kStPage;
  static constexpr uint32_t kSmem = kRing + 256 + (2 * kWarps * kRows + 2 * kRows) * 4 + 128;
  static_assert(kStPage >= kRows * kStORow * 4, "a warp's O fits its buffers");
};

// Transposes the 8 x 8 matrix of 16-bit values whose row g the lanes 4 g .. 4 g + 3 hold in pairs.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// Maximum and sum over the lanes that share l (the 8 values of g).
__device__ __forceinline__ float col_max(float x) {
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
  return x;
}
__device__ __forceinline__ float col_sum(float x) {
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

template <int FMT, int NQ>
__global__ void __launch_bounds__(StreamShape<NQ>::kThreads, 1) kv8_stream_kernel(const Kv8View c, const Kv8AttnArgs a) {
  using Sh = StreamShape<NQ>;
  constexpr int W = Sh::kWarps, ROWS = Sh::kRows;
  extern __shared__ unsigned char smem_dyn[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_dyn) + 127u) & ~uintptr_t(127u));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Sh::kRing);
  float* red_m = reinterpret_cast<float*>(smem + Sh::kRing + 256);   // [warps][rows]
  float* red_l = red_m + W * ROWS;                                   // [warps][rows]
  float* row_l = red_l + W * ROWS;                                   // [rows]
  float* row_m = row_l + ROWS;                                       // [rows]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, l = lane & 3;
  const int head = blockIdx.y, split = blockIdx.z;

  Kv8Item it;
  if (!kv8_find(a.cu, a.lens, c.seqs, a.rows, blockIdx.x,
                [&](int n, int) { return (int)(((int64_t)n * a.group + ROWS - 1) / ROWS); }, it))
    return;
  const int b = it.b, tile = it.idx, r0 = it.r0, n = it.n;
  const int len = kv8_length(c, a, it.len);
  const int row_first = tile * ROWS;
  const int nrows = min(ROWS, n * a.group - row_first);
  const int vis = min(len, kv8_visible(a.causal, len, n, (row_first + nrows - 1) / a.group));
  // this split's run of pages: the same number for every sequence, so that blocks take equally long
  const int per = ((a.max_len + kKv8Page - 1) / kKv8Page + a.nsplit - 1) / a.nsplit;
  const int p0 = min(split * per, (vis + kKv8Page - 1) / kKv8Page);
  const int p1 = min(p0 + per, (vis + kKv8Page - 1) / kKv8Page);
  const int cnt = p1 - p0 > warp ? (p1 - p0 - warp + W - 1) / W : 0;

  // The loads a block starts with depend on one another (offsets, page, codes): what does not is asked for first.
  uint4 qw[NQ][4];                                     // row g of every 8, channels 32 l .. 32 l + 31
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    const int r = row_first + 8 * q + g;
#pragma unroll
    for (int i = 0; i < 4; ++i) qw[q][i] = make_uint4(0u, 0u, 0u, 0u);
    if (8 * q + g < nrows) {
      const uint4* src = reinterpret_cast<const uint4*>(a.q + (int64_t)(r0 + r / a.group) * a.ldq +
                                                        (int64_t)(head * a.group + r % a.group) * kKv8Dim + 32 * l);
#pragma unroll
      for (int i = 0; i < 4; ++i) qw[q][i] = __ldg(src + i);
    }
  }
  uint64_t* full = bars + 2 * warp;                                  // keys, values
  if (lane == 0) {
    mbar_init(&full[0], 1);
    mbar_init(&full[1], 1);
    fence_barrier_init();
  }
  __syncwarp();
  unsigned char* ring = smem + warp * kStPage;
  // 32 of the warp's pages at a time: lane i knows page i, its scales, log2 s_v and 1 / s_v
  int my_page = -1;
  float my_sk = 1.f, my_lsv = 0.f, my_inv = 1.f;
  auto look_up = [&](int i0) { my_page = i0 + lane < cnt ? kv8_page(c, b, p0 + warp + (i0 + lane) * W) : -1; };
  auto look_up_scales = [&]() {
    if (my_page >= 0) {
      const float2 sc = *reinterpret_cast<const float2*>(c.scales + kv8_scale(c, my_page, head, 0));
      my_sk = sc.x;
      my_lsv = log2f(sc.y);
      my_inv = 1.0f / sc.y;
    }
  };
  auto issue = [&](int side, int page) {       // an index outside the pool: the buffer's old contents, skipped below
    if (lane != 0) return;
    if (page >= 0) {
      mbar_arrive_expect_tx(&full[side], kKv8Side);
      bulk_load(ring + side * kKv8Side, c.codes + kv8_tile(c, page, head, side), kKv8Side, &full[side]);
    } else {
      mbar_arrive(&full[side]);
    }
  };
  look_up(0);
  int page = __shfl_sync(0xffffffffu, my_page, 0);
  if (cnt > 0) {
    issue(0, page);
    issue(1, page);
  }
  look_up_scales();

  // query fragments
  uint32_t qb[NQ][8][2];
  float coef[NQ][2];                                   // of rows 2 l and 2 l + 1 of every 8
  int lim[NQ][2];
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    const uint4 (&w)[4] = qw[q];
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t ws[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) amax = max(amax, max(ws[e] & 0x7FFFu, (ws[e] >> 16) & 0x7FFFu));
    }
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    float f, inv;
    kv8_row_scale(amax, f, inv);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int rr = 8 * q + 2 * l + x;
      coef[q][x] = __shfl_sync(0xffffffffu, inv, 4 * (2 * l + x)) * a.scale_log2;
      lim[q][x] = rr < nrows ? kv8_visible(a.causal, len, n, (row_first + rr) / a.group) : vis;
    }
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      const uint4 u = w[kk >> 1];
      const uint32_t w0 = kk & 1 ? u.z : u.x, w1 = kk & 1 ? u.w : u.y;
      const float d0 = __uint_as_float(w0 << 16) * f, d1 = __uint_as_float(w0 & 0xFFFF0000u) * f;
      const float d2 = __uint_as_float(w1 << 16) * f, d3 = __uint_as_float(w1 & 0xFFFF0000u) * f;
      // the pairs kv8_to_f16 makes of a word's four codes
      qb[q][kk][0] = FMT == RBD_CODES_INT8 ? half2_bits(d0, d2) : half2_bits(d0, d1);
      qb[q][kk][1] = FMT == RBD_CODES_INT8 ? half2_bits(d1, d3) : half2_bits(d2, d3);
    }
  }
  int min_lim = lim[0][0];
#pragma unroll
  for (int q = 0; q < NQ; ++q) min_lim = min(min_lim, min(lim[q][0], lim[q][1]));
  min_lim = __reduce_min_sync(0xffffffffu, min_lim);

  float o[NQ][8][4];
  float m_run[NQ][2], l_run[NQ][2];
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[q][j][e] = 0.f;
    m_run[q][0] = m_run[q][1] = -INFINITY;
    l_run[q][0] = l_run[q][1] = 0.f;
  }
  bool ok = true;
  for (int i = 0; i < cnt; ++i) {
    const float sk = __shfl_sync(0xffffffffu, my_sk, i & 31), lsv = __shfl_sync(0xffffffffu, my_lsv, i & 31);
    const float inv_sv = __shfl_sync(0xffffffffu, my_inv, i & 31);
    if (((i + 1) & 31) == 0) {
      look_up(i + 1);
      look_up_scales();
    }
    const int next = __shfl_sync(0xffffffffu, my_page, (i + 1) & 31);
    const bool more = i + 1 < cnt;
    if (!__all_sync(0xffffffffu, mbar_wait(&full[0], i & 1))) { ok = false; break; }
    // a page outside the pool: no query sees its tokens
    const int t0 = page >= 0 ? (p0 + warp + i * W) * kKv8Page : 1 << 30;
    const bool masked = t0 + kKv8Page > min_lim;
    float s[NQ][4][4];                                 // token 16 mt + g (+ 8), rows 2 l, 2 l + 1
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
      for (int q = 0; q < NQ; ++q) s[q][mt][0] = s[q][mt][1] = s[q][mt][2] = s[q][mt][3] = 0.f;
      uint4 u[2][2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        u[x][0] = *reinterpret_cast<const uint4*>(ring + kv8_chunk(16 * mt + 8 * x + g, 2 * l));
        u[x][1] = *reinterpret_cast<const uint4*>(ring + kv8_chunk(16 * mt + 8 * x + g, 2 * l + 1));
      }
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        uint32_t af[4];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint4& v = u[x][kk >> 2];
          const uint32_t w = (kk & 3) == 0 ? v.x : (kk & 3) == 1 ? v.y : (kk & 3) == 2 ? v.z : v.w;
          kv8_to_f16<FMT>(w, af[x], af[2 + x]);
        }
#pragma unroll
        for (int q = 0; q < NQ; ++q) mma_f16(s[q][mt], af, qb[q][kk][0], qb[q][kk][1]);
      }
    }
    __syncwarp();
    fence_async_shared();
    if (more) issue(0, next);                          // the keys' buffer has been read
    float ck[NQ][2];
    uint32_t pb[NQ][4][2];                             // P^T fragments of 16 keys
    float mt_[NQ][2];
    bool move = false;
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      if (masked) {
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (t0 + 16 * mt + g + 8 * (e >> 1) >= lim[q][e & 1]) s[q][mt][e] = -INFINITY;
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float mx = fmaxf(s[q][0][x], s[q][0][2 + x]);
#pragma unroll
        for (int mt = 1; mt < 4; ++mt) mx = fmaxf(mx, fmaxf(s[q][mt][x], s[q][mt][2 + x]));
        mx = col_max(mx);
        ck[q][x] = coef[q][x] * sk;
        mt_[q][x] = mx > -INFINITY ? fmaxf(fmaf(mx, ck[q][x], lsv), -kKv8Far) : -INFINITY;
        move = move || mt_[q][x] > m_run[q][x] + kKv8Lazy;
      }
    }
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        float f[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const bool up = mt_[q][x] > m_run[q][x] + kKv8Lazy;
          f[x] = up ? ex2(m_run[q][x] - mt_[q][x]) : 1.f;
          if (up) m_run[q][x] = mt_[q][x];
          l_run[q][x] *= f[x];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[q][j][e] *= f[e & 1];
      }
    }
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      if (a.logits) {                                  // (of a page outside the pool: no weight for any query)
        const int at = (p0 + warp + i * W) * kKv8Page + g;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int rr = 8 * q + 2 * l + x;
          if (rr < nrows) {
            const int r = row_first + rr;
            float* dst = a.logits + ((int64_t)(r0 + r / a.group) * a.q_heads + head * a.group + r % a.group) * a.logit_ld + at;
#pragma unroll
            for (int e = 0; e < 8; ++e) dst[8 * e] = page >= 0 ? s[q][e >> 1][2 * (e & 1) + x] * ck[q][x] : -INFINITY;
          }
        }
      }
      float base[2], lp[2] = {0.f, 0.f};
#pragma unroll
      for (int x = 0; x < 2; ++x) base[x] = lsv - (m_run[q][x] > -INFINITY ? m_run[q][x] : 0.f);
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float p = ex2(fmaf(s[q][mt][e], ck[q][e & 1], base[e & 1]));
          // (a score factor of zero, from a vanishing query, would turn a masked -inf into a NaN)
          if (masked && t0 + 16 * mt + g + 8 * (e >> 1) >= lim[q][e & 1]) p = 0.f;
          lp[e & 1] += p;
          s[q][mt][e] = p;
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) pb[q][mt][x] = transpose_8x8(half2_bits(s[q][mt][2 * x], s[q][mt][2 * x + 1]));
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) l_run[q][x] = fmaf(lp[x], inv_sv, l_run[q][x]);
    }
    if (!__all_sync(0xffffffffu, mbar_wait(&full[1], i & 1))) { ok = false; break; }
    const unsigned char* vt = ring + kKv8Side;
    const int valid = len - t0;        // rows of the page behind this hold nothing (an E4M3 NaN pattern perhaps)
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      uint32_t w[4][4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int t = 16 * mt + 2 * l + (x & 1) + 8 * (x >> 1);
        uint4 u = *reinterpret_cast<const uint4*>(vt + kv8_chunk(t, g));
        if (FMT != RBD_CODES_INT8 && masked && t >= valid) u = make_uint4(0u, 0u, 0u, 0u);
        w[x][0] = u.x;
        w[x][1] = u.y;
        w[x][2] = u.z;
        w[x][3] = u.w;
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        // byte order in which kv8_to_f16 pairs the two keys of a channel
        constexpr uint32_t lo = FMT == RBD_CODES_INT8 ? 0x5410u : 0x5140u;
        constexpr uint32_t hi = FMT == RBD_CODES_INT8 ? 0x7632u : 0x7362u;
        uint32_t a0[4], a1[4];
        kv8_to_f16<FMT>(prmt(w[0][x], w[1][x], lo), a0[0], a0[1]);
        kv8_to_f16<FMT>(prmt(w[2][x], w[3][x], lo), a0[2], a0[3]);
        kv8_to_f16<FMT>(prmt(w[0][x], w[1][x], hi), a1[0], a1[1]);
        kv8_to_f16<FMT>(prmt(w[2][x], w[3][x], hi), a1[2], a1[3]);
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          mma_f16(o[q][2 * x], a0, pb[q][mt][0], pb[q][mt][1]);
          mma_f16(o[q][2 * x + 1], a1, pb[q][mt][0], pb[q][mt][1]);
        }
      }
    }
    __syncwarp();
    fence_async_shared();
    if (more) issue(1, next);
    page = next;
  }
  if (!ok) {   // copies still in flight land in this block's shared memory
    const uint64_t t = globaltimer_ns();
    while (globaltimer_ns() - t < 200000ull) {}
  }
  // this warp's O over its own ring, every copy into which has been consumed
  float* mine = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int q = 0; q < NQ; ++q)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const float lsum = col_sum(l_run[q][x]);
      const int rr = 8 * q + 2 * l + x;
      float* dst = mine + rr * kStORow + 16 * g;
#pragma unroll
      for (int j = 0; j < 8; j += 2)
        *reinterpret_cast<float4*>(dst + 2 * j) =
            make_float4(o[q][j][x], o[q][j][2 + x], o[q][j + 1][x], o[q][j + 1][2 + x]);
      if (g == 0) {
        red_m[warp * ROWS + rr] = m_run[q][x];
        red_l[warp * ROWS + rr] = lsum;
      }
    }
  __syncthreads();
  if (tid < ROWS) {
    float m = -INFINITY, lsum = 0.f;
    for (int w = 0; w < W; ++w) m = fmaxf(m, red_m[w * ROWS + tid]);
    for (int w = 0; w < W; ++w) {
      const float mw = red_m[w * ROWS + tid];
      // a row of NaN scores has no maximum but a NaN sum
      const float f = mw > -INFINITY ? ex2(mw - m) : 1.f;
      lsum += red_l[w * ROWS + tid] * f;
      red_m[w * ROWS + tid] = f;
    }
    row_m[tid] = m;
    row_l[tid] = lsum;
  }
  __syncthreads();
  for (int e = tid; e < ROWS * 16; e += Sh::kThreads) {
    const int rr = e >> 4, d = (e & 15) * 8;
    if (rr >= nrows) continue;
    float acc[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) acc[x] = 0.f;
    for (int w = 0; w < W; ++w) {
      const float f = red_m[w * ROWS + rr];
      const float* src = reinterpret_cast<const float*>(smem + w * kStPage) + rr * kStORow + d;
      const float4 u = *reinterpret_cast<const float4*>(src), v = *reinterpret_cast<const float4*>(src + 4);
      acc[0] = fmaf(u.x, f, acc[0]);
      acc[1] = fmaf(u.y, f, acc[1]);
      acc[2] = fmaf(u.z, f, acc[2]);
      acc[3] = fmaf(u.w, f, acc[3]);
      acc[4] = fmaf(v.x, f, acc[4]);
      acc[5] = fmaf(v.y, f, acc[5]);
      acc[6] = fmaf(v.z, f, acc[6]);
      acc[7] = fmaf(v.w, f, acc[7]);
    }
    const int r = row_first + rr;
    const int qh = head * a.group + r % a.group;
    const int64_t tok = r0 + r / a.group;
    const int64_t fr = tok * a.q_heads + qh;
    const float lsum = row_l[rr];
    if (a.nsplit == 1) {
      const float inv = kv8_inverse(row_m[rr], lsum);
      uint32_t ow[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const __nv_bfloat162 p2 = __floats2bfloat162_rn(acc[2 * x] * inv, acc[2 * x + 1] * inv);
        ow[x] = *reinterpret_cast<const uint32_t*>(&p2);
      }
      *reinterpret_cast<uint4*>(a.o + tok * a.ldo + (int64_t)qh * kKv8Dim + d) = make_uint4(ow[0], ow[1], ow[2], ow[3]);
      if (a.stats && d == 0) a.stats[fr] = make_float2(row_m[rr] > -INFINITY ? row_m[rr] : 0.f, inv);
    } else {
      if (lsum != 0.f) {               // (the join reads nothing of a split without keys)
        float4* dst = reinterpret_cast<float4*>(a.part_o + (fr * a.nsplit + split) * kKv8Dim + d);
        dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
      }
      if (d == 0) a.part_ml[fr * a.nsplit + split] = make_float2(row_m[rr], lsum);
    }
  }
}

// Joins the splits of query token `tok` and head `qh`, kept in `slot`: a warp, 4 channels a lane.
__device__ __forceinline__ void kv8_join(const Kv8AttnArgs& a, int64_t slot, int64_t tok, int qh) {
  const int lane = threadIdx.x & 31;
  const int64_t fr = tok * a.q_heads + qh;
  const float2* ml = a.part_ml + slot * a.nsplit;          // at most 64 splits: two a lane
  const float2 none = make_float2(-INFINITY, 0.f);
  const float2 x0 = lane < a.nsplit ? ml[lane] : none, x1 = lane + 32 < a.nsplit ? ml[lane + 32] : none;
  float m = fmaxf(x0.x, x1.x);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  // factor of a split; zero for one without keys, which wrote no O (a NaN sum keeps its NaN)
  auto factor = [&](const float2& x) { return x.y == 0.f ? 0.f : (x.x > -INFINITY ? ex2(x.x - m) : 1.f); };
  const float f0 = factor(x0), f1 = factor(x1);
  float lsum = fmaf(x0.y, f0, x1.y * f1);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) lsum += __shfl_xor_sync(0xffffffffu, lsum, off);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  const float4* part = reinterpret_cast<const float4*>(a.part_o + slot * a.nsplit * kKv8Dim) + lane;
  for (int s0 = 0; s0 < a.nsplit; s0 += 4) {
    float4 u[4];
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int s = s0 + i;
      const float y = __shfl_sync(0xffffffffu, s < 32 ? x0.y : x1.y, s & 31);
      f[i] = __shfl_sync(0xffffffffu, s < 32 ? f0 : f1, s & 31);
      u[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s < a.nsplit && y != 0.f) u[i] = part[s * (kKv8Dim / 4)];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc.x = fmaf(u[i].x, f[i], acc.x);
      acc.y = fmaf(u[i].y, f[i], acc.y);
      acc.z = fmaf(u[i].z, f[i], acc.z);
      acc.w = fmaf(u[i].w, f[i], acc.w);
    }
  }
  const float inv = kv8_inverse(m, lsum);
  const __nv_bfloat162 p = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), q = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2*>(a.o + tok * a.ldo + (int64_t)qh * kKv8Dim + 4 * lane) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&p), *reinterpret_cast<const uint32_t*>(&q));
  if (a.stats && lane == 0) a.stats[fr] = make_float2(m > -INFINITY ? m : 0.f, inv);
}

// Joins the splits of every (query token, head): a warp each.  Query tokens are counted through the sequences, as the
// streaming kernel does: rows of none, and of one whose offsets are refused, stay as they are.
__global__ void __launch_bounds__(256) kv8_combine_kernel(const Kv8AttnArgs a) {
  const int64_t at = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t x = at / a.q_heads;
  if (x >= a.rows) return;
  Kv8Item it;
  if (!kv8_find(a.cu, a.lens, a.seqs, a.rows, (int)x, [](int n, int) { return n; }, it)) return;
  const int64_t tok = it.r0 + it.idx;
  const int qh = (int)(at - x * a.q_heads);
  kv8_join(a, tok * a.q_heads + qh, tok, qh);
}

// weights_out = weights_in + sum of a key's weights over the queries and heads of
// its group, from the scores the stream kernel left behind: a thread per key.
__global__ void __launch_bounds__(256)
    kv8_weigh_logits_kernel(const Kv8View c, const Kv8AttnArgs a, const float* w_in, float* w_out, int64_t w_seq,
                            int64_t w_head) {
  const int b = blockIdx.z, head = blockIdx.y;
  const int t = blockIdx.x * 256 + threadIdx.x;
  int r0, n;
  kv8_rows(a.cu, b, a.rows, r0, n);
  const int len = kv8_len(c, a, b);
  if (t >= len) return;
  float acc = 0.f;
  const int i0 = a.causal ? max(0, t - (len - n)) : 0;       // first query that sees key t
  for (int i = i0; i < n; ++i)
    for (int gq = 0; gq < a.group; ++gq) {
      const int64_t fr = (int64_t)(r0 + i) * a.q_heads + head * a.group + gq;
      const float2 st = a.stats[fr];
      acc = fmaf(ex2(a.logits[fr * a.logit_ld + t] - st.x), st.y, acc);
    }
  const int64_t at = b * w_seq + head * w_head + t;
  w_out[at] = w_in[at] + acc;
}

}  // namespace rbd

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
// range whatever the pages' scales.  p is rounded to fp16 for the second product
// (a random half step of 2^-11 each); m, L, O and the scores are float32.
// The maximum moves only when a row exceeds it by 2^8 (p <= 256 then), which
// leaves most rescales of O out.
//
// Two kernels do the work, chosen by the rows (query tokens x heads of a group)
// that share a key/value head:
//   kv8_stream_kernel  up to kStreamRows a sequence on average: bound by reading
//                      the cache once.  Warps stream pages from memory.
//   kv8_tile_kernel    more: bound by the tensor cores (tcgen05).
// Both split the keys over several blocks when there are few items and write
// float32 partial results, which kv8_combine_kernel joins.
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
  float* part_o;       // [rows * q_heads][nsplit][128]: O of a split (null with one split)
  float2* part_ml;     // [rows * q_heads][nsplit]: (m, L)
  float2* stats;       // [rows * q_heads]: (m, 1 / L) of the whole row, or null
  float* logits;       // [rows * q_heads][logit_ld]: base-2 scores (stream kernel), or null
  int64_t logit_ld;
  uint8_t* q_image;    // [heads][items][2][32 KB]: the fp16 query tiles (tile kernel), or null
  float* q_coef;       // [heads][items][2][128]: base-2 score factor of every row of them
  uint8_t* kv_image;   // [seqs][image_steps][heads][2][32 KB]: fp16 operands of every 128-key step, or null
  float4* kv_scale;    // [seqs][image_steps][heads][2]: their page scales (s_k, log2 s_v, 1 / s_v, -)
  int image_steps;
};

namespace {

constexpr float kKv8Lazy = 8.0f;

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// The power of two that brings a row whose largest |bf16| has bits `amax` to [2^14, 2^15), and its inverse.
__device__ __forceinline__ void kv8_row_scale(uint32_t amax, float& f, float& inv) {
  const int e = (int)(amax >> 7);
  const int field = min(268 - e, 253);
  f = __uint_as_float((uint32_t)field << 23);
  inv = __uint_as_float((uint32_t)(254 - field) << 23);
}

// Length of sequence b, or 0 (recorded) when it exceeds what the call declared.
__device__ __forceinline__ int kv8_len(const Kv8View& c, const Kv8AttnArgs& a, int b) {
  const int len = __ldg(a.lens + b);
  if (len >= 0 && len <= a.max_len && len <= c.max_pages * kKv8Page) return len;
  record_refusal();
  return 0;
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

__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

}  // namespace

// ---------------------------------------------------------------------------
// Few rows: warps stream pages
// ---------------------------------------------------------------------------
// A block takes 16 rows of one (sequence, key/value head) and one split of its
// pages; its warps take pages in turn, each with its own ring of bulk copies (16
// KB, keys and values of a page), its own running maximum and its own O, and are
// joined through shared memory at the end: no warp waits for another in the loop.
// Products on mma.sync m16n8k16 (a 128-row tcgen05 tile would be 1/8 full at
// best), fragments straight from the bulk-copied bytes:
//   scores   lane (g, l) of the quad layout holds channels 32 l .. 32 l + 31 of key
//            g of every 8: the contraction order of channels is free, the query
//            fragments use the same one;
//   output   lane (g, l) holds channels 16 g .. 16 g + 15 of keys 2 l, 2 l + 1, 2 l
//            + 8, 2 l + 9 of every 16: output column g of product j is channel 16 g + j.
constexpr int kStWarps = 6;
constexpr int kStStages = 2;
constexpr int kStThreads = 32 * kStWarps;
constexpr int kStRows = 16;
constexpr uint32_t kStPage = 2 * kKv8Side;                          // 16 KB
constexpr uint32_t kStRing = kStWarps * kStStages * kStPage;
constexpr uint32_t kStSmem = kStRing + 256 + 2 * kStWarps * kStRows * 4 + 2 * kStRows * 4 + 128;
constexpr int kStORow = kKv8Dim + 4;                                // padded row of a warp's O in shared memory

template <int FMT>
__global__ void __launch_bounds__(kStThreads, 1) kv8_stream_kernel(const Kv8View c, const Kv8AttnArgs a) {
  extern __shared__ unsigned char smem_dyn[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_dyn) + 127u) & ~uintptr_t(127u));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kStRing);
  float* red_m = reinterpret_cast<float*>(smem + kStRing + 256);   // [warps][16]
  float* red_l = red_m + kStWarps * kStRows;                        // [warps][16]
  float* row_l = red_l + kStWarps * kStRows;                        // [16]
  float* row_m = row_l + kStRows;                                   // [16]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, l = lane & 3;
  const int head = blockIdx.y, split = blockIdx.z;

  auto tiles_of = [&](int b) {
    int r0, n;
    kv8_rows(a.cu, b, a.rows, r0, n);
    return (int)(((int64_t)n * a.group + kStRows - 1) / kStRows);
  };
  int b, tile;
  if (!kv8_find(c.seqs, blockIdx.x, tiles_of, b, tile)) return;
  int r0, n;
  kv8_rows(a.cu, b, a.rows, r0, n);
  const int len = kv8_len(c, a, b);
  const int row_first = tile * kStRows;
  const int nrows = min(kStRows, n * a.group - row_first);
  const int vis = min(len, kv8_visible(a.causal, len, n, (row_first + nrows - 1) / a.group));
  const int npages = (vis + kKv8Page - 1) / kKv8Page;
  const int per = (npages + a.nsplit - 1) / a.nsplit;
  const int p0 = split * per, p1 = min(npages, p0 + per);
  const int cnt = p1 - p0 > warp ? (p1 - p0 - warp + kStWarps - 1) / kStWarps : 0;

  if (lane == 0) {
    for (int s = 0; s < kStStages; ++s) mbar_init(&bars[warp * kStStages + s], 1);
    fence_barrier_init();
  }
  __syncwarp();
  unsigned char* ring = smem + warp * kStStages * kStPage;
  uint64_t* full = bars + warp * kStStages;
  auto page_at = [&](int i) { return i < cnt ? kv8_page(c, b, p0 + warp + i * kStWarps) : -1; };
  auto issue = [&](int i, int page) {
    if (i >= cnt || lane != 0) return;
    uint64_t* bar = &full[i % kStStages];
    if (page >= 0) {
      mbar_arrive_expect_tx(bar, kStPage);
      bulk_load(ring + (i % kStStages) * kStPage, c.codes + kv8_tile(c, page, head, 0), kStPage, bar);
    } else {
      mbar_arrive(bar);
    }
  };
  int pages[kStStages + 1];
#pragma unroll
  for (int i = 0; i <= kStStages; ++i) pages[i] = page_at(i);
#pragma unroll
  for (int i = 0; i < kStStages; ++i) issue(i, pages[i]);

  // query fragments: row g and row g + 8, channels 32 l .. 32 l + 31
  uint32_t qa[8][4];
  float coef[2];
  int lim[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = row_first + g + 8 * h;
    const bool live = g + 8 * h < nrows;
    uint4 w[4];
    if (live) {
      const uint4* src = reinterpret_cast<const uint4*>(a.q + (int64_t)(r0 + r / a.group) * a.ldq +
                                                        (int64_t)(head * a.group + r % a.group) * kKv8Dim + 32 * l);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __ldg(src + i);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
    }
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
    coef[h] = inv * a.scale_log2;
    lim[h] = live ? kv8_visible(a.causal, len, n, r / a.group) : vis;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      const uint4 u = w[kk >> 1];
      const uint32_t w0 = kk & 1 ? u.z : u.x, w1 = kk & 1 ? u.w : u.y;
      const float d0 = __uint_as_float(w0 << 16) * f, d1 = __uint_as_float(w0 & 0xFFFF0000u) * f;
      const float d2 = __uint_as_float(w1 << 16) * f, d3 = __uint_as_float(w1 & 0xFFFF0000u) * f;
      // the pairs kv8_to_f16 makes of a word's four codes
      qa[kk][h] = FMT == RBD_CODES_INT8 ? half2_bits(d0, d2) : half2_bits(d0, d1);
      qa[kk][2 + h] = FMT == RBD_CODES_INT8 ? half2_bits(d1, d3) : half2_bits(d2, d3);
    }
  }
  const int min_lim = __reduce_min_sync(0xffffffffu, min(lim[0], lim[1]));

  float o[16][4];
#pragma unroll
  for (int j = 0; j < 16; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
  float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
  auto scales_of = [&](int page) {
    return page >= 0 ? *reinterpret_cast<const float2*>(c.scales + kv8_scale(c, page, head, 0)) : make_float2(1.f, 1.f);
  };
  float2 sc_next = scales_of(pages[0]);
  bool ok = true;
  for (int i = 0; i < cnt; ++i) {
    const float2 sc = sc_next;
    const int page = pages[0];
    sc_next = scales_of(pages[1]);
    if (!__all_sync(0xffffffffu, mbar_wait(&full[i % kStStages], (i / kStStages) & 1))) { ok = false; break; }
    if (page >= 0) {
      const unsigned char* kt = ring + (i % kStStages) * kStPage;
      const unsigned char* vt = kt + kKv8Side;
      const int t0 = (p0 + warp + i * kStWarps) * kKv8Page;
      float s[8][4];
#pragma unroll
      for (int nt = 0; nt < 8; ++nt) {
        s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
        const int t = 8 * nt + g;
        const uint4 u0 = *reinterpret_cast<const uint4*>(kt + kv8_chunk(t, 2 * l));
        const uint4 u1 = *reinterpret_cast<const uint4*>(kt + kv8_chunk(t, 2 * l + 1));
        const uint32_t ws[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          uint32_t b0, b1;
          kv8_to_f16<FMT>(ws[kk], b0, b1);
          mma_f16(s[nt], qa[kk], b0, b1);
        }
      }
      const bool masked = t0 + kKv8Page > min_lim;
      if (masked) {
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (t0 + 8 * nt + 2 * l + (e & 1) >= lim[e >> 1]) s[nt][e] = -INFINITY;
      }
      const float lsv = log2f(sc.y), inv_sv = 1.0f / sc.y;
      float base[2], ck[2];
      bool move = false;
      float mt[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mx = -INFINITY;
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) mx = fmaxf(mx, fmaxf(s[nt][2 * h], s[nt][2 * h + 1]));
        mx = quad_max(mx);
        ck[h] = coef[h] * sc.x;
        mt[h] = mx > -INFINITY ? fmaf(mx, ck[h], lsv) : -INFINITY;
        move = move || mt[h] > m_run[h] + kKv8Lazy;
      }
      if (__any_sync(0xffffffffu, move)) {
        float f[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bool up = mt[h] > m_run[h] + kKv8Lazy;
          f[h] = up ? ex2(m_run[h] - mt[h]) : 1.f;
          if (up) m_run[h] = mt[h];
          l_run[h] *= f[h];
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          o[j][0] *= f[0];
          o[j][1] *= f[0];
          o[j][2] *= f[1];
          o[j][3] *= f[1];
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) base[h] = lsv - (m_run[h] > -INFINITY ? m_run[h] : 0.f);
      if (a.logits) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = row_first + g + 8 * h;
          if (g + 8 * h < nrows) {
            float* dst = a.logits + ((int64_t)(r0 + r / a.group) * a.q_heads + head * a.group + r % a.group) * a.logit_ld +
                         t0 + 2 * l;
#pragma unroll
            for (int nt = 0; nt < 8; ++nt)
              *reinterpret_cast<float2*>(dst + 8 * nt) = make_float2(s[nt][2 * h] * ck[h], s[nt][2 * h + 1] * ck[h]);
          }
        }
      }
      float lp[2] = {0.f, 0.f};
#pragma unroll
      for (int nt = 0; nt < 8; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float p = ex2(fmaf(s[nt][e], ck[e >> 1], base[e >> 1]));
          if (masked && t0 + 8 * nt + 2 * l + (e & 1) >= lim[e >> 1]) p = 0.f;
          lp[e >> 1] += p;
          s[nt][e] = p;
        }
#pragma unroll
      for (int h = 0; h < 2; ++h) l_run[h] = fmaf(lp[h], inv_sv, l_run[h]);
      const int valid = len - t0;      // rows of the page behind this hold nothing (an E4M3 NaN pattern perhaps)
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const uint32_t pa[4] = {half2_bits(s[2 * kk][0], s[2 * kk][1]), half2_bits(s[2 * kk][2], s[2 * kk][3]),
                                half2_bits(s[2 * kk + 1][0], s[2 * kk + 1][1]),
                                half2_bits(s[2 * kk + 1][2], s[2 * kk + 1][3])};
        uint32_t w[4][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int t = 16 * kk + 2 * l + (q & 1) + 8 * (q >> 1);
          uint4 u = *reinterpret_cast<const uint4*>(vt + kv8_chunk(t, g));
          if (FMT != RBD_CODES_INT8 && t >= valid) u = make_uint4(0u, 0u, 0u, 0u);
          w[q][0] = u.x;
          w[q][1] = u.y;
          w[q][2] = u.z;
          w[q][3] = u.w;
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          // byte order in which kv8_to_f16 pairs the two keys of a channel
          constexpr uint32_t lo = FMT == RBD_CODES_INT8 ? 0x5410u : 0x5140u;
          constexpr uint32_t hi = FMT == RBD_CODES_INT8 ? 0x7632u : 0x7362u;
          uint32_t a0, a1, a2, a3, c0, c1, c2, c3;
          kv8_to_f16<FMT>(prmt(w[0][x], w[1][x], lo), a0, a1);
          kv8_to_f16<FMT>(prmt(w[0][x], w[1][x], hi), a2, a3);
          kv8_to_f16<FMT>(prmt(w[2][x], w[3][x], lo), c0, c1);
          kv8_to_f16<FMT>(prmt(w[2][x], w[3][x], hi), c2, c3);
          mma_f16(o[4 * x], pa, a0, c0);
          mma_f16(o[4 * x + 1], pa, a1, c1);
          mma_f16(o[4 * x + 2], pa, a2, c2);
          mma_f16(o[4 * x + 3], pa, a3, c3);
        }
      }
    }
    __syncwarp();
    fence_async_shared();
    issue(i + kStStages, pages[kStStages]);
#pragma unroll
    for (int q = 0; q < kStStages; ++q) pages[q] = pages[q + 1];
    pages[kStStages] = page_at(i + kStStages + 1);
  }
  if (!ok) {   // copies still in flight land in this block's shared memory
    const uint64_t t = globaltimer_ns();
    while (globaltimer_ns() - t < 200000ull) {}
  }
  l_run[0] = quad_sum(l_run[0]);
  l_run[1] = quad_sum(l_run[1]);
  // this warp's O over its own ring, every copy into which has been consumed
  float* mine = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float* dst = mine + (g + 8 * h) * kStORow + 32 * l;
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
      *reinterpret_cast<float4*>(dst + j) =
          make_float4(o[j][2 * h], o[j + 1][2 * h], o[j + 2][2 * h], o[j + 3][2 * h]);
      *reinterpret_cast<float4*>(dst + 16 + j) =
          make_float4(o[j][2 * h + 1], o[j + 1][2 * h + 1], o[j + 2][2 * h + 1], o[j + 3][2 * h + 1]);
    }
    if (l == 0) {
      red_m[warp * kStRows + g + 8 * h] = m_run[h];
      red_l[warp * kStRows + g + 8 * h] = l_run[h];
    }
  }
  __syncthreads();
  if (tid < kStRows) {
    float m = -INFINITY, lsum = 0.f;
    for (int w = 0; w < kStWarps; ++w) m = fmaxf(m, red_m[w * kStRows + tid]);
    for (int w = 0; w < kStWarps; ++w) {
      const float mw = red_m[w * kStRows + tid];
      const float f = mw > -INFINITY ? ex2(mw - m) : 0.f;
      // a row of NaN scores has no maximum but a NaN sum
      lsum += red_l[w * kStRows + tid] * (mw > -INFINITY ? f : 1.f);
      red_m[w * kStRows + tid] = mw > -INFINITY ? f : 1.f;
    }
    row_m[tid] = m;
    row_l[tid] = lsum;
  }
  __syncthreads();
  for (int e = tid; e < kStRows * 16; e += kStThreads) {
    const int rr = e >> 4, d = (e & 15) * 8;
    if (rr >= nrows) continue;
    float acc[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) acc[x] = 0.f;
    for (int w = 0; w < kStWarps; ++w) {
      const float f = red_m[w * kStRows + rr];
      const float* src = reinterpret_cast<const float*>(smem + w * kStStages * kStPage) + rr * kStORow + d;
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
      const float inv = lsum == 0.f ? 0.f : 1.0f / lsum;
      uint32_t ow[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const __nv_bfloat162 p2 = __floats2bfloat162_rn(acc[2 * x] * inv, acc[2 * x + 1] * inv);
        ow[x] = *reinterpret_cast<const uint32_t*>(&p2);
      }
      *reinterpret_cast<uint4*>(a.o + tok * a.ldo + (int64_t)qh * kKv8Dim + d) = make_uint4(ow[0], ow[1], ow[2], ow[3]);
      if (a.stats && d == 0) a.stats[fr] = make_float2(row_m[rr] > -INFINITY ? row_m[rr] : 0.f, inv);
    } else {
      float4* dst = reinterpret_cast<float4*>(a.part_o + (fr * a.nsplit + split) * kKv8Dim + d);
      dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
      if (d == 0) a.part_ml[fr * a.nsplit + split] = make_float2(row_m[rr], lsum);
    }
  }
}

// Joins the splits of every (query token, head): a warp each, 4 channels a lane.
__global__ void __launch_bounds__(256) kv8_combine_kernel(const Kv8AttnArgs a) {
  const int64_t fr = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (fr >= (int64_t)a.rows * a.q_heads) return;
  const int64_t tok = fr / a.q_heads;
  if (tok < __ldg(a.cu) || tok >= __ldg(a.cu + a.seqs)) return;      // rows of no sequence stay as they are
  const float2* ml = a.part_ml + fr * a.nsplit;
  float m = -INFINITY;
  for (int s = 0; s < a.nsplit; ++s) m = fmaxf(m, ml[s].x);
  float lsum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < a.nsplit; ++s) {
    const float2 x = ml[s];
    if (x.y == 0.f) continue;                     // a split without keys wrote no O
    const float f = x.x > -INFINITY ? ex2(x.x - m) : 1.f;
    const float4 u = *reinterpret_cast<const float4*>(a.part_o + (fr * a.nsplit + s) * kKv8Dim + 4 * lane);
    lsum = fmaf(x.y, f, lsum);
    acc.x = fmaf(u.x, f, acc.x);
    acc.y = fmaf(u.y, f, acc.y);
    acc.z = fmaf(u.z, f, acc.z);
    acc.w = fmaf(u.w, f, acc.w);
  }
  const float inv = lsum == 0.f ? 0.f : 1.0f / lsum;
  const __nv_bfloat162 p = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), q = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2*>(a.o + tok * a.ldo + (fr - tok * a.q_heads) * kKv8Dim + 4 * lane) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&p), *reinterpret_cast<const uint32_t*>(&q));
  if (a.stats && lane == 0) a.stats[fr] = make_float2(m > -INFINITY ? m : 0.f, inv);
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

// Attention over the 8-bit paged cache for many query rows: the tensor-core
// kernels.  The mathematics (value scales in the exponent, power-of-two query
// scaling) is described in rbd_kv8_attn.cu.
//
// kv8_tile_kernel, one block per 256 rows (two query tiles of 128) of one
// (sequence, key/value head) and one split of its keys:
//   warps 0-3, 4-7   softmax of query tile 0 / 1, a thread a row (TMEM lane);
//   warp 8           TMEM owner and MMA issuer;
//   warp 9           loader of prepared operands (a bulk copy each), or
//   warps 12-15      converters: codes from global memory to fp16 operands.
// Per step and query tile t: S_t = Q_t K^T into TMEM columns 128 t .. (fp16 operands
// from shared memory), the softmax writes P_t as fp16 over the first 64 of those
// columns, and O_t += P_t V takes P_t from TMEM and V from shared memory as it is
// stored, token by token (an MN-major operand), so V is never transposed.  The
// issuer interleaves the tiles: while softmax t works, the tensor core runs P.V and
// Q.K^T of the other tile.
// Operands come in one of two ways.  Where a key is used by several blocks (prompts,
// image blocks), kv8_prepare_kernel converts every step's codes once into operand
// images in the workspace; converting in every block cost the softmax its integer
// pipe (4096 queries over 16384 keys x 24 heads, at an early stage: 2157 us against 748
// without softmax and converters).  Where it is used once, the images' traffic (5 bytes a value
// against 1) would dominate, and the block converts for itself.
// Measured: 4096 queries over 16384 keys x 24 heads with the images (47 us of it) and
// the join of what is split (15) in 705 us, 1.17 PFLOP/s, where something else runs
// between the calls, and 785 us, 1.05 PFLOP/s, call after call under the power cap; the
// tensor pipe is 63% busy.  What bounds it is the chain of a query tile: a softmax step
// (128 scores a thread, about 2000 cycles, 1275 of them exponentials) and then its P.V
// and Q.K^T (1024), of which the other tile hides the latter; of ragged causal prompts
// (21186 tokens x 48 heads: 1011 and 1030 us, 0.84 PFLOP/s) also setting up and leaving
// a block, some 14000 of 75000 cycles.
#include <type_traits>

#include "rbd_kv8.cuh"
#include "rbd_internal.cuh"

namespace rbd {

namespace {

constexpr int kTlRows = 128;                       // rows of a query tile (TMEM lanes)
constexpr int kTlKeys = 128;                       // keys per step
constexpr int kTlThreads = 384;                    // with a loader
constexpr int kTlConvThreads = 512;                // with converters
constexpr uint32_t kTlTile = 32768;                // a 128 x 128 fp16 operand: two 64-channel halves of 128-byte rows
constexpr uint32_t kTlK = 2 * kTlTile;             // keys, 2 stages
constexpr uint32_t kTlV = kTlK + 2 * kTlTile;      // values, 2 stages
constexpr uint32_t kTlScale = kTlV + 2 * kTlTile;  // page scales: 4 slots x 2 pages x (s_k, log2 s_v, 1 / s_v, least maximum)
constexpr uint32_t kTlCoef = kTlScale + 4 * 32;    // base-2 score factor of the 256 rows
constexpr uint32_t kTlBar = kTlCoef + 256 * 4;
constexpr uint32_t kTlSmem = kTlBar + 256 + 1024;  // + alignment slack

// Two float32 operations in one issue slot: the softmax is short of slots, not of FMA lanes.
__device__ __forceinline__ uint64_t pack_f32(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void unpack_f32(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// 2^x and 2^y on the FMA pipe, for a quarter of the keys: the special-function unit takes 8 cycles a warp for each
// 2^x and is the longest phase of the softmax (1590 cycles of a 128-key step without this, 1275 with; 960 -> 922 us
// at 4096 queries over 16384 keys x 24 heads; half of the keys: 985 us).  x = n + f with n the nearest whole number
// and |f| <= 1/2; 2^f by its degree-4 polynomial of least largest relative error (2.6e-6, far under P's half step of
// 2^-11); n added to the exponent.  A NaN comes out as a number: a row has one from a query that is not finite alone,
// and then in every key, so that the other three quarters keep it.
__device__ __forceinline__ void ex2_poly(float& x, float& y) {
  const uint64_t v = pack_f32(fmaxf(x, -126.f), fmaxf(y, -126.f));
  const uint64_t t = add_f32x2(v, pack_f32(12582912.f, 12582912.f));               // 1.5 * 2^23: rounds to whole
  const uint64_t f = fma_f32x2(add_f32x2(t, pack_f32(-12582912.f, -12582912.f)), pack_f32(-1.f, -1.f), v);
  uint64_t p = fma_f32x2(f, pack_f32(0.009570086374878883f, 0.009570086374878883f),
                         pack_f32(0.055917851626873016f, 0.055917851626873016f));
  p = fma_f32x2(f, p, pack_f32(0.240247443318367f, 0.240247443318367f));
  p = fma_f32x2(f, p, pack_f32(0.6931217908859253f, 0.6931217908859253f));
  p = fma_f32x2(f, p, pack_f32(0.9999992847442627f, 0.9999992847442627f));
  float p0, p1, t0, t1;
  unpack_f32(p, p0, p1);
  unpack_f32(t, t0, t1);
  x = __int_as_float(__float_as_int(p0) + (__float_as_int(t0) << 23));
  y = __int_as_float(__float_as_int(p1) + (__float_as_int(t1) << 23));
}
// The larger of three (one instruction on sm_100).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Shared-memory descriptor of an MN-major fp16 operand with the 128-byte swizzle: rows of 64 MN elements (128
// bytes), one row per K index; 8-row groups sbo bytes apart along K, 64-element blocks lbo bytes apart along MN.
__device__ __forceinline__ uint64_t smem_desc_mnmajor(uint32_t smem_addr, uint32_t lbo, uint32_t sbo) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr >> 4) & 0x3FFFu);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)((sbo >> 4) & 0x3FFFu) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}

// The issuing warp runs its loop with all lanes, so that descriptors stay in uniform registers, and only the lane
// with `leader` set issues: computed in one lane's branch they cost 90-115 cycles per product beside the softmax
// warps, against 64 of the tensor core.
// D[tmem] (+)= A[smem] * B[smem]^T, 16-bit float inputs, fp32 accumulation.
__device__ __forceinline__ void mma_f16_ss_if(uint32_t leader, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]^T.
__device__ __forceinline__ void mma_f16_ts_if(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void tc_commit_if(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(leader)
      : "memory");
}
// Items (256 rows) of a sequence with n query tokens.
struct Kv8TileItems {
  int group;
  __device__ int operator()(int n, int) const {
    return (int)(((int64_t)n * group + 2 * kTlRows - 1) / (2 * kTlRows));
  }
};

// The (head, item) pair of a block, its split and the number of splits: first the blocks of whole pairs, then
// those of the pairs behind them, whose keys are split.
__device__ __forceinline__ int kv8_tile_place(const Kv8AttnArgs& a, int& head, int& split, int& nsplit) {
  int at = blockIdx.x;
  split = 0;
  nsplit = 1;
  if (at >= a.whole) {
    nsplit = a.nsplit;
    split = (at - a.whole) % nsplit;
    at = a.whole + (at - a.whole) / nsplit;
  }
  head = at / a.items;
  return at;
}

constexpr uint32_t kIdescBMn = 1u << 16;           // B is MN-major

template <int N>
__device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Byte offset of 16-byte chunk ch (0..15, 8 channels each) of row t in a 128 x 128 fp16 operand.
__device__ __forceinline__ uint32_t tile_chunk(int t, int ch) {
  return (uint32_t)(ch >> 3) * 16384u + (uint32_t)t * 128u + (uint32_t)(((ch & 7) ^ (t & 7)) << 4);
}

// Eight codes as fp16, in order.
template <int FMT>
__device__ __forceinline__ uint4 eight_codes(const uint2& w) {
  uint4 h;
  kv8_to_f16<FMT>(FMT == RBD_CODES_INT8 ? prmt(w.x, 0u, 0x3120u) : w.x, h.x, h.y);
  kv8_to_f16<FMT>(FMT == RBD_CODES_INT8 ? prmt(w.y, 0u, 0x3120u) : w.y, h.z, h.w);
  return h;
}
// What the softmax takes of a page: the keys' factor, log2 and inverse of the values' one, and the least that its
// maximum counts for.  A page that the table does not name has zeros for codes and a value scale of zero: all its keys
// get 2^(0 + log2 0) = 0, and none of that joins L.
__device__ __forceinline__ float4 page_scales(float2 sc) {
  return make_float4(sc.x, log2f(sc.y), sc.y > 0.f ? 1.0f / sc.y : 0.f, sc.y > 0.f ? -kKv8Far : -INFINITY);
}
// Sixteen codes of one token as fp16, channels 16 c .. 16 c + 15, into an operand tile.
template <int FMT>
__device__ __forceinline__ void store_codes(unsigned char* tile, int t, int c, const uint4& w) {
  *reinterpret_cast<uint4*>(tile + tile_chunk(t, 2 * c)) = eight_codes<FMT>(make_uint2(w.x, w.y));
  *reinterpret_cast<uint4*>(tile + tile_chunk(t, 2 * c + 1)) = eight_codes<FMT>(make_uint2(w.z, w.w));
}

}  // namespace

// Operand images of every 128-key step of the sequences: [seqs][steps][heads] x (32
// KB of keys, 32 KB of values, as the tensor core reads them) and the page scales.
template <int FMT>
__global__ void __launch_bounds__(256)
    kv8_prepare_kernel(const Kv8View c, const Kv8AttnArgs a) {
  const int b = blockIdx.z, head = blockIdx.y, step = blockIdx.x;
  const int len = kv8_len(c, a, b);
  if (step * kTlKeys >= len) return;
  const int64_t img = ((int64_t)b * gridDim.x + step) * c.heads + head;
  int page[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int p = 2 * step + h;
    page[h] = p * kKv8Page < len ? kv8_page(c, b, p) : -1;
  }
  if (threadIdx.x < 2) {
    float2 sc = make_float2(1.f, 0.f);
    if (page[threadIdx.x] >= 0)
      sc = *reinterpret_cast<const float2*>(c.scales + kv8_scale(c, page[threadIdx.x], head, 0));
    a.kv_scale[img * 2 + threadIdx.x] = page_scales(sc);
  }
  // eight codes a thread and turn: 16 bytes out, whole 128-byte lines a warp
  uint2 raw[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int e = threadIdx.x + 256 * (i & 7);
    const int t = e >> 4, ch = e & 15, side = i >> 3;
    const int pg = page[t >> 6];
    raw[i] = make_uint2(0u, 0u);
    if (pg >= 0 && step * kTlKeys + t < len)
      raw[i] = *reinterpret_cast<const uint2*>(c.codes + kv8_tile(c, pg, head, side) + kv8_chunk(t & 63, ch >> 1) +
                                               8 * (ch & 1));
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int e = threadIdx.x + 256 * (i & 7);
    *reinterpret_cast<uint4*>(a.kv_image + img * 2 * kTlTile + (i >> 3) * kTlTile + tile_chunk(e >> 4, e & 15)) =
        eight_codes<FMT>(raw[i]);
  }
}

template <int FMT, bool CONV>
__global__ void __launch_bounds__(CONV ? kTlConvThreads : kTlThreads, 1)
    kv8_tile_kernel(const Kv8View c, const Kv8AttnArgs a) {
  extern __shared__ unsigned char smem_dyn[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023u) & ~uintptr_t(1023u));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kTlBar);
  uint64_t* k_full = bars;          // [2] keys and page scales: bulk copies, or 4 converter warps
  uint64_t* k_empty = bars + 2;     // [2] commit
  uint64_t* v_full = bars + 4;      // [2]
  uint64_t* v_empty = bars + 6;     // [2]
  uint64_t* s_full = bars + 8;      // [2] per query tile, commit
  uint64_t* p_full = bars + 10;     // [2] per query tile, 4 softmax warps
  uint64_t* q_full = bars + 12;     // [2] per query tile, 4 softmax warps
  uint64_t* o_done = bars + 14;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 15);
  float* coef = reinterpret_cast<float*>(smem + kTlCoef);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int head, split, nsplit;
  const int at = kv8_tile_place(a, head, split, nsplit);
  // items of a launch run from the last to the first: with a causal mask the later rows of a sequence see the
  // most keys, and long blocks had better start early
  const int item = a.items - 1 - at % a.items;
  Kv8Item it;
  if (!kv8_find(a.cu, a.lens, c.seqs, a.rows, item, Kv8TileItems{a.group}, it)) return;
  const int b = it.b, tile = it.idx, r0 = it.r0, n = it.n;
  const int len = kv8_length(c, a, it.len);
  const int row_first = tile * 2 * kTlRows;
  const int nrows = min(2 * kTlRows, n * a.group - row_first);
  // 128-key steps of either query tile, and the ones of this split
  int steps[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int last = min(nrows, (t + 1) * kTlRows) - 1;
    const int vis = last >= t * kTlRows ? min(len, kv8_visible(a.causal, len, n, (row_first + last) / a.group)) : 0;
    steps[t] = (vis + kTlKeys - 1) / kTlKeys;
  }
  const int all = max(steps[0], steps[1]);
  const int per = (all + nsplit - 1) / nsplit;
  const int j0 = split * per, j1 = min(all, j0 + per);
  const int cnt = max(0, j1 - j0);
  int cnt_t[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) cnt_t[t] = max(0, min(j1, steps[t]) - j0);

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], CONV ? 4 : 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], CONV ? 4 : 1);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&q_full[i], 4);
    }
    mbar_init(o_done, 1);
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  if (warp >= 12) {
    // ------------------------------------------------------------ converters
    // a warp takes 32 tokens of a step (half a page); a lane, 16 channels of 8 of them
    if (CONV) {
      reg_dec<104>();
      const int w4 = warp - 12;
      uint4 raw_k[8], raw_v[8];                                  // a step ahead
      float2 sc = make_float2(1.f, 0.f);
      auto fetch = [&](int side, int j, uint4 (&raw)[8]) {
        const int p = (j0 + j) * 2 + (w4 >> 1);
        const int held = len - p * kKv8Page;                     // tokens of the page
        const int page = held > 0 ? kv8_page(c, b, p) : -1;
        const uint8_t* src = page >= 0 ? c.codes + kv8_tile(c, page, head, side) : nullptr;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int row = 32 * (w4 & 1) + 8 * (i >> 1) + (lane >> 2);
          const int ch = (lane & 3) + 4 * (i & 1);
          raw[i] = make_uint4(0u, 0u, 0u, 0u);
          if (src && row < held) raw[i] = *reinterpret_cast<const uint4*>(src + kv8_chunk(row, ch));
        }
        if (side == 0) {
          sc = make_float2(1.f, 0.f);
          if (page >= 0) sc = *reinterpret_cast<const float2*>(c.scales + kv8_scale(c, page, head, 0));
        }
      };
      auto put = [&](int side, int j, const uint4 (&raw)[8]) {
        unsigned char* dst = smem + (side ? kTlV : kTlK) + (j & 1) * kTlTile;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          store_codes<FMT>(dst, 32 * w4 + 8 * (i >> 1) + (lane >> 2), (lane & 3) + 4 * (i & 1), raw[i]);
      };
      if (cnt > 0) {
        fetch(0, 0, raw_k);
        fetch(1, 0, raw_v);
      }
      for (int j = 0; j < cnt; ++j) {
        const uint32_t par = ((j >> 1) & 1) ^ 1;
        if (!__all_sync(0xffffffffu, mbar_wait(&k_empty[j & 1], par))) break;
        put(0, j, raw_k);
        // Slot j % 4 was last read for step j - 4, whose P V (awaited before its K stage came free for step j - 2)
        // follows that softmax.
        if ((w4 & 1) == 0 && lane == 0)
          *reinterpret_cast<float4*>(smem + kTlScale + (j & 3) * 32 + (w4 >> 1) * 16) = page_scales(sc);
        if (j + 1 < cnt) fetch(0, j + 1, raw_k);
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&k_full[j & 1]);
        if (!__all_sync(0xffffffffu, mbar_wait(&v_empty[j & 1], par))) break;
        put(1, j, raw_v);
        if (j + 1 < cnt) fetch(1, j + 1, raw_v);
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_full[j & 1]);
      }
    }
  } else if (warp >= 8) {
    reg_dec<CONV ? 40 : 56>();
    if (warp == 8 && cnt > 0) {
      // ------------------------------------------------------------ MMA issuer
      const uint32_t lead = elect_one();
      constexpr uint32_t id_qk = idesc_f16(kTlRows, kTlKeys);
      constexpr uint32_t id_pv = idesc_f16(kTlRows, kKv8Dim) | kIdescBMn;
      const uint64_t q_desc = smem_desc_kmajor(smem_u32(smem), 128);
      const uint64_t k_desc = smem_desc_kmajor(smem_u32(smem + kTlK), 128);
      const uint64_t v_desc = smem_desc_mnmajor(smem_u32(smem + kTlV), 16384, 1024);
      auto wait_warp = [](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity)) != 0;
      };
      auto issue_qk = [&](int t, int j) {
        const uint64_t qd = q_desc + (uint32_t)t * (kTlTile >> 4), kd = k_desc + (uint32_t)(j & 1) * (kTlTile >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = ((uint32_t)(kk >> 2) * 16384u + (uint32_t)(kk & 3) * 32u) >> 4;
          mma_f16_ss_if(lead, tmem + t * kTlKeys, qd + off, kd + off, id_qk, kk > 0);
        }
        tc_commit_if(lead, &s_full[t]);
      };
      // A wait costs about 100 cycles even when there is nothing to wait for, and the tensor core's queue is short:
      // every wait stands behind eight products that are still running.
      bool ok = wait_warp(&k_full[0], 0);
      if (ok) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          ok = ok && wait_warp(&q_full[t], 0);
          tc_fence_after();
          if (ok && cnt_t[t] > 0) issue_qk(t, 0);
        }
        tc_commit_if(lead, &k_empty[0]);
        ok = ok && wait_warp(&v_full[0], 0);
      }
      for (int j = 0; j < cnt && ok; ++j) {
        const bool more = j + 1 < cnt;
        bool k_ready = false, v_ready = false;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (j >= cnt_t[t]) continue;
          if (!wait_warp(&p_full[t], j & 1)) { ok = false; break; }
          tc_fence_after();
          const uint64_t vd = v_desc + (uint32_t)(j & 1) * (kTlTile >> 4);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_f16_ts_if(lead, tmem + 256 + t * kKv8Dim, tmem + t * kTlKeys + 8 * kk, vd + kk * (2048 >> 4), id_pv,
                          (j > 0 || kk > 0) ? 1u : 0u);
          if (more && !k_ready) {
            if (!wait_warp(&k_full[(j + 1) & 1], ((j + 1) >> 1) & 1)) { ok = false; break; }
            k_ready = true;
            tc_fence_after();
          } else if (more && !v_ready) {
            if (!wait_warp(&v_full[(j + 1) & 1], ((j + 1) >> 1) & 1)) { ok = false; break; }
            v_ready = true;
          }
          if (j + 1 < cnt_t[t]) issue_qk(t, j + 1);
        }
        if (!ok) break;
        tc_commit_if(lead, &v_empty[j & 1]);
        if (more) {
          tc_commit_if(lead, &k_empty[(j + 1) & 1]);
          if (!v_ready && !wait_warp(&v_full[(j + 1) & 1], ((j + 1) >> 1) & 1)) ok = false;
        }
      }
      tc_commit_if(lead, o_done);
      mbar_wait(o_done, 0, 100000000ull);
    } else if (!CONV && warp == 9 && lane == 0) {
      // ------------------------------------------------------------ loader
      bool ok = true;
      for (int j = 0; j < cnt && ok; ++j) {
        const int st = j & 1;
        const uint32_t par = ((j >> 1) & 1) ^ 1;
        const int64_t img = ((int64_t)b * a.image_steps + j0 + j) * c.heads + head;
        const uint8_t* src = a.kv_image + img * 2 * kTlTile;
        if (!mbar_wait(&k_empty[st], par)) { ok = false; break; }
        // The page scales come with the keys, in slot j % 4: last read for step j - 4, whose P V (awaited before its
        // K stage came free for step j - 2) follows that softmax.
        mbar_arrive_expect_tx(&k_full[st], kTlTile + 32);
        bulk_load(smem + kTlScale + (j & 3) * 32, a.kv_scale + img * 2, 32, &k_full[st]);
        bulk_load(smem + kTlK + st * kTlTile, src, kTlTile / 2, &k_full[st]);
        bulk_load(smem + kTlK + st * kTlTile + kTlTile / 2, src + kTlTile / 2, kTlTile / 2, &k_full[st]);
        if (!mbar_wait(&v_empty[st], par)) { ok = false; break; }
        mbar_arrive_expect_tx(&v_full[st], kTlTile);
        bulk_load(smem + kTlV + st * kTlTile, src + kTlTile, kTlTile / 2, &v_full[st]);
        bulk_load(smem + kTlV + st * kTlTile + kTlTile / 2, src + kTlTile + kTlTile / 2, kTlTile / 2, &v_full[st]);
      }
      if (!ok) {   // copies still in flight land in this block's shared memory
        const uint64_t t = globaltimer_ns();
        while (globaltimer_ns() - t < 200000ull) {}
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    reg_inc<CONV ? 184 : 224>();
    // First the queries: bf16 rows to fp16 tiles, 16 lanes a row, a warp the 32 rows it will work on.  All loads
    // first, and one division a lane (a load and two divisions a row in two rounds took 9600 cycles, an eighth of a
    // block of a ragged prompt).
    {
      const int ch = lane & 15;
      uint4 w[16];
      const int rr0 = row_first + 32 * warp + (lane >> 4);
      int tok = rr0 / a.group, gq = rr0 - tok * a.group;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        w[i] = make_uint4(0u, 0u, 0u, 0u);
        if (32 * warp + 2 * i + (lane >> 4) < nrows)
          w[i] = __ldg(reinterpret_cast<const uint4*>(a.q + (int64_t)(r0 + tok) * a.ldq +
                                                      (int64_t)(head * a.group + gq) * kKv8Dim + 8 * ch));
        gq += 2;
        while (gq >= a.group) {
          gq -= a.group;
          ++tok;
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int r = 32 * warp + 2 * i + (lane >> 4);
        const uint32_t ws[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        uint32_t amax = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) amax = __vmaxu2(amax, ws[e] & 0x7FFF7FFFu);
        amax = max(amax & 0xFFFFu, amax >> 16);
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, off));
        float f, inv;
        kv8_row_scale(amax, f, inv);
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          h[e] = half2_bits(__uint_as_float(ws[e] << 16) * f, __uint_as_float(ws[e] & 0xFFFF0000u) * f);
        const uint4 hv = make_uint4(h[0], h[1], h[2], h[3]);
        const int qt = r >> 7, tr = r & 127;
        *reinterpret_cast<uint4*>(smem + qt * kTlTile + tile_chunk(tr, ch)) = hv;
        if (ch == 0) coef[r] = inv * a.scale_log2;
        if (a.q_image && split == 0) {
          const int64_t img = ((int64_t)head * a.items + item) * 2 + qt;
          *reinterpret_cast<uint4*>(a.q_image + img * kTlTile + tile_chunk(tr, ch)) = hv;
          if (ch == 0) a.q_rows[img * 3 * kTlRows + tr] = inv * a.scale_log2;
        }
      }
    }
    fence_async_shared();
    __syncwarp();
    if (lane == 0) mbar_arrive(&q_full[warp >> 2]);
    const int t = warp >> 2;
    const int r = tid;                                          // row of the block
    const bool live = r < nrows;
    const int rr = row_first + r;
    const int lim = live ? kv8_visible(a.causal, len, n, rr / a.group) : 0;
    const int min_lim = __reduce_min_sync(0xffffffffu, live ? lim : 0x7FFFFFFF);
    const float cq = coef[r];
    const uint32_t lane_addr = (32u * (uint32_t)(warp & 3)) << 16;
    const uint32_t t_s = tmem + lane_addr + t * kTlKeys, t_o = tmem + lane_addr + 256 + t * kKv8Dim;
    auto wait_warp = [](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity)) != 0;
    };
    float m_run = -INFINITY, l_run = 0.f;
    bool ok = true;
    const int mine = t ? cnt_t[1] : cnt_t[0];
    for (int j = 0; j < mine; ++j) {
      if (!wait_warp(&s_full[t], j & 1)) { ok = false; break; }
      tc_fence_after();
      uint32_t s[128];
#pragma unroll
      for (int q = 0; q < 4; ++q) tmem_ld32(t_s + 32 * q, s + 32 * q);
      const float4 sc0 = *reinterpret_cast<const float4*>(smem + kTlScale + (j & 3) * 32);
      const float4 sc1 = *reinterpret_cast<const float4*>(smem + kTlScale + (j & 3) * 32 + 16);
      const float c0 = cq * sc0.x, c1 = cq * sc1.x;
      const int k0 = (j0 + j) * kTlKeys;
      const bool full = min_lim >= k0 + kTlKeys;                // the warp's rows all see every key of the step
      const int nv = lim - k0;
      tmem_wait_ld();
#pragma unroll
      for (int q = 0; q < 8; ++q) tmem_reg_fence(*reinterpret_cast<uint32_t(*)[16]>(s + 16 * q));
      if (!full) {
#pragma unroll
        for (int e = 0; e < 128; ++e)
          if (e >= nv) s[e] = 0xFF800000u;                      // -inf
      }
      float mx[8];                                              // four chains per page
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const int e = (x >> 2) * 64 + (x & 3);
        mx[x] = max3(__uint_as_float(s[e]), __uint_as_float(s[e + 4]), __uint_as_float(s[e + 8]));
      }
#pragma unroll
      for (int e = 12; e < 60; e += 8)
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const int at = (x >> 2) * 64 + e + (x & 3);
          mx[x] = max3(mx[x], __uint_as_float(s[at]), __uint_as_float(s[at + 4]));
        }
#pragma unroll
      for (int x = 0; x < 8; ++x) mx[x] = fmaxf(mx[x], __uint_as_float(s[(x >> 2) * 64 + 60 + (x & 3)]));
      const float mx0 = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]), mx1 = max3(fmaxf(mx[4], mx[5]), mx[6], mx[7]);
      const float mt = fmaxf(mx0 > -INFINITY ? fmaxf(fmaf(mx0, c0, sc0.y), sc0.w) : -INFINITY,
                             mx1 > -INFINITY ? fmaxf(fmaf(mx1, c1, sc1.y), sc1.w) : -INFINITY);
      const bool move = mt > m_run + kKv8Lazy;
      if (__any_sync(0xffffffffu, move)) {
        const float f = move ? ex2(m_run - mt) : 1.f;
        if (j > 0) {       // O holds steps 0 .. j - 1: their P V precede S of step j on the tensor core
#pragma unroll 1
          for (int q = 0; q < 8; ++q) {
            uint32_t ov[16];
            tmem_ld16(t_o + 16 * q, ov);
#pragma unroll
            for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * f);
            tmem_st16(t_o + 16 * q, ov);
          }
          tmem_wait_st();
        }
        l_run *= f;
        if (move) m_run = mt;
      }
      const float m_use = m_run > -INFINITY ? m_run : 0.f;
      const float b0 = sc0.y - m_use, b1 = sc1.y - m_use;
      const uint64_t cc[2] = {pack_f32(c0, c0), pack_f32(c1, c1)}, bb[2] = {pack_f32(b0, b0), pack_f32(b1, b1)};
      uint64_t lp[4] = {0ull, 0ull, 0ull, 0ull};                 // two pairs of partial sums per page
      // (a score factor of zero, from a vanishing query, would turn a masked -inf into a NaN: masked keys get p = 0)
      auto probs = [&](auto all_seen) {
#pragma unroll
        for (int e = 0; e < 128; e += 2) {
          const int h = e >> 6;
          float x, y;
          unpack_f32(fma_f32x2(pack_f32(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), cc[h], bb[h]), x, y);
          if ((e >> 1) % 4 == 3) {
            ex2_poly(x, y);
          } else {
            x = ex2(x);
            y = ex2(y);
          }
          if (!decltype(all_seen)::value) {
            x = e < nv ? x : 0.f;
            y = e + 1 < nv ? y : 0.f;
          }
          lp[2 * h + ((e >> 1) & 1)] = add_f32x2(lp[2 * h + ((e >> 1) & 1)], pack_f32(x, y));
          s[e >> 1] = half2_bits(x, y);
          if (e == 62) tmem_st32(t_s, s);
        }
      };
      if (full) probs(std::true_type{});
      else probs(std::false_type{});
      tmem_st32(t_s + 32, s + 32);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x, y;
        unpack_f32(add_f32x2(lp[2 * h], lp[2 * h + 1]), x, y);
        l_run = fmaf(x + y, h ? sc1.z : sc0.z, l_run);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[t]);
    }
    // output: O / L, or the split's O, m and L
    const bool have = mine > 0;
    // A block whose rows see no key has no products to wait for, but the rows below are staged over queries that the
    // tile's other warps may still be writing.
    ok = ok && wait_warp(&q_full[t], 0) && (cnt == 0 || wait_warp(o_done, 0));
    tc_fence_after();
    if (ok) {
      const int gq = rr % a.group, qh = head * a.group + gq;
      const int64_t tok = r0 + rr / a.group;
      const int64_t fr = tok * a.q_heads + qh;
      const float inv = kv8_inverse(m_run, l_run);
      const bool whole = nsplit == 1;
      const int64_t slot = ((int64_t)(at - a.whole) * 2 * kTlRows + r) * nsplit + split;
      if (live) {
        if (!whole) a.part_ml[slot] = make_float2(m_run, l_run);
        else if (a.stats) a.stats[fr] = make_float2(m_run > -INFINITY ? m_run : 0.f, inv);
      }
      // Whole rows go through 8 KB of the query tile's memory, which holds rows of other warps of the tile (all written
      // by now, and read by the tensor core for the last time):
      // written a row a thread, they leave two rows an instruction (straight to global memory they took 5200 cycles).
      unsigned char* stage = smem + 32 * warp * 256;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t ov[32];
        if (have) {
          tmem_ld32(t_o + 32 * q, ov);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) ov[e] = 0u;
        }
        if (whole) {
#pragma unroll
          for (int e8 = 0; e8 < 4; ++e8) {
            uint32_t w[4];
#pragma unroll
            for (int e2 = 0; e2 < 4; ++e2) {
              const __nv_bfloat162 p2 = __floats2bfloat162_rn(__uint_as_float(ov[8 * e8 + 2 * e2]) * inv,
                                                              __uint_as_float(ov[8 * e8 + 2 * e2 + 1]) * inv);
              w[e2] = *reinterpret_cast<const uint32_t*>(&p2);
            }
            *reinterpret_cast<uint4*>(stage + lane * 256 + (((4 * q + e8) ^ (lane & 7)) << 4)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else if (have && live) {
          uint4* dst = reinterpret_cast<uint4*>(a.part_o + slot * kKv8Dim + 32 * q);
#pragma unroll
          for (int e4 = 0; e4 < 8; ++e4) dst[e4] = make_uint4(ov[4 * e4], ov[4 * e4 + 1], ov[4 * e4 + 2], ov[4 * e4 + 3]);
        }
      }
      if (whole) {
        __syncwarp();
        const int64_t at = tok * a.ldo + (int64_t)qh * kKv8Dim;      // of this lane's row
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int x = 2 * i + (lane >> 4), ch = lane & 15;
          const int64_t to = __shfl_sync(0xffffffffu, at, x);
          if (32 * warp + x < nrows)
            *reinterpret_cast<uint4*>(a.o + to + 8 * ch) =
                *reinterpret_cast<const uint4*>(stage + x * 256 + ((ch ^ (x & 7)) << 4));
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the splits of the pairs that have them: a warp a row.
__global__ void __launch_bounds__(256) kv8_tile_combine_kernel(const Kv8AttnArgs a) {
  const int at = a.whole + (int)blockIdx.x, r = (int)(blockIdx.y * 8 + (threadIdx.x >> 5));
  Kv8Item it;
  if (!kv8_find(a.cu, a.lens, a.seqs, a.rows, a.items - 1 - at % a.items, Kv8TileItems{a.group}, it)) return;
  const int rr = it.idx * 2 * kTlRows + r;
  if (rr >= it.n * a.group) return;
  kv8_join(a, (int64_t)blockIdx.x * 2 * kTlRows + r, it.r0 + rr / a.group, at / a.items * a.group + rr % a.group);
}

// ---------------------------------------------------------------------------
// Weights of the keys, many query rows
// ---------------------------------------------------------------------------
// A block per (128 keys, key/value head, sequence) computes S^T = K Q^T for every
// query tile that sees them, the keys on the TMEM lanes: a thread owns a key and
// adds 2^(x - m) / L = 2^(x + c) over the columns, c = -(m + log2 L) from the rows'
// final m and L, in a fixed order and without atomics.  The query tiles come from
// the images the attention left behind (one 32 KB bulk copy each), and so do the rows'
// factors, constants and numbers of keys, which kv8_rows_kernel completes (gathered by
// a warp of this kernel they took 4700 cycles a tile, most of its time).  Bound by the
// special-function unit (1024 cycles a 128 x 128 tile, Q.K^T 512); the columns'
// factors and constants are broadcast reads, four columns at a time.  Two blocks an
// SM, so that one sums while the other waits.  Under a causal mask the first keys see
// every tile and the last ones one: with few blocks the tiles of each are cut into
// `parts`, whose sums kv8_weigh_add_kernel adds in order.
// Measured: two causal prompts of 3001 and 1954 tokens, 48 heads in groups of 4: 155 us
// for this pass, of 380 with the attention; about six blocks an SM, half or twice as
// many being 1 to 3% slower, and a polynomial for part of the exponentials no faster.
//   warps 0-3, 4-7  sums, query tiles in turn;  warp 8  producer;  warp 9  TMEM owner and MMA issuer.
namespace {
constexpr int kWgThreads = 320;
constexpr uint32_t kWgQ = kTlTile;                                  // after the keys: 2 query tiles
constexpr uint32_t kWgRowsBytes = 3 * kTlRows * 4;                  // (factor, constant, keys seen) of 128 rows
constexpr uint32_t kWgPar = kWgQ + 2 * kTlTile;                     // 4 slots of those
constexpr uint32_t kWgSum = kWgPar + 4 * kWgRowsBytes;              // 128 floats
constexpr uint32_t kWgBar = kWgSum + 512;
constexpr uint32_t kWgSmem = kWgBar + 256 + 1024;
}  // namespace

// The rows' constants c = -(m + log2 L) and numbers of keys seen, beside their factors: [heads][items][2][3][128].
__global__ void __launch_bounds__(2 * kTlRows) kv8_rows_kernel(const Kv8View c, const Kv8AttnArgs a) {
  Kv8Item it;
  if (!kv8_find(a.cu, a.lens, c.seqs, a.rows, blockIdx.x, Kv8TileItems{a.group}, it)) return;
  const int tile = it.idx, r0 = it.r0, n = it.n;
  const int len = kv8_length(c, a, it.len);
  const int head = blockIdx.y;
  const int rr = tile * 2 * kTlRows + threadIdx.x;
  float k = -INFINITY;                          // no such row, or one without keys: 2^(-inf) = 0
  int seen = 0;
  if (rr < n * a.group) {
    const int i = rr / a.group;
    const float2 s = a.stats[(int64_t)(r0 + i) * a.q_heads + head * a.group + (rr - i * a.group)];
    if (s.y != 0.f) k = log2f(s.y) - s.x;
    seen = kv8_visible(a.causal, len, n, i);
  }
  const int64_t img = ((int64_t)head * a.items + blockIdx.x) * 2 + (threadIdx.x >> 7);
  float* rows = a.q_rows + img * 3 * kTlRows + (threadIdx.x & 127);
  rows[kTlRows] = k;
  reinterpret_cast<int*>(rows)[2 * kTlRows] = seen;
}

template <int FMT>
__global__ void __launch_bounds__(kWgThreads, 2)
    kv8_weigh_tile_kernel(const Kv8View c, const Kv8AttnArgs a, const float* w_in, float* w_out, int64_t w_seq,
                          int64_t w_head, float* part_out, int parts) {
  extern __shared__ unsigned char smem_dyn[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023u) & ~uintptr_t(1023u));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kWgBar);
  uint64_t* q_full = bars;          // [2] bulk copies
  uint64_t* q_empty = bars + 2;     // [2] commit
  uint64_t* s_full = bars + 6;      // [2] commit
  uint64_t* s_empty = bars + 8;     // [2] 4 summing warps
  uint64_t* drain = bars + 10;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 12);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the key block is the slowest index: under a causal mask the first ones take longest and start first
  const int each = parts * c.heads * c.seqs;
  const int k0 = (int)(blockIdx.x / each) * kTlKeys;
  int rest = (int)(blockIdx.x % each);
  const int part = rest % parts;
  rest /= parts;
  const int head = rest % c.heads, b = rest / c.heads;
  const int len = kv8_len(c, a, b);
  if (k0 >= len) return;
  // first item (256 query rows) of this sequence in the images: the items of the sequences in front of it
  int item0 = 0;
  for (int i = lane; i < b; i += 32) {
    int x0, xn;
    kv8_rows(a.cu, i, a.rows, x0, xn);
    item0 = min(a.items, item0 + Kv8TileItems{a.group}(xn, 0));
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) item0 += __shfl_xor_sync(0xffffffffu, item0, off);
  int r0, n;
  kv8_rows(a.cu, b, a.rows, r0, n);
  const int total = n * a.group;
  const int i_first = a.causal ? max(0, k0 - (len - n)) : 0;          // first query token that sees key k0
  const int seen0 = min(i_first, n) * a.group / kTlRows;
  const int nseen = max(0, (total + kTlRows - 1) / kTlRows - seen0);
  const int per = (nseen + parts - 1) / parts;
  const int tile0 = seen0 + part * per;
  // offsets that are not in order, so that sequences overlap, make more items than there are images
  const int held = 2 * max(0, a.items - item0) - tile0;
  const int mine = max(0, min(per, nseen - part * per));
  const int cnt = max(0, min(mine, held));
  if (cnt < mine && tid == 0) record_refusal();

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 4);
    }
    mbar_init(drain, 1);
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_holder, 256);
    tmem_relinquish();
    tc_fence_before();
  }
  // the block's keys: 128 tokens x 8 chunks
  {
    uint4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = tid + i * kWgThreads, t = e >> 3;
      w[i] = make_uint4(0u, 0u, 0u, 0u);
      if (e < kTlKeys * 8 && k0 + t < len) {
        const int page = kv8_page(c, b, (k0 + t) / kKv8Page);
        if (page >= 0)
          w[i] = *reinterpret_cast<const uint4*>(c.codes + kv8_tile(c, page, head, 0) + kv8_chunk(t & 63, e & 7));
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = tid + i * kWgThreads;
      if (e < kTlKeys * 8) store_codes<FMT>(smem, e >> 3, e & 7, w[i]);
    }
  }
  fence_async_shared();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  if (warp == 8) {
    if (lane == 0) {
      bool ok = true;
      for (int i = 0; i < cnt && ok; ++i) {
        const int qt = tile0 + i, st = i & 1;
        const int64_t img = ((int64_t)head * a.items + item0 + (qt >> 1)) * 2 + (qt & 1);
        if (!mbar_wait(&q_empty[st], ((i >> 1) & 1) ^ 1)) { ok = false; break; }
        // Row slot i % 4 held tile i - 4, whose sums were awaited before the products of tile i - 2, which freed
        // this stage.
        mbar_arrive_expect_tx(&q_full[st], kTlTile + kWgRowsBytes);
        bulk_load(smem + kWgQ + st * kTlTile, a.q_image + img * kTlTile, kTlTile, &q_full[st]);
        bulk_load(smem + kWgPar + (i & 3) * kWgRowsBytes, a.q_rows + img * 3 * kTlRows, kWgRowsBytes, &q_full[st]);
      }
      if (!ok) {   // copies still in flight land in this block's shared memory
        const uint64_t t = globaltimer_ns();
        while (globaltimer_ns() - t < 200000ull) {}
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    const uint32_t lead = elect_one();
    constexpr uint32_t id = idesc_f16(kTlKeys, kTlRows);
    const uint64_t k_desc = smem_desc_kmajor(smem_u32(smem), 128);
    const uint64_t q_desc = smem_desc_kmajor(smem_u32(smem + kWgQ), 128);
    for (int i = 0; i < cnt; ++i) {
      const int st = i & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(&q_full[st], (i >> 1) & 1) && mbar_wait(&s_empty[st], ((i >> 1) & 1) ^ 1)))
        break;
      tc_fence_after();
      const uint64_t qd = q_desc + (uint32_t)st * (kTlTile >> 4);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const uint32_t off = ((uint32_t)(kk >> 2) * 16384u + (uint32_t)(kk & 3) * 32u) >> 4;
        mma_f16_ss_if(lead, tmem + st * 128, k_desc + off, qd + off, id, kk > 0);
      }
      tc_commit_if(lead, &s_full[st]);
      tc_commit_if(lead, &q_empty[st]);
    }
    tc_commit_if(lead, drain);
    mbar_wait(drain, 0, 100000000ull);
    __syncwarp();
  }
  float acc = 0.f;
  bool ok = true;
  if (warp < 8) {
    const int key = k0 + 32 * (warp & 3) + lane;
    float sk = 1.f;
    bool there = true;                                         // the key's page is one of the pool
    if (key < len) {
      const int page = kv8_page(c, b, key / kKv8Page);
      there = page >= 0;
      if (there) sk = c.scales[kv8_scale(c, page, head, 0)];
    }
    const uint64_t sk2 = pack_f32(sk, sk);
    const uint32_t lane_addr = (32u * (uint32_t)(warp & 3)) << 16;
    const int st = warp >> 2;                                  // this warpgroup's slot and TMEM buffer
    for (int i = st; i < cnt; i += 2) {
      const float* par = reinterpret_cast<const float*>(smem + kWgPar) + (i & 3) * 3 * kTlRows;
      if (!__all_sync(0xffffffffu, mbar_wait(&s_full[st], (i >> 1) & 1))) {
        ok = false;
        break;
      }
      tc_fence_after();
      // rows come in the order of their tokens: if the tile's first row sees the block's last key, all do (rows behind
      // the last have c = -inf)
      const bool all_seen = reinterpret_cast<const int*>(par)[2 * kTlRows] >= k0 + kTlKeys;
      uint64_t sums[2] = {0ull, 0ull};
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        uint32_t s[32];
        tmem_ld32(tmem + lane_addr + st * 128 + 32 * q, s);
        tmem_wait_ld();
        tmem_reg_fence(*reinterpret_cast<uint32_t(*)[16]>(s));
        tmem_reg_fence(*reinterpret_cast<uint32_t(*)[16]>(s + 16));
        const float4* f4 = reinterpret_cast<const float4*>(par + 32 * q);
        const float4* k4 = reinterpret_cast<const float4*>(par + kTlRows + 32 * q);
        const int4* n4 = reinterpret_cast<const int4*>(reinterpret_cast<const int*>(par) + 2 * kTlRows + 32 * q);
        auto sum = [&](auto every) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 f = f4[e >> 2], k = k4[e >> 2];
            uint64_t x01 = fma_f32x2(fma_f32x2(pack_f32(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), sk2, 0ull),
                                     pack_f32(f.x, f.y), pack_f32(k.x, k.y));
            uint64_t x23 = fma_f32x2(fma_f32x2(pack_f32(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])), sk2, 0ull),
                                     pack_f32(f.z, f.w), pack_f32(k.z, k.w));
            float p[4];
            unpack_f32(x01, p[0], p[1]);
            unpack_f32(x23, p[2], p[3]);
#pragma unroll
            for (int x = 0; x < 4; ++x)
              p[x] = ex2(p[x]);
            if (!decltype(every)::value) {
              const int4 v = n4[e >> 2];
              p[0] = key < v.x ? p[0] : 0.f;
              p[1] = key < v.y ? p[1] : 0.f;
              p[2] = key < v.z ? p[2] : 0.f;
              p[3] = key < v.w ? p[3] : 0.f;
            }
            sums[0] = add_f32x2(sums[0], pack_f32(p[0], p[1]));
            sums[1] = add_f32x2(sums[1], pack_f32(p[2], p[3]));
          }
        };
        if (all_seen) sum(std::true_type{});
        else sum(std::false_type{});
      }
      float x, y;
      unpack_f32(add_f32x2(sums[0], sums[1]), x, y);
      acc += x + y;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_empty[st]);
    }
    if (!there) acc = 0.f;
    if (warp >= 4) reinterpret_cast<float*>(smem + kWgSum)[tid - 128] = acc;
  }
  tc_fence_before();
  __syncthreads();
  if (warp < 4 && ok && k0 + tid < len) {
    acc += reinterpret_cast<const float*>(smem + kWgSum)[tid];
    if (part_out) {
      part_out[(((int64_t)part * c.seqs + b) * c.heads + head) * a.max_len + k0 + tid] = acc;
    } else {
      const int64_t at = b * w_seq + head * w_head + k0 + tid;
      w_out[at] = w_in[at] + acc;
    }
  }
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// weights_out = weights_in + the parts' sums, in order: a thread per key.
__global__ void __launch_bounds__(256)
    kv8_weigh_add_kernel(const Kv8View c, const Kv8AttnArgs a, const float* w_in, float* w_out, int64_t w_seq,
                         int64_t w_head, const float* part_out, int parts) {
  const int b = blockIdx.z, head = blockIdx.y, t = blockIdx.x * 256 + threadIdx.x;
  if (t >= kv8_len(c, a, b)) return;
  float acc = 0.f;
  for (int r = 0; r < parts; ++r) acc += part_out[(((int64_t)r * c.seqs + b) * c.heads + head) * a.max_len + t];
  const int64_t at = b * w_seq + head * w_head + t;
  w_out[at] = w_in[at] + acc;
}

// ---------------------------------------------------------------------------
// Host launchers
// ---------------------------------------------------------------------------
// How a call runs, from its sizes alone (the workspace is sized by the same rule).
struct Kv8Plan {
  int nq;              // streaming kernel with 8 nq rows a block; 0: the tile kernel
  int items, nsplit;
  int whole;           // tile kernel: (head, item) pairs whose keys are not split
  bool prepare;        // operand images
  int image_steps;     // 128-key steps of a sequence in them
  int parts;           // parts of a key block's query tiles
  int64_t part_o, part_ml, stats, logits, q_image, q_rows, kv_image, kv_scale, w_part, bytes;   // workspace offsets, -1 for none
  int64_t logit_ld;
};

// Query rows that share a key/value head, per sequence, up to which the streaming kernel runs, 16 to a block (32
// rows over 3000 keys x 24 x 8: 84 us against the tile kernel's 137; 44 rows: 92 against 100).
constexpr int kStreamRows = 40;
// Operand images are made when a key is used by at least this many blocks on average, and fit in this much.
constexpr int kPrepareItems = 3;
constexpr int64_t kPrepareBytes = (int64_t)1 << 31;

Kv8Plan kv8_plan(int seqs, int heads, int q_heads, int rows, int max_len, bool weigh) {
  Kv8Plan p{};
  const int group = q_heads / heads;
  const int64_t packed = (int64_t)rows * group;
  p.nq = packed <= 8 * (int64_t)seqs ? 1 : packed <= (int64_t)kStreamRows * seqs ? 2 : 0;
  const int unit = p.nq ? 8 * p.nq : 2 * kTlRows;
  // sequences that can have queries (one where there is no row at all: it divides below)
  const int busy = std::max(1, std::min(seqs, rows));
  // the most that sequences of at least one row each can have
  p.items = (int)std::min<int64_t>(packed, std::max<int64_t>(packed - busy, 0) / unit + busy);
  const int64_t blocks = (int64_t)p.items * heads;
  const int steps = std::max(1, (max_len + kTlKeys - 1) / kTlKeys);
  p.nsplit = 1;
  p.whole = (int)blocks;
  if (p.nq) {
    // A split costs its partial result: the streaming kernel splits into four blocks an SM where there are fewer than
    // two, at least eight 128-key steps each (3 sequences of up to 120001 keys: 104 us, 115 with two a SM; 24
    // sequences x 8 heads x 2 blocks: 55 us unsplit, 67 split in two).
    if (blocks > 0 && blocks < 148 * 2)
      p.nsplit = (int)std::max<int64_t>(1, std::min<int64_t>({(148 * 4 + blocks - 1) / blocks, steps / 8, 64}));
  } else if (blocks <= 148 || 2 * (int64_t)rows <= (int64_t)max_len * busy) {
    // Blocks of the tile kernel that last alike (where a sequence's queries are few beside its keys) run in waves.
    // Those of a last, partly filled wave are split when that is shorter by an estimate in steps: a block's setup
    // counts as four, the join as two and 1/32 for every split (4096 queries over 16384 keys x 24 heads, 384 blocks:
    // 739 us whole, 705 with the last 88 split in three; 1024 queries, 96 blocks: 290-320 us whole, 262-275 split in
    // three).
    const int tail = (int)(blocks % 148);
    int64_t best = 32 * (int64_t)(steps + 4);
    for (int k = 2; tail > 0 && k <= std::min(64, steps / 8); ++k) {
      const int64_t cost = 32 * (int64_t)((tail * k + 147) / 148 * ((steps + k - 1) / k + 4) + 2) + tail * k;
      if (cost < best) {
        best = cost;
        p.nsplit = k;
        p.whole = (int)blocks - tail;
      }
    }
  }
  p.image_steps = steps;
  const int64_t images = (int64_t)seqs * steps * heads;
  p.prepare = p.nq == 0 && p.items >= kPrepareItems * (int64_t)busy && images <= kPrepareBytes / (2 * kTlTile);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  const int64_t fr = (int64_t)rows * q_heads;
  const int64_t slots = p.nq ? fr : (blocks - p.whole) * 2 * kTlRows;
  p.part_o = p.nsplit > 1 ? take(slots * p.nsplit * kKv8Dim * 4) : -1;
  p.part_ml = p.nsplit > 1 ? take(slots * p.nsplit * 8) : -1;
  p.stats = weigh ? take(fr * 8) : -1;
  p.logit_ld = (max_len + kKv8Page - 1) / kKv8Page * (int64_t)kKv8Page;
  p.logits = weigh && p.nq ? take(fr * p.logit_ld * 4) : -1;
  p.q_image = weigh && p.nq == 0 ? take((int64_t)heads * p.items * 2 * kTlTile) : -1;
  p.q_rows = weigh && p.nq == 0 ? take((int64_t)heads * p.items * 2 * kTlRows * 12) : -1;
  p.kv_image = p.prepare ? take(images * 2 * kTlTile) : -1;
  p.kv_scale = p.prepare ? take(images * 2 * 16) : -1;
  // parts: at least eight query tiles each, until the blocks fill the device (two an SM) three times over
  p.parts = (int)std::max<int64_t>(
      1, std::min<int64_t>({(148 * 6 + images - 1) / std::max<int64_t>(images, 1), packed / (8 * kTlRows * (int64_t)busy), 8}));
  p.w_part = weigh && p.nq == 0 && p.parts > 1 ? take(p.parts * (int64_t)seqs * heads * max_len * 4) : -1;
  p.bytes = at;
  return p;
}

int64_t kv8_attn_workspace_bytes(int seqs, int heads, int q_heads, int rows, int max_len, bool weigh) {
  return kv8_plan(seqs, heads, q_heads, rows, max_len, weigh).bytes;
}

namespace {
template <int FMT, int NQ>
cudaError_t launch_stream(const dim3& grid, const Kv8View& c, const Kv8AttnArgs& a, cudaStream_t st) {
  using Sh = StreamShape<NQ>;
  static SmemAllowance allowed;
  const cudaError_t e = allowed.raise(kv8_stream_kernel<FMT, NQ>, Sh::kSmem);
  if (e != cudaSuccess) return e;
  kv8_stream_kernel<FMT, NQ><<<grid, Sh::kThreads, Sh::kSmem, st>>>(c, a);
  return cudaSuccess;
}

template <int FMT>
cudaError_t launch_kv8_attn_fmt(const Kv8View& c, const Kv8AttnArgs& a, const Kv8Plan& p, const float* w_in,
                                float* w_out, int64_t w_seq, int64_t w_head, void* work, cudaStream_t st) {
  cudaError_t e;
  if (a.rows > 0) {
    const int split_pairs = p.items * c.heads - p.whole;
    const dim3 grid = p.nq ? dim3(p.items, c.heads, p.nsplit) : dim3(p.whole + split_pairs * p.nsplit);
    if (p.nq) {
      e = p.nq == 1 ? launch_stream<FMT, 1>(grid, c, a, st) : launch_stream<FMT, 2>(grid, c, a, st);
      if (e != cudaSuccess) return e;
    } else {
      if (p.prepare) {
        kv8_prepare_kernel<FMT><<<dim3(p.image_steps, c.heads, c.seqs), 256, 0, st>>>(c, a);
        static SmemAllowance allowed;
        e = allowed.raise(kv8_tile_kernel<FMT, false>, kTlSmem);
        if (e != cudaSuccess) return e;
        kv8_tile_kernel<FMT, false><<<grid, kTlThreads, kTlSmem, st>>>(c, a);
      } else {
        static SmemAllowance allowed;
        e = allowed.raise(kv8_tile_kernel<FMT, true>, kTlSmem);
        if (e != cudaSuccess) return e;
        kv8_tile_kernel<FMT, true><<<grid, kTlConvThreads, kTlSmem, st>>>(c, a);
      }
    }
    if (p.nsplit > 1 && p.nq == 0) {
      kv8_tile_combine_kernel<<<dim3(split_pairs, 2 * kTlRows / 8), 256, 0, st>>>(a);
    } else if (p.nsplit > 1) {
      const int64_t fr = (int64_t)a.rows * a.q_heads;
      kv8_combine_kernel<<<(unsigned)((fr + 7) / 8), 256, 0, st>>>(a);
    }
  }
  if (w_out && a.max_len > 0) {
    if (p.nq) {
      kv8_weigh_logits_kernel<<<dim3((a.max_len + 255) / 256, c.heads, c.seqs), 256, 0, st>>>(c, a, w_in, w_out, w_seq,
                                                                                              w_head);
    } else {
      if (p.items > 0) kv8_rows_kernel<<<dim3(p.items, c.heads), 2 * kTlRows, 0, st>>>(c, a);
      static SmemAllowance allowed;
      e = allowed.raise(kv8_weigh_tile_kernel<FMT>, kWgSmem);
      if (e != cudaSuccess) return e;
      float* part_out = p.w_part < 0 ? nullptr : reinterpret_cast<float*>(static_cast<uint8_t*>(work) + p.w_part);
      kv8_weigh_tile_kernel<FMT><<<(unsigned)((int64_t)p.image_steps * c.heads * c.seqs * p.parts), kWgThreads, kWgSmem,
                                   st>>>(c, a, w_in, w_out, w_seq, w_head, part_out, p.parts);
      if (part_out)
        kv8_weigh_add_kernel<<<dim3((a.max_len + 255) / 256, c.heads, c.seqs), 256, 0, st>>>(c, a, w_in, w_out, w_seq,
                                                                                           w_head, part_out, p.parts);
    }
  }
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_kv8_attn(const Kv8View& c, bool e4m3, const int32_t* lens, const int32_t* cu, const uint16_t* q,
                            int64_t ldq, int rows, int q_heads, bool causal, float scale_log2, int max_len,
                            uint16_t* o, int64_t ldo, const float* w_in, float* w_out, int64_t w_seq, int64_t w_head,
                            void* work, cudaStream_t st) {
  const Kv8Plan p = kv8_plan(c.seqs, c.heads, q_heads, rows, max_len, w_out != nullptr);
  uint8_t* ws = static_cast<uint8_t*>(work);
  auto at = [&](int64_t off) { return off < 0 ? nullptr : ws + off; };
  Kv8AttnArgs a{};
  a.q = q;
  a.ldq = ldq;
  a.o = o;
  a.ldo = ldo;
  a.cu = cu;
  a.lens = lens;
  a.rows = rows;
  a.q_heads = q_heads;
  a.group = q_heads / c.heads;
  a.causal = causal;
  a.seqs = c.seqs;
  a.max_len = max_len;
  a.nsplit = p.nsplit;
  a.whole = p.whole;
  a.items = p.items;
  a.scale_log2 = scale_log2;
  a.part_o = reinterpret_cast<float*>(at(p.part_o));
  a.part_ml = reinterpret_cast<float2*>(at(p.part_ml));
  a.stats = reinterpret_cast<float2*>(at(p.stats));
  a.logits = reinterpret_cast<float*>(at(p.logits));
  a.logit_ld = p.logit_ld;
  a.q_image = at(p.q_image);
  a.q_rows = reinterpret_cast<float*>(at(p.q_rows));
  a.kv_image = at(p.kv_image);
  a.kv_scale = reinterpret_cast<float4*>(at(p.kv_scale));
  a.image_steps = p.image_steps;
  return e4m3 ? launch_kv8_attn_fmt<RBD_CODES_E4M3>(c, a, p, w_in, w_out, w_seq, w_head, work, st)
              : launch_kv8_attn_fmt<RBD_CODES_INT8>(c, a, p, w_in, w_out, w_seq, w_head, work, st);
}

}  // namespace rbd

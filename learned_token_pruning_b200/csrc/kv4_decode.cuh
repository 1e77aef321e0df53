// Decode attention over the paged 4-bit KV cache: for each request the new
// token's query heads over its cached rows,
//     l_c = temp_h ratio_r sm_scale (q_h . k_c) + gain_h bias_c,  out_h = sum_c softmax_c(l) v_c,
// with k_c and v_c the values the 4-bit rows stand for.  A key whose bias is
// -infinity is left out altogether, whatever its row holds; a request without
// keys gets zeros (lse -infinity).
//
// The cache is read once: 2 (D/2 + D/16) bytes per row and KV head, a third of bf16, are the
// floor.  What stands in the way is the work per value, so the products run on the
// tensor cores through the warp-level matrix instruction (m16n8k16, fp16 in, fp32
// out).  Its operands come from registers, where the codes are widened with one
// conversion per two values.  The wide tcgen05 form, keys as its 128 rows and the codes
// taken by it from shared memory as they are, has not been tried.
//
//   Keys and values are the A operand (16 keys or 16 dimensions x 16), the query
//   heads and the weights the B operand (8 columns).  E2M1 codes are exact in
//   fp16, and the scales stay outside: per group of 32 dimensions the scores are
//   accumulated on their own and added up times the key's scale in fp32, and the
//   weights are multiplied by the value row's scale before they are rounded to
//   fp16 (11 bits; fp32 queries carry query and weights as two fp16 parts, 22 bits).
//   Both factors meet a power of two that keeps them in fp16's range: the query one
//   per head (its largest value lands at 2^8), the weights one per head and scale
//   group, the unit: the largest product of a weight and a value scale met so far lands at
//   2^6 or above, so that products down to 2^-20 of it keep their 11 bits.  The unit moves with
//   the softmax's reference and follows the products, not the scales: a huge row without weight
//   must not cost the others their digits.
//   The 8 columns hold HP heads (2, 4 or 8) times 8 / HP scale groups: with two
//   heads, one B operand serves all four groups of D = 128.  A lane reads the
//   accumulator columns of its own group and leaves the others.
//
// Work split: the (request, KV head, 64-key tile) units are laid out in that
// order and cut into runs of equal cost, one per warp, so ragged batches are balanced to a tile.
// Every warp streams its own run through a ring in shared memory by bulk copies
// (a page holds a head's rows contiguously; no barrier between warps), keeps its own
// online softmax, and writes a result directly when a (request, head) lies
// inside its run.  Pieces of longer ones are merged per CTA in shared memory and,
// where they cross CTAs, by a second small kernel, always in order of position:
// reruns are bit-identical.
//
// Measured (16 + 8 heads of 128, bf16 queries, both kernels): 131137 rows of one request, pages
// of 128: 40.3 us, 152 MB, 3.8 TB/s (57 % of a copy's 6.55); pages of 16: 45.3; a ragged batch of
// 33 requests of up to 8321 rows, pages of 16: 48.2; 2129 rows: 10.4; fp32 queries over 131137
// rows, pages of 64: 49.5 (the weights and queries in two parts each: more matrix instructions and
// registers, 8 warps).  From 131072 to 262144 rows 25.3 us are added, 25.1 where the tables
// name 8 pages over and over, which L2 holds: the stream of 25 us is not bound by memory, though it
// runs at 91 % of a copy's rate, but by the instructions.  There are 18.3 M warp instructions,
// over the whole kernel 0.47 a cycle and scheduler, with the logic pipe that takes the codes apart
// 44 % busy.  The other 15 us are latency: the plan, the first page ids and keys, a
// run's whole tiles, the pieces and the second kernel.
// Tried: tiles of 32 keys, 41 .. 52 us; 16-byte copies by every lane in place of the bulk
// copies, 51.5 (pages of 16: 55.7 against 56.5 then), for the scales and biases alone 41.7 (pages
// of 16: 43.6 against 45.2); two or three CTAs per SM, 42 .. 59; merging by a ticket
// in this kernel, 45.2.
#pragma once

#include <cfloat>

#include "attn_tc.cuh"
#include "common.cuh"
#include "kv4.cuh"

namespace tg {

constexpr int kKv4MaxGroup = 8;
constexpr int kKv4Tile = 64;  // keys per unit of work: four matrix blocks whose chains overlap
constexpr float kKv4Slack = 4.0f;   // a weight may exceed 1 by 2^4 before the running maximum follows
constexpr int kKv4WeightExp = 10;   // a weight times a scale that is one unit lands at 2^10: 2^15 at most in fp16
// A unit is set 2^3 above the largest product of a weight and a scale.  More makes moves rarer and
// rounds coarser: 131137 rows (16 + 8 heads), value scales that spread by 2^4 (one standard deviation)
// and biases of 6 between rows, 2^3 43.4 us, 2^6 43.0; ordinary rows 40.3 with both.
constexpr int kKv4Over = 3;
constexpr int kKv4LeastUnit = 14;   // the smallest unit: its factor, 2^123, times a weight, 2^4 at most, is a float

// Warps of one CTA (one CTA per SM): as many as registers hold.  bf16, 12 against 8: the ragged
// batch 48.2 / 52.4 us, 64 requests of 200 rows 13.8 / 16.3, 131137 rows 40.3 / 41.4, 4 requests
// of 32761 rows of 4 + 4 heads 22.3 / 21.4.  With 8 heads
// a B operand, or two parts of queries and weights, a thread needs up to 248 registers.
template <typename T, int HP>
struct Kv4Cfg {
  static constexpr int kWarps = HP == 8 || sizeof(T) == 4 ? 8 : 12;
};

struct Kv4DecodeParams {
  Kv4Cache c;
  const void* q;
  int64_t ldq;
  const int32_t* tables;
  int32_t max_pages;
  const int32_t* lens;
  int32_t nreq, hq, group;
  const float* gain;
  const float* temp;
  const float* ratio;  // [nreq] or null
  float scale_log2;    // sm_scale * log2 e
  void* out;
  int64_t ldo;
  float* lse;          // [nreq][hq] or null
  float* part;         // [CTAs][2] pieces
};

// Cost a CTA takes before another one joins (3 at least: see kv4_tiles_before).  4 against 12:
// 2129 rows 10.4 / 11.0 us, fp32 queries over 5 requests of up to 997 rows 10.0 / 10.5.
constexpr int kKv4MinCost = 4;

// one piece of a (request, head): group rows of D sums, then the maxima, then the weight sums
__host__ __device__ constexpr int kv4_piece_floats(int group, int d) { return (group * (d + 2) + 3) / 4 * 4; }

// a warp's share of shared memory: two tiles of keys (codes, scales, biases), one of values
template <int D>
struct Kv4Ring {
  static constexpr int kCodes = kKv4Tile * D / 2, kScales = kKv4Tile * D / 16;
  static constexpr int kBias = kCodes + kScales, kKeys = kBias + kKv4Tile * 4;  // in a tile of keys
  static constexpr int kValues = 2 * kKeys, kBytes = kValues + kCodes + kScales;
};

__host__ __device__ constexpr size_t kv4_decode_head_smem(int nreq) {  // tile prefix sums
  return static_cast<size_t>(nreq + 1 + 31) / 32 * 128;
}
template <typename T, int D, int HP>
constexpr size_t kv4_decode_smem(int nreq, int group) {
  using Cfg = Kv4Cfg<T, HP>;
  return kv4_decode_head_smem(nreq) + static_cast<size_t>(Cfg::kWarps) * Kv4Ring<D>::kBytes +
         static_cast<size_t>(Cfg::kWarps) * kv4_piece_floats(group, D) * 4;
}

__device__ __forceinline__ float kv4_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float kv4_lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float exp_bits(int field) { return __uint_as_float(static_cast<uint32_t>(field) << 23); }
// A unit (the exponent field of a float, kKv4LeastUnit .. 254), the factor that brings it to
// 2^kKv4WeightExp, and that factor's inverse.  Both are normal floats.
__device__ __forceinline__ float factor_of(int unit) { return exp_bits(254 + kKv4WeightExp - unit); }
__device__ __forceinline__ int unit_of(float factor) { return 254 + kKv4WeightExp - static_cast<int>(__float_as_uint(factor) >> 23); }
__device__ __forceinline__ float inverse_of(float factor) { return exp_bits(unit_of(factor) - kKv4WeightExp); }

// N neighbouring words of shared memory.  Plain loads, like the matrix instructions below
// without `volatile`: the compiler may move them past one another, which is what
// hides their latencies.
template <int N>
__device__ __forceinline__ void words(const uint8_t* at, uint32_t (&v)[N]) {
  if constexpr (N == 4) {
    const uint4 w = *reinterpret_cast<const uint4*>(at);
    v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
  } else if constexpr (N == 2) {
    const uint2 w = *reinterpret_cast<const uint2*>(at);
    v[0] = w.x, v[1] = w.y;
  } else {
    v[0] = *reinterpret_cast<const uint32_t*>(at);
  }
}

// the four bytes of w (two E2M1 codes each) as fp16 pairs
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same from a zero accumulator
__device__ __forceinline__ void mma_f16_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float f16_lo(uint32_t h) {
  float f;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(f) : "r"(h));
  return f;
}
__device__ __forceinline__ float f16_hi(uint32_t h) {
  float f;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.f32.f16 %0, u;\n\t}" : "=f"(f) : "r"(h));
  return f;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float rows_max(float v) {  // over the 8 lanes of a column pair
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
}
__device__ __forceinline__ float rows_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  v += __shfl_xor_sync(0xffffffffu, v, 8);
  return v + __shfl_xor_sync(0xffffffffu, v, 16);
}

// four consecutive output values
__device__ __forceinline__ void store4(__nv_bfloat16* p, float a, float b, float c, float d) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d));
}
__device__ __forceinline__ void store4(float* p, float a, float b, float c, float d) {
  *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}

// rows a request attends to: a length outside its table counts as none
__device__ __forceinline__ int kv4_length(const Kv4DecodeParams& p, int r) {
  const int n = p.lens[r];
  return n < 0 || n > static_cast<int64_t>(p.max_pages) * p.c.page_rows ? 0 : n;
}

// The work is cut by cost: 2 for a tile and 1 more for starting on a (request, head) (its
// query, an empty state, a result to hand over: about half a tile's time).  A run has
// the tiles whose cost begins in it; a run of 3 inside a (request, head) has at least
// one.  Tiles of one (request, head) of nt tiles before position z of its 2 nt + 1:
__device__ __forceinline__ int kv4_tiles_before(int z, int nt) { return min(z == 0 ? 0 : max(1, z >> 1), nt); }

template <typename T, int D, int HP>
__global__ void __launch_bounds__(32 * Kv4Cfg<T, HP>::kWarps, 1) k_kv4_decode(const Kv4DecodeParams p) {
  using Ring = Kv4Ring<D>;
  constexpr int W = Kv4Cfg<T, HP>::kWarps, TP = 32 * W, MT = kKv4Tile / 16;
  constexpr bool kSplit = sizeof(T) == 4;      // fp32: query and weights in two fp16 parts
  constexpr int NG = D / 32, SL = 8 / HP, NB = NG > SL ? NG / SL : 1;
  constexpr int kSwap = D == 128 ? 1 : 2;      // key order inside 16 rows, see below
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_warp[W];
  __shared__ int s_seg[W][2];          // (request, head) of the warp's unfinished pieces, -1: none
  __shared__ int s_edge[W][2];         // bit 0: the piece begins the (request, head), bit 1: it ends it
  __shared__ uint64_t s_full[W][3];     // keys (two tiles), values
  __shared__ int s_stop;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, t = lane & 3, n8 = lane >> 2;
  int* s_cum = reinterpret_cast<int*>(smem);   // [nreq + 1] tiles of the requests before
  uint8_t* ring = smem + kv4_decode_head_smem(p.nreq) + static_cast<size_t>(warp) * Ring::kBytes;
  float* piece0 = reinterpret_cast<float*>(smem + kv4_decode_head_smem(p.nreq) +
                                           static_cast<size_t>(W) * Ring::kBytes) +
                  warp * kv4_piece_floats(p.group, D);
  const int hkv = p.c.hkv, P = p.c.page_rows, group = p.group;

  if (lane < 3) mbar_init(&s_full[warp][lane], 1);
  if (lane < 2) s_seg[warp][lane] = -1;
  if (tid == 0) s_stop = 0;
  fence_mbar_init();
  pdl_wait();
  pdl_launch_dependents();

  // ---- tiles of every request
  const int per = (p.nreq + TP - 1) / TP, rq0 = min(tid * per, p.nreq), rq1 = min(rq0 + per, p.nreq);
  int mine = 0;
  for (int r = rq0; r < rq1; ++r) {
    const int n = kv4_length(p, r);
    if (n != p.lens[r] && blockIdx.x == 0) raise_error(kErrKvPage, 1);
    mine += (n + kKv4Tile - 1) / kKv4Tile;
  }
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  int base = inc - mine, total = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < warp) base += s_warp[w];
    total += s_warp[w];
  }
  for (int r = rq0; r < rq1; ++r) {
    s_cum[r] = base;
    base += (kv4_length(p, r) + kKv4Tile - 1) / kKv4Tile;
  }
  if (tid == 0) s_cum[p.nreq] = total;
  __syncthreads();

  // ---- requests without rows
  for (int r = blockIdx.x; r < p.nreq; r += gridDim.x) {
    if (s_cum[r + 1] != s_cum[r]) continue;
    for (int i = tid; i < p.hq * D; i += TP) static_cast<T*>(p.out)[r * p.ldo + i] = from_f32<T>(0.0f);
    for (int i = tid; i < p.hq && p.lse; i += TP) p.lse[static_cast<int64_t>(r) * p.hq + i] = -INFINITY;
  }

  // ---- this warp's run: CTA c takes `each` of the cost, the first `more` CTAs one extra
  const int cost = (2 * total + p.nreq) * hkv;  // < 2^31, checked by the caller
  const int ctas = min(static_cast<int>(gridDim.x), max(1, cost / kKv4MinCost)), cta = blockIdx.x;
  if (cta >= ctas || total == 0) return;
  const int each = cost / ctas, more = cost - each * ctas;
  const int mine_n = each + (cta < more ? 1 : 0), x0 = each * cta + min(cta, more);
  int tiles = 0;  // even lanes: tiles before this warp's run, odd lanes: before the next one's
  {
    const int x = x0 + mine_n * (warp + (lane & 1)) / W;
    int lo = 0, hi = p.nreq - 1;  // largest request that starts at or before x
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((2 * s_cum[mid] + mid) * hkv <= x) lo = mid;
      else hi = mid - 1;
    }
    const int nt = s_cum[lo + 1] - s_cum[lo], y = x - (2 * s_cum[lo] + lo) * hkv, g = y / (2 * nt + 1);
    tiles = s_cum[lo] * hkv + g * nt + kv4_tiles_before(y - g * (2 * nt + 1), nt);
  }
  const int ua = __shfl_sync(0xffffffffu, tiles, 0), left = __shfl_sync(0xffffffffu, tiles, 1) - ua;

  // position of the next unit to load: request, head, tile of the request's lnt, its rows
  int lr = 0, lg = 0, lt = 0, lnt = 1, llen = 0;
  if (left > 0) {
    int lo = 0, hi = p.nreq - 1;  // largest request whose tiles start at or before ua: it has some
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_cum[mid] * hkv <= ua) lo = mid;
      else hi = mid - 1;
    }
    lr = lo;
    lnt = s_cum[lr + 1] - s_cum[lr];
    const int x = ua - s_cum[lr] * hkv;
    lg = x / lnt;
    lt = x - lg * lnt;
    llen = kv4_length(p, lr);
  }
  int cr = lr, cg = lg, ct = lt, cnt = lnt, clen = llen;  // position of the unit being computed
  auto next_head = [&](int& r, int& g, int& tt, int& nt, int& len) {
    tt = 0;
    if (++g < hkv) return;
    g = 0;
    do ++r; while (r < p.nreq && s_cum[r + 1] == s_cum[r]);
    if (r < p.nreq) {
      nt = s_cum[r + 1] - s_cum[r];
      len = kv4_length(p, r);
    }
  };
  // Lane i moves array i / MT, from 16-row block i % MT on, up to the end of the page or of
  // the tile: K codes, K scales, biases, V codes, V scales
  const int what = lane / MT, blk = lane % MT;
  const bool keys = what < (p.c.bias ? 3 : 2), values = what == 3 || what == 4;
  const uint32_t row_bytes = what == 0 || what == 3 ? D / 2 : what == 2 ? 4 : D / 16;
  const uint8_t* src0 = what == 0   ? p.c.k_codes
                        : what == 1 ? reinterpret_cast<const uint8_t*>(p.c.k_scales)
                        : what == 2 ? reinterpret_cast<const uint8_t*>(p.c.bias)
                        : what == 3 ? p.c.v_codes
                                    : reinterpret_cast<const uint8_t*>(p.c.v_scales);
  uint8_t* dst0 = ring + blk * 16 * row_bytes +
                  (what == 0 ? 0 : what == 1 ? Ring::kCodes : what == 2 ? Ring::kBias : what == 3 ? Ring::kValues : Ring::kValues + Ring::kCodes);
  const int64_t page_bytes = static_cast<int64_t>(what == 2 ? 1 : hkv) * P * row_bytes;
  const uint32_t head_bytes = what == 2 ? 0 : P * row_bytes;  // biases are shared by the heads
  const uint32_t key_tx = 16 * (D / 2 + D / 16 + (p.c.bias ? 4 : 0)), value_tx = 16 * (D / 2 + D / 16);
  const uint32_t full0 = smem_u32(&s_full[warp][0]);
  // The request's next 32 page ids, one per lane: fetched when the position moves past
  // them or to another request, used by a later load.
  int32_t pages = 0;
  int page0 = 0;
  auto fetch_pages = [&]() {
    page0 = (lt * kKv4Tile) >> p.c.page_shift;
    pages = 0;
    if (lr < p.nreq && (page0 + lane) << p.c.page_shift < llen)
      pages = p.tables[static_cast<int64_t>(lr) * p.max_pages + page0 + lane];
  };
  // The keys of the next tile into key tile `st`; where its values are is kept for load_values,
  // one tile behind (blocks of both, this lane's source and size)
  const uint8_t* vsrc0 = nullptr;
  const uint8_t* vsrc1 = nullptr;
  uint32_t vbytes0 = 0, vbytes1 = 0;
  int vblocks0 = 0, vblocks1 = 0;
  auto load_values = [&]() {
    if (lane == 0) mbar_arrive_expect_tx(&s_full[warp][2], vblocks0 * value_tx);
    __syncwarp();
    if (values && vbytes0) bulk_load(dst0, vsrc0, vbytes0, &s_full[warp][2]);
    vsrc0 = vsrc1;
    vbytes0 = vbytes1;
    vblocks0 = vblocks1;
  };
  auto load_keys = [&](int st) {
    const int row0 = lt * kKv4Tile, blocks = min(MT, (llen - row0 + 15) >> 4);
    const int row = row0 + 16 * blk, in_page = row & (P - 1);
    int32_t page = __shfl_sync(0xffffffffu, pages, (row >> p.c.page_shift) - page0);
    if (lane == 0) mbar_arrive_expect_tx(&s_full[warp][st], blocks * key_tx);
    __syncwarp();
    uint32_t bytes = 0;
    if (blk < blocks && (blk == 0 || in_page == 0)) {
      if (page < 0 || page >= p.c.num_pages) {
        raise_error(kErrKvPage, 2);
        page = 0;
      }
      bytes = min(blocks - blk, (P - in_page) >> 4) * 16 * row_bytes;
    }
    const uint8_t* src = src0 + page * page_bytes + lg * static_cast<uint64_t>(head_bytes) + in_page * row_bytes;
    if (keys && bytes) bulk_load(dst0 + st * Ring::kKeys, src, bytes, &s_full[warp][st]);
    vsrc1 = src;
    vbytes1 = bytes;
    vblocks1 = blocks;
    if (++lt == lnt) {
      const int r = lr;
      next_head(lr, lg, lt, lnt, llen);
      if (lr != r || page0 != 0) fetch_pages();
    } else if (((lt * kKv4Tile + kKv4Tile - 1) >> p.c.page_shift) - page0 >= 32) {
      fetch_pages();
    }
  };

  // ---- per-lane state.  Accumulator columns 2t, 2t + 1 are heads hd, hd + 1 of scale
  // group slot `slot`; accumulator rows n8 and n8 + 8 are keys (scores) or dimensions.
  const int hd = (2 * t) % HP, slot = 2 * t / HP;
  // Shifts left as products with factors the compiler does not see: they go to the multiply-add
  // pipe, and the integer pipe that the conversions share is what bounds the loop.
  uint32_t shl4, shl16;
  asm volatile("mov.u32 %0, 16;\n\tmov.u32 %1, 65536;" : "=r"(shl4), "=r"(shl16));
  // Row i of a score tile is key key_of(i): even rows keys i / 2, odd rows the other
  // four, ordered so that the 16-byte key loads of 8 lanes and the value loads of
  // 4 keys x 4 lanes both spread over all banks (values: lane t takes the keys of
  // rows 2t, 2t + 1, 2t + 8, 2t + 9).
  const int key0 = n8 & 1 ? 4 + ((n8 >> 1) ^ kSwap) : n8 >> 1;
  const int kswz = D == 128 ? (key0 & 2) << 4 : 0, vswz = D == 128 ? (t & 2) << 4 : 0;
  const uint32_t at0 = static_cast<uint32_t>(ring - smem);
  const uint32_t kbase = at0 + key0 * (D / 2) + ((t * (D / 8)) ^ kswz);
  const uint32_t vbase = at0 + Ring::kValues + ((n8 * (D / 16)) ^ vswz) + t * (D / 2);  // key t of 16
  const uint32_t vother = (4 + (t ^ kSwap) - t) * (D / 2);                              // to its odd row's key
  const uint32_t sbase = at0 + Ring::kCodes + key0 * (D / 16);
  const uint32_t wbase = at0 + Ring::kValues + Ring::kCodes + key0 * (D / 16) + 2 * slot;
  const uint32_t bbase = at0 + Ring::kBias + 4 * key0;
  if (!p.c.bias)  // no copy writes the biases then
    for (int i = lane; i < 2 * kKv4Tile; i += 32)
      *reinterpret_cast<float*>(smem + at0 + i / kKv4Tile * Ring::kKeys + Ring::kBias + i % kKv4Tile * 4) = 0.0f;

  uint32_t qf[kSplit ? 2 : 1][NG][2][2];
  float o[NG][2][4];
  float bias_most = 0.0f;  // gain times a bias up to this is finite in base 2
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f, a0 = 0.0f, a1 = 0.0f, g0 = 0.0f, g1 = 0.0f;
  float fac0[NB], fac1[NB];  // the weights' factors

  auto begin = [&]() {  // a new (request, head): its query, factors, and empty sums
    const int h0 = cg * group;
    const int u = n8 % HP;
    float x[NG][8];
    float top = 0.0f;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      if (u < group)
        load8(static_cast<const T*>(p.q) + cr * p.ldq + static_cast<int64_t>(h0 + u) * D + 32 * g + 8 * t, x[g]);
      else
#pragma unroll
        for (int e = 0; e < 8; ++e) x[g][e] = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[g][e]));
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // 2^(8 - exponent of the largest): exact, and so is its inverse
    const int field = min(262 - static_cast<int>(__float_as_uint(top) >> 23), 253);
    const float f = exp_bits(field), back = exp_bits(254 - field);
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float lo = x[g][4 * s + 2 * e] * f, hi = x[g][4 * s + 2 * e + 1] * f;
          qf[0][g][s][e] = f16x2(lo, hi);
          if constexpr (kSplit) qf[1][g][s][e] = f16x2(lo - f16_lo(qf[0][g][s][e]), hi - f16_hi(qf[0][g][s][e]));
        }
    const float b0 = __shfl_sync(0xffffffffu, back, 4 * hd), b1 = __shfl_sync(0xffffffffu, back, 4 * hd + 4);
    const float rs = (p.ratio ? p.ratio[cr] : 1.0f) * p.scale_log2;
    a0 = hd < group ? p.temp[h0 + hd] * rs * b0 : 0.0f;
    a1 = hd + 1 < group ? p.temp[h0 + hd + 1] * rs * b1 : 0.0f;
    g0 = hd < group ? p.gain[h0 + hd] * 1.4426950408889634f : 0.0f;
    g1 = hd + 1 < group ? p.gain[h0 + hd + 1] * 1.4426950408889634f : 0.0f;
    float gmax = fmaxf(fabsf(g0), fabsf(g1));
    gmax = fmaxf(gmax, __shfl_xor_sync(0xffffffffu, gmax, 1));
    gmax = fmaxf(gmax, __shfl_xor_sync(0xffffffffu, gmax, 2));
    bias_most = FLT_MAX / fmaxf(gmax, 1.0f) * 0.999f;
    m0 = m1 = -INFINITY;
    l0 = l1 = 0.0f;
#pragma unroll
    for (int b = 0; b < NB; ++b) fac0[b] = factor_of(hd < group ? kKv4LeastUnit : 254), fac1[b] = factor_of(hd + 1 < group ? kKv4LeastUnit : 254);
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[g][j][c] = 0.0f;
  };

  // the finished run of tiles: to the output (whole) or to a piece in shared memory
  auto finish = [&](bool whole, float* dst) {
    const float s0 = rows_sum(l0), s1 = rows_sum(l1);
    const int h0 = cg * group;
    float f0 = 1.0f, f1 = 1.0f;
    if (whole) {
      f0 = s0 == 0.0f ? 0.0f : 1.0f / s0;
      f1 = s1 == 0.0f ? 0.0f : 1.0f / s1;
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      if (g % SL != slot) continue;
      const float back0 = inverse_of(fac0[g / SL]), back1 = inverse_of(fac1[g / SL]);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (hd + c >= group) continue;
        const float f = c ? f1 : f0;
        const float unit = c ? back1 : back0;
        const float y0 = o[g][0][c] * f * unit, y1 = o[g][0][c + 2] * f * unit;
        const float y2 = o[g][1][c] * f * unit, y3 = o[g][1][c + 2] * f * unit;
        const int at = 32 * g + 4 * n8;
        if (whole) store4(static_cast<T*>(p.out) + cr * p.ldo + static_cast<int64_t>(h0 + hd + c) * D + at, y0, y1, y2, y3);
        else store4(dst + (hd + c) * D + at, y0, y1, y2, y3);
      }
    }
    if (n8 == 0 && slot == 0) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (hd + c >= group) continue;
        const float mm = c ? m1 : m0, ss = c ? s1 : s0;
        if (!whole) {
          dst[group * D + hd + c] = mm;
          dst[group * (D + 1) + hd + c] = ss;
        } else if (p.lse) {
          p.lse[static_cast<int64_t>(cr) * p.hq + h0 + hd + c] = ss == 0.0f ? -INFINITY : (mm + log2f(ss)) * 0.6931471805599453f;
        }
      }
    }
  };

  bool ok = true;
  if (left > 0) {
    fetch_pages();
    load_keys(0);
    vsrc0 = vsrc1, vbytes0 = vbytes1, vblocks0 = vblocks1;
    if (left > 1) load_keys(1);
    load_values();
    bool begun = ct == 0;  // the current (request, head) begins in this run
    bool fresh = true;     // its state is not set up yet
#pragma unroll 1
    for (int i = 0; i < left; ++i) {
      if (fresh) begin();
      fresh = false;
      const uint32_t st = i & 1;
      if (!__all_sync(0xffffffffu, mbar_try_wait(full0 + 8 * st, i >> 1 & 1))) {
        ok = warp_wait(&s_full[warp][st], i >> 1 & 1, kErrWaitAttention);
        if (!ok) break;
      }
      const uint32_t stage = st * Ring::kKeys;
      const int rows = min(kKv4Tile, clen - ct * kKv4Tile);
      // Keys past the request's rows and keys with bias -infinity: their scales and biases
      // are zeroed (whatever they hold must not meet the sums) and their logits set to -infinity.
      uint32_t dead[(MT + 1) / 2];
      bool any_dead = false, huge = false;
#pragma unroll
      for (int h = 0; h < (MT + 1) / 2; ++h) {
        const int key = 32 * h + lane;
        bool d = false;
        if (key < kKv4Tile && key < rows) {
          const float bias = *reinterpret_cast<const float*>(smem + at0 + stage + Ring::kBias + 4 * key);
          d = bias == -INFINITY;
          huge |= fabsf(bias) > bias_most;  // infinities too
        } else {
          d = true;
        }
        dead[h] = __ballot_sync(0xffffffffu, d);
        any_dead |= dead[h] != 0;
      }
      huge = __any_sync(0xffffffffu, huge);
      if (any_dead) {
#pragma unroll
        for (int h = 0; h < (MT + 1) / 2; ++h)
          if (dead[h] >> lane & 1u) {
            const uint32_t key = 32 * h + lane;
#pragma unroll
            for (int g = 0; g < NG / 2; ++g)
              *reinterpret_cast<uint32_t*>(smem + at0 + stage + Ring::kCodes + key * (D / 16) + 4 * g) = 0;
            *reinterpret_cast<float*>(smem + at0 + stage + Ring::kBias + 4 * key) = 0.0f;
          }
        fence_proxy_async_smem();  // before the next copy into this tile
        __syncwarp();
      }

      // ---- scores of the tile's keys
      float x[MT][4];
      float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        uint32_t w0[NG], w1[NG];  // halves (unit 2t: groups 0..), (unit 2t + 1: groups 0..)
        const uint8_t* ka = smem + kbase + stage + mt * 8 * D;
        words(ka, w0);
        words(ka + 4 * D, w1);
        uint32_t h0[NG][4], h1[NG][4];  // [word][byte]: word s * NG / 2 + g / 2, bytes 2 (g & 1), + 1
#pragma unroll
        for (int w = 0; w < NG; ++w) {
          e2m1x8(w0[w], h0[w]);
          e2m1x8(w1[w], h1[w]);
        }
        uint32_t sc0[NG / 2], sc1[NG / 2];  // bf16 scale pairs of both keys
        words(smem + sbase + stage + mt * D, sc0);
        words(smem + sbase + stage + mt * D + D / 2, sc1);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          float acc[4];
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const int w = s * (NG / 2) + g / 2, b = 2 * (g & 1);
            if (s == 0) mma_f16_zero(acc, h0[w][b], h1[w][b], h0[w][b + 1], h1[w][b + 1], qf[0][g][0][0], qf[0][g][0][1]);
            else mma_f16(acc, h0[w][b], h1[w][b], h0[w][b + 1], h1[w][b + 1], qf[0][g][1][0], qf[0][g][1][1]);
            if constexpr (kSplit) mma_f16(acc, h0[w][b], h1[w][b], h0[w][b + 1], h1[w][b + 1], qf[1][g][s][0], qf[1][g][s][1]);
          }
          const float k0 = g & 1 ? bf16_hi(sc0[g / 2]) : __uint_as_float(sc0[g / 2] * shl16);
          const float k1 = g & 1 ? bf16_hi(sc1[g / 2]) : __uint_as_float(sc1[g / 2] * shl16);
          x[mt][0] = g ? fmaf(k0, acc[0], x[mt][0]) : k0 * acc[0];
          x[mt][1] = g ? fmaf(k0, acc[1], x[mt][1]) : k0 * acc[1];
          x[mt][2] = g ? fmaf(k1, acc[2], x[mt][2]) : k1 * acc[2];
          x[mt][3] = g ? fmaf(k1, acc[3], x[mt][3]) : k1 * acc[3];
        }
        const float bias0 = *reinterpret_cast<const float*>(smem + bbase + stage + 64 * mt);
        const float bias1 = *reinterpret_cast<const float*>(smem + bbase + stage + 64 * mt + 32);
        x[mt][0] = fmaf(a0, x[mt][0], g0 * bias0);
        x[mt][1] = fmaf(a1, x[mt][1], g1 * bias0);
        x[mt][2] = fmaf(a0, x[mt][2], g0 * bias1);
        x[mt][3] = fmaf(a1, x[mt][3], g1 * bias1);
      }
      if (huge) {  // a finite bias makes a finite logit
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (fabsf(x[mt][c]) == INFINITY && fabsf(*reinterpret_cast<const float*>(smem + bbase + stage + 64 * mt + 32 * (c >> 1))) < INFINITY)
              x[mt][c] = copysignf(FLT_MAX, x[mt][c]);
      }
      if (any_dead) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const uint32_t m = dead[mt / 2] >> (16 * (mt & 1) + key0);
          if (m & 1u) x[mt][0] = x[mt][1] = -INFINITY;
          if (m >> 8 & 1u) x[mt][2] = x[mt][3] = -INFINITY;
        }
      }
      __syncwarp();  // every lane has read the keys
      if (i + 2 < left) load_keys(st);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        t0 = fmax3(t0, x[mt][0], x[mt][2]);
        t1 = fmax3(t1, x[mt][1], x[mt][3]);
      }

      // ---- running maxima of the logits and of the value scales' exponents
      if (!__all_sync(0xffffffffu, mbar_try_wait(full0 + 16, i & 1))) {
        ok = warp_wait(&s_full[warp][2], i & 1, kErrWaitAttention);
        if (!ok) break;
      }
      if (any_dead) {
#pragma unroll
        for (int h = 0; h < (MT + 1) / 2; ++h)
          if (dead[h] >> lane & 1u)
#pragma unroll
            for (int g = 0; g < NG / 2; ++g)
              *reinterpret_cast<uint32_t*>(smem + at0 + Ring::kValues + Ring::kCodes + (32 * h + lane) * (D / 16) + 4 * g) = 0;
        fence_proxy_async_smem();
        __syncwarp();
      }
      uint32_t vs0[MT][NB], vs1[MT][NB];  // bf16 value scales of this lane's groups, as fp32 bits
      float vtop[NB];  // largest magnitude; NaN is passed over
#pragma unroll
      for (int b = 0; b < NB; ++b) vtop[b] = 0.0f;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          vs0[mt][b] = static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(smem + wbase + mt * D + 2 * SL * b)) * shl16;
          vs1[mt][b] = static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(smem + wbase + mt * D + D / 2 + 2 * SL * b)) * shl16;
          vtop[b] = fmax3(vtop[b], fabsf(__uint_as_float(vs0[mt][b])), fabsf(__uint_as_float(vs1[mt][b])));
        }
      // The reference m and the units of the weights move only when a weight would pass
      // 2^kKv4Slack or a value scale is twice a unit (a warp vote; the first tile always does).
      bool moved = t0 > m0 + kKv4Slack || t1 > m1 + kKv4Slack;
#pragma unroll
      for (int b = 0; b < NB; ++b) moved |= vtop[b] * fmaxf(fac0[b], fac1[b]) >= exp_bits(128 + kKv4WeightExp);
      bool far = false;  // a scale so far above its unit that a weight below the normal floats counts
      if (__any_sync(0xffffffffu, moved)) {
        const float tile0 = rows_max(t0), tile1 = rows_max(t1), n0 = fmaxf(m0, tile0), n1 = fmaxf(m1, tile1);
        const float d0 = n0 == m0 ? 0.0f : m0 - n0, d1 = n1 == m1 ? 0.0f : m1 - n1;
        l0 *= kv4_ex2(d0);
        l1 *= kv4_ex2(d1);
        // A unit falls with its head's sums as the reference rises, and rises to 2^kKv4Over times
        // the tile's largest product of a weight and a scale: so it is never further than that (and
        // a rounding up) above the largest product so far, whatever came before, and scales
        // have to grow that much before the next tile moves it.
        const bool real0 = hd < group, real1 = hd + 1 < group;
        const int fall0 = static_cast<int>(floorf(fmaxf(d0, -300.0f))), fall1 = static_cast<int>(floorf(fmaxf(d1, -300.0f)));
        const float r0 = fmaxf(n0, -FLT_MAX), r1 = fmaxf(n1, -FLT_MAX);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          float u0 = -300.0f, u1 = -300.0f;  // base 2
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const float e0 = kv4_lg2(fabsf(__uint_as_float(vs0[mt][b]))), e1 = kv4_lg2(fabsf(__uint_as_float(vs1[mt][b])));
            u0 = fmax3(u0, x[mt][0] - r0 + e0, x[mt][2] - r0 + e1);
            u1 = fmax3(u1, x[mt][1] - r1 + e0, x[mt][3] - r1 + e1);
          }
          u0 = rows_max(u0), u1 = rows_max(u1);
          const int old0 = unit_of(fac0[b]), old1 = unit_of(fac1[b]);
          const int new0 = real0 ? max(max(old0 + fall0, kKv4LeastUnit), 127 + min(kKv4Over + static_cast<int>(ceilf(fminf(u0, 128.0f))), 127)) : 254;
          const int new1 = real1 ? max(max(old1 + fall1, kKv4LeastUnit), 127 + min(kKv4Over + static_cast<int>(ceilf(fminf(u1, 128.0f))), 127)) : 254;
          far |= static_cast<int>(__float_as_uint(vtop[b]) >> 23) - min(new0, new1) > 90;
          const float c0 = kv4_ex2(d0 + static_cast<float>(old0 - new0)), c1 = kv4_ex2(d1 + static_cast<float>(old1 - new1));
          fac0[b] = factor_of(new0);
          fac1[b] = factor_of(new1);
#pragma unroll
          for (int g = b * SL; g < (b + 1) * SL && g < NG; ++g)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              o[g][j][0] *= c0;
              o[g][j][1] *= c1;
              o[g][j][2] *= c0;
              o[g][j][3] *= c1;
            }
        }
        far = __any_sync(0xffffffffu, far);
        m0 = n0;
        m1 = n1;
      }
      const float use0 = m0 == -INFINITY ? 0.0f : m0, use1 = m1 == -INFINITY ? 0.0f : m1;

      // ---- weights, and their products with the values.  The matrix unit cuts its fp32 sums where an
      // addition rounds them, and the cuts of a long run add up: with fp32 queries a tile is summed
      // on its own and added to the run's.  Relative error of 131137 rows 4.8e-7, without it 1.8e-6
      // (and growing with the rows: 76 million rows of one KV head 3.6e-4); 49.5 us, without it 48.2.
      // With bf16 queries the cuts stay below 2^-12 up to some 150 million rows.
      float tile_o[kSplit ? NG : 1][2][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float p00 = kv4_ex2(x[mt][0] - use0), p01 = kv4_ex2(x[mt][1] - use1);
        float p10 = kv4_ex2(x[mt][2] - use0), p11 = kv4_ex2(x[mt][3] - use1);
        if (far) {
          p00 = exp2f(x[mt][0] - use0), p01 = exp2f(x[mt][1] - use1);
          p10 = exp2f(x[mt][2] - use0), p11 = exp2f(x[mt][3] - use1);
        }
        l0 += p00 + p10;
        l1 += p01 + p11;
        uint32_t pf[kSplit ? 2 : 1][NB][2];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          // the factor goes to the weight: a scale far above the unit (its weight far below 1) times
          // the factor may pass the largest float, weight times factor cannot
          const float s0 = __uint_as_float(vs0[mt][b]), s1 = __uint_as_float(vs1[mt][b]);
          const uint64_t fac = f2_pack(fac0[b], fac1[b]);
          float w00, w01, w10, w11;
          f2_unpack(f2_mul(f2_mul(f2_pack(p00, p01), fac), f2_pack(s0, s0)), w00, w01);
          f2_unpack(f2_mul(f2_mul(f2_pack(p10, p11), fac), f2_pack(s1, s1)), w10, w11);
          const uint32_t r0 = f16x2(w00, w01), r1 = f16x2(w10, w11);
          pf[0][b][0] = transpose8x8(r0);
          pf[0][b][1] = transpose8x8(r1);
          if constexpr (kSplit) {
            pf[1][b][0] = transpose8x8(f16x2(w00 - f16_lo(r0), w01 - f16_hi(r0)));
            pf[1][b][1] = transpose8x8(f16x2(w10 - f16_lo(r1), w11 - f16_hi(r1)));
          }
        }
        const uint8_t* va = smem + vbase + mt * 8 * D;
        uint32_t wa[NG / 2], wb[NG / 2], wc[NG / 2], wd[NG / 2];
        words(va, wa);
        words(va + vother, wb);
        words(va + 4 * D, wc);
        words(va + vother + 4 * D, wd);
#pragma unroll
        for (int w = 0; w < NG / 2; ++w) {
          // low nibbles of two keys side by side, then the high ones: byte 2i + j holds
          // dimensions 2j (lo) or 2j + 1 (hi) of group 2w + i for both keys
          constexpr uint32_t M = 0x0f0f0f0fu;
          uint32_t loab[4], hiab[4], locd[4], hicd[4];
          e2m1x8((wa[w] & M) | (wb[w] * shl4 & ~M), loab);
          e2m1x8((wa[w] >> 4 & M) | (wb[w] & ~M), hiab);
          e2m1x8((wc[w] & M) | (wd[w] * shl4 & ~M), locd);
          e2m1x8((wc[w] >> 4 & M) | (wd[w] & ~M), hicd);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int v = 0; v < (kSplit ? 2 : 1); ++v) {
                const int g = 2 * w + i, b = g / SL;
                const uint32_t a0 = loab[2 * i + j], a1 = hiab[2 * i + j], a2 = locd[2 * i + j], a3 = hicd[2 * i + j];
                if constexpr (!kSplit) mma_f16(o[g][j], a0, a1, a2, a3, pf[v][b][0], pf[v][b][1]);
                else if (mt + v == 0) mma_f16_zero(tile_o[g][j], a0, a1, a2, a3, pf[v][b][0], pf[v][b][1]);
                else mma_f16(tile_o[g][j], a0, a1, a2, a3, pf[v][b][0], pf[v][b][1]);
              }
        }
      }
      if constexpr (kSplit) {
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[g][j][c] += tile_o[g][j][c];
      }
      __syncwarp();  // every lane has read the values
      if (i + 1 < left) load_values();
      const bool ends = ct + 1 == cnt;
      if (ends || i + 1 == left) {
        if (begun && ends) {
          finish(true, nullptr);
        } else {
          // a piece: one that begins here ends the run, so the ring is free for it
          finish(false, begun ? reinterpret_cast<float*>(ring) : piece0);
          if (lane == 0) {
            s_seg[warp][begun] = cr * hkv + cg;
            s_edge[warp][begun] = begun | (ends ? 2 : 0);
          }
        }
        begun = fresh = true;
      }
      if (ends) next_head(cr, cg, ct, cnt, clen);
      else ++ct;
    }
  }
  if (!ok && lane == 0) s_stop = 1;
  __syncthreads();
  if (s_stop) return;  // a wait ran out (recorded in the error word)

  // ---- pieces of this CTA, in order of position, to the output or to the workspace.
  // Every warp walks the list (piece 2w is what warp w continued, 2w + 1 what it began);
  // a thread takes four neighbouring values.
  const int pf = kv4_piece_floats(group, D), vals = group * D;
  const int my_seg = lane < 2 * W ? s_seg[lane >> 1][lane & 1] : -1;
  const int my_edge = lane < 2 * W ? s_edge[lane >> 1][lane & 1] : 0;
  const uint8_t* rings = smem + kv4_decode_head_smem(p.nreq);
  const float* kept = reinterpret_cast<const float*>(rings + static_cast<size_t>(W) * Ring::kBytes);
  auto piece_at = [&](int i) -> const float* {
    return i & 1 ? reinterpret_cast<const float*>(rings + static_cast<size_t>(i >> 1) * Ring::kBytes) : kept + (i >> 1) * pf;
  };
  // four values, the reference and the weight sum of head u: to the output, or kept as a piece
  auto emit = [&](int seg, bool whole, float* dst, int e, int u, float4 y, float top, float sum) {
    if (!whole) {
      *reinterpret_cast<float4*>(dst + e) = y;
      if (e % D == 0) {
        dst[vals + u] = top;
        dst[vals + group + u] = sum;
      }
      return;
    }
    const int r = seg / hkv, h0 = seg % hkv * group;
    const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
    store4(static_cast<T*>(p.out) + r * p.ldo + static_cast<int64_t>(h0) * D + e, y.x * f, y.y * f, y.z * f, y.w * f);
    if (e % D == 0 && p.lse)
      p.lse[static_cast<int64_t>(r) * p.hq + h0 + u] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
  };
  for (uint32_t todo = __ballot_sync(0xffffffffu, my_seg >= 0); todo;) {
    const int i = __ffs(todo) - 1, seg = __shfl_sync(0xffffffffu, my_seg, i);
    const uint32_t members = __ballot_sync(0xffffffffu, my_seg == seg);
    todo &= ~members;
    const bool begins = __shfl_sync(0xffffffffu, my_edge, i) & 1;
    const bool whole = begins && (__shfl_sync(0xffffffffu, my_edge, 31 - __clz(members)) & 2);
    for (int e = 4 * tid; e < vals; e += 4 * TP) {
      const int u = e / D;
      float top = -INFINITY;
      for (uint32_t m = members; m; m &= m - 1) top = fmaxf(top, piece_at(__ffs(m) - 1)[vals + u]);
      const float use = top == -INFINITY ? 0.0f : top;
      float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float sum = 0.0f;
      for (uint32_t m = members; m; m &= m - 1) {
        const float* pc = piece_at(__ffs(m) - 1);
        const float f = kv4_ex2(pc[vals + u] - use);
        const float4 v = *reinterpret_cast<const float4*>(pc + e);
        y.x = fmaf(f, v.x, y.x);
        y.y = fmaf(f, v.y, y.y);
        y.z = fmaf(f, v.z, y.z);
        y.w = fmaf(f, v.w, y.w);
        sum = fmaf(f, pc[vals + group + u], sum);
      }
      emit(seg, whole, p.part + (static_cast<int64_t>(cta) * 2 + begins) * pf, e, u, y, top, sum);
    }
  }

}

// The (request, head)s that cross CTAs of k_kv4_decode: block c adds the parts of the one
// that begins in CTA c and goes on after it, in CTA order (blocks without one return).  Block
// row y takes 256 of the group * D values: 4 slices of the parts side by side, 64 threads each.
// Launched right behind the main kernel: the plan is formed while that one still runs.  Bound by
// latency, about 3 us; as the last CTA's work in the main kernel, behind a counter to be
// zeroed before the call, 131137 rows took 45.2 us against 40.3.
template <typename T, int D>
__global__ void __launch_bounds__(256) k_kv4_merge(const Kv4DecodeParams p, int ctas_max) {
  constexpr int kVals = 256, kHeads = kVals / D, kAhead = 6;
  extern __shared__ float s_w[];  // [CTAs][kHeads] weights
  __shared__ int s_warp[8], s_find[5];
  __shared__ float s_top[kHeads], s_sum[kHeads];
  __shared__ float4 s_y[256];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, hkv = p.c.hkv, vals = p.group * D;
  // the kernels before the main one are done: it began this launch after its own wait for them
  const int per = (p.nreq + 255) / 256, rq0 = min(tid * per, p.nreq), rq1 = min(rq0 + per, p.nreq);
  int mine = 0;
  for (int r = rq0; r < rq1; ++r) mine += (kv4_length(p, r) + kKv4Tile - 1) / kKv4Tile;
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  if (lane == 31) s_warp[warp] = inc;
  if (tid == 0) s_find[0] = s_find[1] = s_find[2] = s_find[3] = 0, s_find[4] = 1;
  __syncthreads();
  int base = inc - mine, total = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    if (w < warp) base += s_warp[w];
    total += s_warp[w];
  }
  const int cost = (2 * total + p.nreq) * hkv;
  const int ctas = min(ctas_max, max(1, cost / kKv4MinCost)), cta = blockIdx.x;
  // a block leaves only after the main kernel: the next launch waits for this one alone
  if (cta + 1 >= ctas || total == 0) {
    pdl_wait();
    return;
  }
  const int each = cost / ctas, more = cost - each * ctas;
  const int x0 = each * cta + min(cta, more), x1 = x0 + each + (cta < more ? 1 : 0);
  // tiles before this CTA's run and before the next one's
  for (int r = rq0, b = base; r < rq1; ++r) {
    const int n = (kv4_length(p, r) + kKv4Tile - 1) / kKv4Tile, seg = 2 * n + 1;
    const int y0 = x0 - (2 * b + r) * hkv, y1 = x1 - (2 * b + r) * hkv;
    if (y0 >= 0 && y0 < seg * hkv) s_find[0] = b * hkv + y0 / seg * n + kv4_tiles_before(y0 % seg, n);
    if (y1 >= 0 && y1 < seg * hkv) s_find[1] = b * hkv + y1 / seg * n + kv4_tiles_before(y1 % seg, n);
    b += n;
  }
  __syncthreads();
  const int u0 = s_find[0], end = s_find[1];
  // the request of the CTA's last tile
  for (int r = rq0, b = base; r < rq1; ++r) {
    const int n = (kv4_length(p, r) + kKv4Tile - 1) / kKv4Tile;
    if (n && b * hkv < end && end <= (b + n) * hkv) {
      s_find[2] = r;
      s_find[3] = b;
      s_find[4] = n;
    }
    b += n;
  }
  __syncthreads();
  const int r = s_find[2], nt = s_find[4];
  const int g = u0 < end ? (end - 1 - s_find[3] * hkv) / nt : 0, first = s_find[3] * hkv + g * nt, stop = first + nt;
  if (u0 == end || first < u0 || stop <= end) {  // no tiles, begun earlier, or finished here
    pdl_wait();
    return;
  }
  const int xl = (2 * s_find[3] + r) * hkv + g * (2 * nt + 1) + (nt == 1 ? 0 : 2 * nt - 1);  // where its last tile's cost begins
  const int last = xl < more * (each + 1) ? xl / (each + 1) : more + (xl - more * (each + 1)) / each;
  const int parts = last - cta + 1, pf = kv4_piece_floats(p.group, D);
  const int v0 = blockIdx.y * kVals, h0 = v0 / D;  // this block's values and heads of the group
  // part 0: slot 1 of the CTA it begins in, then slot 0 of those after it
  auto part_at = [&](int j) { return p.part + (static_cast<int64_t>(cta + j) * 2 + (j == 0 ? 1 : 0)) * pf; };
  pdl_wait();
  pdl_launch_dependents();
  const int e = v0 + 4 * (tid & 63), sl = tid >> 6;
  const bool in = e < vals;
  float4 ahead[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if (in && sl + 4 * i < parts) ahead[i] = __ldcg(reinterpret_cast<const float4*>(part_at(sl + 4 * i) + e));
  if (warp < kHeads && h0 + warp < p.group) {
    const int u = h0 + warp;
    float top = -INFINITY;
    for (int j = lane; j < parts; j += 32) {
      const float m = __ldcg(part_at(j) + vals + u);
      s_w[j * kHeads + warp] = m;
      top = fmaxf(top, m);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float sum = 0.0f;
    for (int j = lane; j < parts; j += 32) {
      const float w = kv4_ex2(s_w[j * kHeads + warp] - (top == -INFINITY ? 0.0f : top));
      s_w[j * kHeads + warp] = w;
      sum = fmaf(w, __ldcg(part_at(j) + vals + p.group + u), sum);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
      s_top[warp] = top;
      s_sum[warp] = sum;
    }
  }
  __syncthreads();
  float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const int hh = (e - v0) / D;
  auto add = [&](int j, float4 v) {
    const float f = s_w[j * kHeads + hh];
    y.x = fmaf(f, v.x, y.x);
    y.y = fmaf(f, v.y, y.y);
    y.z = fmaf(f, v.z, y.z);
    y.w = fmaf(f, v.w, y.w);
  };
  if (in) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (sl + 4 * i < parts) add(sl + 4 * i, ahead[i]);
#pragma unroll 6
    for (int j = sl + 4 * kAhead; j < parts; j += 4) add(j, __ldcg(reinterpret_cast<const float4*>(part_at(j) + e)));
  }
  s_y[tid] = y;
  __syncthreads();
  if (sl == 0 && in) {
#pragma unroll
    for (int k = 1; k < 4; ++k) {
      const float4 v = s_y[64 * k + tid];
      y.x += v.x;
      y.y += v.y;
      y.z += v.z;
      y.w += v.w;
    }
    const float sum = s_sum[hh], f = sum == 0.0f ? 0.0f : 1.0f / sum;
    store4(static_cast<T*>(p.out) + r * p.ldo + static_cast<int64_t>(g) * vals + e, y.x * f, y.y * f, y.z * f, y.w * f);
    if (e % D == 0 && p.lse)
      p.lse[static_cast<int64_t>(r) * p.hq + g * p.group + h0 + hh] =
          sum == 0.0f ? -INFINITY : (s_top[hh] + log2f(sum)) * 0.6931471805599453f;
  }
}

}  // namespace tg

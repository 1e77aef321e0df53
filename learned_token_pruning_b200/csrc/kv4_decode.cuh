// Decode attention over the paged 4-bit KV cache: for each request the new
// token's query heads over its cached rows,
//     l_c = temp_h ratio_r sm_scale (q_h . k_c) + gain_h bias_c,  out_h = sum_c softmax_c(l) v_c,
// with k_c and v_c the values the 4-bit rows stand for.  A key whose bias is
// -infinity is left out altogether, whatever its row holds; a request without
// keys gets zeros (lse -infinity).
//
// The cache is read once and the step is bound by memory: 2 (D/2 + D/16) bytes per
// row and KV head, a third of bf16.  What stands in the way is the work per value,
// so the products run on the tensor cores through the warp-level matrix
// instruction (m16n8k16, fp16 in, fp32 out).  Its operands come from registers,
// where the codes are widened with one conversion per two values; the wide
// tcgen05 form would need them written back to shared memory first, and its
// 128-row tiles have nothing to fill them with at 1 to 8 query heads.
//
//   Keys and values are the A operand (16 keys or 16 dimensions x 16), the query
//   heads and the weights the B operand (8 columns).  E2M1 codes are exact in
//   fp16, and the scales stay outside: per group of 32 dimensions the scores are
//   accumulated on their own and added up times the key's scale in fp32, and the
//   weights are multiplied by the value row's scale before they are rounded to
//   fp16 (11 bits; fp32 queries carry query and weights as two fp16 parts, 22 bits).
//   Both factors meet a power of two that keeps them in fp16's range: the query one
//   per head (its largest value lands at 2^8), the weights one per head and scale
//   group (weight 1 times the largest value scale met so far lands at 2^14; the
//   running exponent moves with the running maximum of the softmax).
//   The 8 columns hold HP heads (2, 4 or 8) times 8 / HP scale groups: with two
//   heads, one B operand serves all four groups of D = 128.  A lane reads the
//   accumulator columns of its own group and leaves the others.
//
// Work split: the (request, KV head, 64-key tile) units are laid out in that
// order and cut into equal runs, one per warp, so ragged batches are balanced to a tile.
// Every warp streams its own run through a ring in shared memory by bulk copies
// (a page holds a head's rows contiguously; no barrier between warps), keeps its own
// online softmax, and writes a result directly when a (request, head) lies
// inside its run.  Pieces of longer ones are merged per CTA in shared memory and
// then, where they cross CTAs, by the CTA that arrives last, always in order of
// position: reruns are bit-identical.
#pragma once

#include "common.cuh"
#include "kv4.cuh"

namespace tg {

constexpr int kKv4MaxGroup = 8;
constexpr int kKv4Warps = 8;
constexpr int kKv4Stages = 2;
constexpr int kKv4Tile = 64;  // keys per unit

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
  float* part;         // [CTAs][2][group * (D + 2)]
  unsigned* counters;  // [CTAs], zero between calls
};

// one piece of a (request, head): group rows of D sums, then the maxima, then the weight sums
__host__ __device__ constexpr int kv4_piece_floats(int group, int d) { return (group * (d + 2) + 3) / 4 * 4; }

template <int D>
struct Kv4Stage {
  static constexpr int kCodes = kKv4Tile * D / 2, kScales = kKv4Tile * D / 16;
  static constexpr int kVCodes = kCodes, kKScales = 2 * kCodes, kVScales = kKScales + kScales;
  static constexpr int kBias = kVScales + kScales, kBytes = kBias + kKv4Tile * 4;
};

__host__ __device__ constexpr size_t kv4_decode_head_smem(int nreq) {  // tile prefix sums
  return static_cast<size_t>(nreq + 1 + 31) / 32 * 128;
}
template <int D>
constexpr size_t kv4_decode_smem(int nreq, int group) {
  return kv4_decode_head_smem(nreq) + static_cast<size_t>(kKv4Warps) * kKv4Stages * Kv4Stage<D>::kBytes +
         static_cast<size_t>(kKv4Warps) * kv4_piece_floats(group, D) * 4;
}

__device__ __forceinline__ float kv4_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float exp_bits(int field) { return __uint_as_float(static_cast<uint32_t>(field) << 23); }

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
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
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

template <typename T, int D, int HP>
__global__ void __launch_bounds__(32 * kKv4Warps, 1) k_kv4_decode(const Kv4DecodeParams p) {
  using St = Kv4Stage<D>;
  constexpr bool kSplit = sizeof(T) == 4;      // fp32: query and weights in two fp16 parts
  constexpr int NG = D / 32, SL = 8 / HP, NB = NG > SL ? NG / SL : 1;
  constexpr int S = kKv4Stages, TP = 32 * kKv4Warps;
  constexpr int kSwap = D == 128 ? 1 : 2;      // key order inside 16 rows, see below
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t s_full[kKv4Warps][S];
  __shared__ int s_warp[kKv4Warps];
  __shared__ int s_seg[kKv4Warps][2];          // (request, head) of the warp's unfinished pieces, -1: none
  __shared__ int s_edge[kKv4Warps][2];         // bit 0: the piece begins the (request, head), bit 1: it ends it
  __shared__ int s_stop, s_last[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, t = lane & 3, n8 = lane >> 2;
  int* s_cum = reinterpret_cast<int*>(smem);   // [nreq + 1] tiles of the requests before
  uint8_t* ring = smem + kv4_decode_head_smem(p.nreq) + static_cast<size_t>(warp) * S * St::kBytes;
  float* piece0 = reinterpret_cast<float*>(smem + kv4_decode_head_smem(p.nreq) +
                                           static_cast<size_t>(kKv4Warps) * S * St::kBytes) +
                  warp * kv4_piece_floats(p.group, D);
  const int hkv = p.c.hkv, P = p.c.page_rows, group = p.group;

  if (lane < S) mbar_init(&s_full[warp][lane], 1);
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
  for (int w = 0; w < kKv4Warps; ++w) {
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

  // ---- this warp's run of units
  const int64_t units = static_cast<int64_t>(total) * hkv;
  const int64_t ctas = min(static_cast<int64_t>(gridDim.x), units), cta = blockIdx.x;
  if (cta >= ctas) return;
  const int64_t u0 = units * cta / ctas, u1 = units * (cta + 1) / ctas;
  const int64_t ua = u0 + (u1 - u0) * warp / kKv4Warps, ub = u0 + (u1 - u0) * (warp + 1) / kKv4Warps;
  const int left = static_cast<int>(ub - ua);  // units to compute

  // position of the next unit to load: request, head, tile, the request's rows
  const int prow = min(P, kKv4Tile), np = kKv4Tile / prow;  // rows of a page in a tile, pages in a tile
  int lr = 0, lg = 0, lt = 0, llen = 0;
  if (left > 0) {
    int lo = 0, hi = p.nreq - 1;  // largest request that starts at or before ua
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (static_cast<int64_t>(s_cum[mid]) * hkv <= ua) lo = mid;
      else hi = mid - 1;
    }
    lr = lo;
    const int nt = s_cum[lr + 1] - s_cum[lr];
    const int x = static_cast<int>(ua - static_cast<int64_t>(s_cum[lr]) * hkv);
    lg = x / nt;
    lt = x - lg * nt;
    llen = kv4_length(p, lr);
  }
  int cr = lr, cg = lg, ct = lt, clen = llen;  // position of the unit being computed
  auto advance = [&](int& r, int& g, int& tt, int& len) {
    if (++tt < (len + kKv4Tile - 1) / kKv4Tile) return;
    tt = 0;
    if (++g < hkv) return;
    g = 0;
    do ++r; while (r < p.nreq && s_cum[r + 1] == s_cum[r]);
    len = r < p.nreq ? kv4_length(p, r) : 0;
  };
  // lane i moves array i / np of page i % np: K codes, V codes, K scales, V scales, biases
  const int what = lane / np, piece = lane % np;
  auto page_id = [&](int r, int tt, int len) -> int32_t {
    const int row = tt * kKv4Tile + piece * prow;
    if (what > 4 || row >= len) return 0;
    return p.tables[static_cast<int64_t>(r) * p.max_pages + (row >> p.c.page_shift)];
  };
  auto load = [&](int st, int r, int g, int tt, int len, int32_t page) {
    const int rows = min(kKv4Tile, len - tt * kKv4Tile), pieces = (rows + prow - 1) / prow;
    if (lane == 0)
      mbar_arrive_expect_tx(&s_full[warp][st], pieces * prow * (D + D / 8 + (p.c.bias ? 4 : 0)));
    __syncwarp();
    if (what <= (p.c.bias ? 4 : 3) && piece < pieces) {
      if (page < 0 || page >= p.c.num_pages) {
        raise_error(kErrKvPage, 2);
        page = 0;
      }
      const int off = (tt * kKv4Tile) & (P - 1);  // 0 unless a page holds several tiles
      const int64_t row = ((static_cast<int64_t>(page) * hkv + g) << p.c.page_shift) + off;
      uint8_t* dst = ring + st * St::kBytes;
      const void* src;
      uint32_t bytes;
      if (what < 2) {
        src = (what ? p.c.v_codes : p.c.k_codes) + row * (D / 2);
        bytes = prow * (D / 2);
        dst += what * St::kVCodes + piece * bytes;
      } else if (what < 4) {
        src = (what == 3 ? p.c.v_scales : p.c.k_scales) + row * (D / 32);
        bytes = prow * (D / 16);
        dst += (what == 3 ? St::kVScales : St::kKScales) + piece * bytes;
      } else {
        src = p.c.bias + ((static_cast<int64_t>(page) << p.c.page_shift) + off);
        bytes = prow * 4;
        dst += St::kBias + piece * bytes;
      }
      bulk_load(dst, src, bytes, &s_full[warp][st]);
    }
  };

  // ---- per-lane state.  Accumulator columns 2t, 2t + 1 are heads hd, hd + 1 of scale
  // group slot `slot`; accumulator rows n8 and n8 + 8 are keys (scores) or dimensions.
  const int hd = (2 * t) % HP, slot = 2 * t / HP;
  // Row i of a score tile is key key_of(i): even rows keys i / 2, odd rows the other
  // four, ordered so that the 16-byte key loads of 8 lanes and the value loads of
  // 4 keys x 4 lanes both spread over all banks (values: lane t takes the keys of
  // rows 2t, 2t + 1, 2t + 8, 2t + 9).
  const int key0 = n8 & 1 ? 4 + ((n8 >> 1) ^ kSwap) : n8 >> 1;
  const int kswz = D == 128 ? (key0 & 2) << 4 : 0, vswz = D == 128 ? (t & 2) << 4 : 0;
  const uint32_t kbase = smem_u32(ring) + key0 * (D / 2) + ((t * (D / 8)) ^ kswz);
  const uint32_t vbase = smem_u32(ring) + St::kVCodes + ((n8 * (D / 16)) ^ vswz);
  const int va = t, vb = 4 + (t ^ kSwap);

  uint32_t qf[kSplit ? 2 : 1][NG][2][2];
  float o[NG][2][4];
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f, a0 = 0.0f, a1 = 0.0f, g0 = 0.0f, g1 = 0.0f;
  int ex[NB];

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
    m0 = m1 = -INFINITY;
    l0 = l1 = 0.0f;
#pragma unroll
    for (int b = 0; b < NB; ++b) ex[b] = 15;  // 2^(141 - ex) and its inverse are both normal floats from here on
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
      const float unit = exp_bits(ex[g / SL] - 14);  // 2^(ex - 141)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (hd + c >= group) continue;
        const float f = c ? f1 : f0;
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
    // fill the ring: the page ids first, so that their loads overlap
    int32_t first_page[S], next_page = 0;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      first_page[i] = i < left ? page_id(lr, lt, llen) : 0;
      if (i < left) advance(lr, lg, lt, llen);
    }
    if (S < left) next_page = page_id(lr, lt, llen);
    int fr = cr, fg = cg, ft = ct, flen = clen;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      if (i < left) {
        load(i, fr, fg, ft, flen, first_page[i]);
        advance(fr, fg, ft, flen);
      }
    }
    bool first_unit = true;
    int begun = ct == 0;  // the current (request, head) begins in this run
    for (int i = 0; i < left; ++i) {
      if (first_unit || ct == 0) begin();
      first_unit = false;
      const int st = i % S;
      ok = warp_wait(&s_full[warp][st], (i / S) & 1, kErrWaitAttention);
      if (!ok) break;
      const uint32_t stage = st * St::kBytes;
      const uint8_t* sp = ring + stage;
      const int rows = min(kKv4Tile, clen - ct * kKv4Tile);

      // ---- scores of 64 keys
      float x[4][4];
      bool live0[4], live1[4];
      float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        uint32_t w0[NG], w1[NG];  // halves (unit 2t: groups 0..), (unit 2t + 1: groups 0..)
        const uint32_t ka = kbase + stage + mt * 16 * (D / 2);
        if constexpr (D == 128) {
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w0[0]), "=r"(w0[1]), "=r"(w0[2]), "=r"(w0[3]) : "r"(ka));
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w1[0]), "=r"(w1[1]), "=r"(w1[2]), "=r"(w1[3]) : "r"(ka + 8 * (D / 2)));
        } else {
          asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w0[0]), "=r"(w0[1]) : "r"(ka));
          asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w1[0]), "=r"(w1[1]) : "r"(ka + 8 * (D / 2)));
        }
        uint32_t h0[NG][4], h1[NG][4];  // [word][byte]: word s * NG / 2 + g / 2, bytes 2 (g & 1), + 1
#pragma unroll
        for (int w = 0; w < NG; ++w) {
          e2m1x8(w0[w], h0[w]);
          e2m1x8(w1[w], h1[w]);
        }
        const int key = mt * 16 + key0;
        uint32_t sc0[NG / 2], sc1[NG / 2];  // bf16 scale pairs of both keys
#pragma unroll
        for (int g = 0; g < NG / 2; ++g) {
          sc0[g] = *reinterpret_cast<const uint32_t*>(sp + St::kKScales + key * (D / 16) + 4 * g);
          sc1[g] = *reinterpret_cast<const uint32_t*>(sp + St::kKScales + (key + 8) * (D / 16) + 4 * g);
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const int w = s * (NG / 2) + g / 2, b = 2 * (g & 1);
#pragma unroll
            for (int v = 0; v < (kSplit ? 2 : 1); ++v)
              mma_f16(acc, h0[w][b], h1[w][b], h0[w][b + 1], h1[w][b + 1], qf[v][g][s][0], qf[v][g][s][1]);
          }
          const float k0 = g & 1 ? bf16_hi(sc0[g / 2]) : bf16_lo(sc0[g / 2]);
          const float k1 = g & 1 ? bf16_hi(sc1[g / 2]) : bf16_lo(sc1[g / 2]);
          x[mt][0] = g ? fmaf(k0, acc[0], x[mt][0]) : k0 * acc[0];
          x[mt][1] = g ? fmaf(k0, acc[1], x[mt][1]) : k0 * acc[1];
          x[mt][2] = g ? fmaf(k1, acc[2], x[mt][2]) : k1 * acc[2];
          x[mt][3] = g ? fmaf(k1, acc[3], x[mt][3]) : k1 * acc[3];
        }
        float bias0 = 0.0f, bias1 = 0.0f;
        if (p.c.bias) {
          bias0 = *reinterpret_cast<const float*>(sp + St::kBias + 4 * key);
          bias1 = *reinterpret_cast<const float*>(sp + St::kBias + 4 * key + 32);
        }
        live0[mt] = key < rows && bias0 != -INFINITY;
        live1[mt] = key + 8 < rows && bias1 != -INFINITY;
        x[mt][0] = live0[mt] ? fmaf(a0, x[mt][0], g0 * bias0) : -INFINITY;
        x[mt][1] = live0[mt] ? fmaf(a1, x[mt][1], g1 * bias0) : -INFINITY;
        x[mt][2] = live1[mt] ? fmaf(a0, x[mt][2], g0 * bias1) : -INFINITY;
        x[mt][3] = live1[mt] ? fmaf(a1, x[mt][3], g1 * bias1) : -INFINITY;
        t0 = fmaxf(t0, fmaxf(x[mt][0], x[mt][2]));
        t1 = fmaxf(t1, fmaxf(x[mt][1], x[mt][3]));
      }

      // ---- running maxima of the logits and of the value scales' exponents
      uint32_t vs0[4][NB], vs1[4][NB];  // bf16 value scales of this lane's groups, as fp32 bits
      uint32_t vtop[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) vtop[b] = 0;
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const int key = mt * 16 + key0, g = b * SL + slot;
          const uint32_t s0 = *reinterpret_cast<const uint16_t*>(sp + St::kVScales + key * (D / 16) + 2 * g);
          const uint32_t s1 = *reinterpret_cast<const uint16_t*>(sp + St::kVScales + (key + 8) * (D / 16) + 2 * g);
          vs0[mt][b] = live0[mt] ? s0 << 16 : 0u;
          vs1[mt][b] = live1[mt] ? s1 << 16 : 0u;
          vtop[b] = max(vtop[b], max(vs0[mt][b], vs1[mt][b]));
        }
      t0 = rows_max(t0);
      t1 = rows_max(t1);
      const float n0 = fmaxf(m0, t0), n1 = fmaxf(m1, t1);
      bool moved = n0 != m0 || n1 != m1;
      int nex[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        uint32_t v = vtop[b];
        v = max(v, __shfl_xor_sync(0xffffffffu, v, 4));
        v = max(v, __shfl_xor_sync(0xffffffffu, v, 8));
        v = max(v, __shfl_xor_sync(0xffffffffu, v, 16));
        nex[b] = max(ex[b], min(static_cast<int>(v >> 23), 254));  // NaN scales (255) set no unit
        moved |= nex[b] != ex[b];
      }
      const float use0 = n0 == -INFINITY ? 0.0f : n0, use1 = n1 == -INFINITY ? 0.0f : n1;
      if (__any_sync(0xffffffffu, moved)) {
        const float d0 = m0 - use0, d1 = m1 - use1;
        l0 *= kv4_ex2(d0);
        l1 *= kv4_ex2(d1);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const float de = static_cast<float>(ex[g / SL] - nex[g / SL]);
          const float c0 = kv4_ex2(d0 + de), c1 = kv4_ex2(d1 + de);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            o[g][j][0] *= c0;
            o[g][j][1] *= c1;
            o[g][j][2] *= c0;
            o[g][j][3] *= c1;
          }
        }
        m0 = n0;
        m1 = n1;
#pragma unroll
        for (int b = 0; b < NB; ++b) ex[b] = nex[b];
      }
      float fac[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) fac[b] = exp_bits(268 - ex[b]);  // 2^(141 - ex)

      // ---- weights, and their products with the values
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        const float p00 = kv4_ex2(x[mt][0] - use0), p01 = kv4_ex2(x[mt][1] - use1);
        const float p10 = kv4_ex2(x[mt][2] - use0), p11 = kv4_ex2(x[mt][3] - use1);
        l0 += p00 + p10;
        l1 += p01 + p11;
        uint32_t pf[kSplit ? 2 : 1][NB][2];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const float s0 = __uint_as_float(vs0[mt][b]) * fac[b], s1 = __uint_as_float(vs1[mt][b]) * fac[b];
          const float w00 = p00 * s0, w01 = p01 * s0, w10 = p10 * s1, w11 = p11 * s1;
          const uint32_t r0 = f16x2(w00, w01), r1 = f16x2(w10, w11);
          pf[0][b][0] = transpose8x8(r0);
          pf[0][b][1] = transpose8x8(r1);
          if constexpr (kSplit) {
            pf[1][b][0] = transpose8x8(f16x2(w00 - f16_lo(r0), w01 - f16_hi(r0)));
            pf[1][b][1] = transpose8x8(f16x2(w10 - f16_lo(r1), w11 - f16_hi(r1)));
          }
        }
        const uint32_t va0 = vbase + stage + (mt * 16 + va) * (D / 2), vb0 = vbase + stage + (mt * 16 + vb) * (D / 2);
        uint32_t wa[NG / 2], wb[NG / 2], wc[NG / 2], wd[NG / 2];
        if constexpr (D == 128) {
          asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(wa[0]), "=r"(wa[1]) : "r"(va0));
          asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(wb[0]), "=r"(wb[1]) : "r"(vb0));
          asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(wc[0]), "=r"(wc[1]) : "r"(va0 + 8 * (D / 2)));
          asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(wd[0]), "=r"(wd[1]) : "r"(vb0 + 8 * (D / 2)));
        } else {
          asm volatile("ld.shared.u32 %0, [%1];" : "=r"(wa[0]) : "r"(va0));
          asm volatile("ld.shared.u32 %0, [%1];" : "=r"(wb[0]) : "r"(vb0));
          asm volatile("ld.shared.u32 %0, [%1];" : "=r"(wc[0]) : "r"(va0 + 8 * (D / 2)));
          asm volatile("ld.shared.u32 %0, [%1];" : "=r"(wd[0]) : "r"(vb0 + 8 * (D / 2)));
        }
#pragma unroll
        for (int w = 0; w < NG / 2; ++w) {
          // low nibbles of two keys side by side, then the high ones: byte 2i + j holds
          // dimensions 2j (lo) or 2j + 1 (hi) of group 2w + i for both keys
          constexpr uint32_t M = 0x0f0f0f0fu;
          uint32_t loab[4], hiab[4], locd[4], hicd[4];
          e2m1x8((wa[w] & M) | (wb[w] << 4 & ~M), loab);
          e2m1x8((wa[w] >> 4 & M) | (wb[w] & ~M), hiab);
          e2m1x8((wc[w] & M) | (wd[w] << 4 & ~M), locd);
          e2m1x8((wc[w] >> 4 & M) | (wd[w] & ~M), hicd);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int v = 0; v < (kSplit ? 2 : 1); ++v)
                mma_f16(o[2 * w + i][j], loab[2 * i + j], hiab[2 * i + j], locd[2 * i + j], hicd[2 * i + j],
                        pf[v][(2 * w + i) / SL][0], pf[v][(2 * w + i) / SL][1]);
        }
      }
      __syncwarp();  // every lane has read the stage
      if (i + S < left) {
        load(st, lr, lg, lt, llen, next_page);
        advance(lr, lg, lt, llen);
        if (i + S + 1 < left) next_page = page_id(lr, lt, llen);
      }
      const bool ends = (ct + 1) * kKv4Tile >= clen;
      if (ends || i + 1 == left) {
        if (begun && ends) {
          finish(true, nullptr);
        } else {
          // a piece: one that begins here ends the run, so the ring is free for it
          float* dst = begun ? reinterpret_cast<float*>(ring) : piece0;
          finish(false, dst);
          if (lane == 0) {
            s_seg[warp][begun] = cr * hkv + cg;
            s_edge[warp][begun] = begun | (ends ? 2 : 0);
          }
        }
        begun = 1;
      }
      advance(cr, cg, ct, clen);
    }
  }
  if (!ok && lane == 0) s_stop = 1;
  __syncthreads();
  if (s_stop) return;  // a wait ran out (recorded in the error word)

  // ---- pieces of this CTA, in order of position, to the output or to the workspace
  const int pf4 = kv4_piece_floats(group, D);
  float* pieces = reinterpret_cast<float*>(smem + kv4_decode_head_smem(p.nreq) +
                                           static_cast<size_t>(kKv4Warps) * S * St::kBytes);
  auto piece_at = [&](int i) -> const float* {  // piece i: warp i / 2, slot i % 2
    return i & 1 ? reinterpret_cast<const float*>(smem + kv4_decode_head_smem(p.nreq) +
                                                  static_cast<size_t>(i >> 1) * S * St::kBytes)
                 : pieces + (i >> 1) * pf4;
  };
  int open[2] = {-1, -1};  // (request, head) continued from an earlier CTA, and into a later one
  for (int i = 0; i < 2 * kKv4Warps;) {
    const int seg = s_seg[i >> 1][i & 1];
    if (seg < 0) {
      ++i;
      continue;
    }
    int end = i + 1, last = i;
    while (end < 2 * kKv4Warps && (s_seg[end >> 1][end & 1] == seg || s_seg[end >> 1][end & 1] < 0)) {
      if (s_seg[end >> 1][end & 1] == seg) last = end;
      ++end;
    }
    const bool begins = s_edge[i >> 1][i & 1] & 1, whole = begins && (s_edge[last >> 1][last & 1] & 2);
    const int r = seg / hkv, h0 = seg % hkv * group;
    float* part = p.part + (cta * 2 + (begins ? 1 : 0)) * pf4;
    for (int e = tid; e < group * D; e += TP) {
      const int u = e / D;
      float top = -INFINITY;
      for (int k = i; k <= last; ++k)
        if (s_seg[k >> 1][k & 1] == seg) top = fmaxf(top, piece_at(k)[group * D + u]);
      const float use = top == -INFINITY ? 0.0f : top;
      float y = 0.0f, sum = 0.0f;
      for (int k = i; k <= last; ++k)
        if (s_seg[k >> 1][k & 1] == seg) {
          const float* pc = piece_at(k);
          const float f = kv4_ex2(pc[group * D + u] - use);
          y = fmaf(f, pc[e], y);
          sum = fmaf(f, pc[group * (D + 1) + u], sum);
        }
      if (whole) {
        static_cast<T*>(p.out)[r * p.ldo + static_cast<int64_t>(h0) * D + e] = from_f32<T>(sum == 0.0f ? 0.0f : y / sum);
        if (e % D == 0 && p.lse)
          p.lse[static_cast<int64_t>(r) * p.hq + h0 + u] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
      } else {
        part[e] = y;
        if (e % D == 0) {
          part[group * D + u] = top;
          part[group * (D + 1) + u] = sum;
        }
      }
    }
    if (!whole) open[begins] = seg;
    i = end;
  }

  // ---- (request, head)s that cross CTAs: the last CTA to arrive adds the parts in CTA order
  if (open[0] < 0 && open[1] < 0) return;
  __threadfence();
  __syncthreads();
  int64_t c0[2], c1[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int r = max(open[k], 0) / hkv, g = max(open[k], 0) % hkv;
    const int nt = s_cum[r + 1] - s_cum[r];
    const int64_t first = static_cast<int64_t>(s_cum[r]) * hkv + static_cast<int64_t>(g) * nt;
    c0[k] = ((first + 1) * ctas - 1) / units;     // CTA of a unit u: the largest c with units * c / ctas <= u
    c1[k] = ((first + nt) * ctas - 1) / units;
    if (tid == 0)
      s_last[k] = open[k] >= 0 && atomicAdd(&p.counters[c0[k]], 1u) == static_cast<unsigned>(c1[k] - c0[k]);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (!s_last[k]) continue;
    __threadfence();
    const int r = open[k] / hkv, h0 = open[k] % hkv * group, cnt = static_cast<int>(c1[k] - c0[k]) + 1;
    const float* first = p.part + (c0[k] * 2 + 1) * pf4;          // begins in CTA c0: its slot 1
    const float* rest = p.part + (c0[k] + 1) * 2 * pf4;           // then slot 0 of the CTAs after it
    for (int e = tid; e < group * D; e += TP) {
      const int u = e / D;
      float top = __ldcg(first + group * D + u);
      for (int j = 0; j < cnt - 1; ++j) top = fmaxf(top, __ldcg(rest + static_cast<int64_t>(j) * 2 * pf4 + group * D + u));
      const float use = top == -INFINITY ? 0.0f : top;
      float f = kv4_ex2(__ldcg(first + group * D + u) - use);
      float y = f * __ldcg(first + e), sum = f * __ldcg(first + group * (D + 1) + u);
#pragma unroll 4
      for (int j = 0; j < cnt - 1; ++j) {
        const float* pc = rest + static_cast<int64_t>(j) * 2 * pf4;
        f = kv4_ex2(__ldcg(pc + group * D + u) - use);
        y = fmaf(f, __ldcg(pc + e), y);
        sum = fmaf(f, __ldcg(pc + group * (D + 1) + u), sum);
      }
      static_cast<T*>(p.out)[r * p.ldo + static_cast<int64_t>(h0) * D + e] = from_f32<T>(sum == 0.0f ? 0.0f : y / sum);
      if (e % D == 0 && p.lse)
        p.lse[static_cast<int64_t>(r) * p.hq + h0 + u] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
    }
    if (tid == 0) p.counters[c0[k]] = 0u;  // ready for the next call
  }
}

}  // namespace tg

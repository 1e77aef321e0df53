// Per-head RMSNorm of q and k with the position rotation in the same pass, and
// its gradients.  With x a head row, r = 1 / sqrt(mean x^2 + eps), w the norm
// weight, R the rotate-half rotation by the angles pos * theta^(-2i/D):
//     y = R (x r w)
//     g = R^T dy,  dw = sum over rows and heads of g x r,
//     dx = r g w - x r^3 mean(g w x)
// The angle is formed and reduced modulo 2 pi in double (positions reach 2^31),
// sine and cosine of the remainder are taken in fp32; every other value and sum
// is fp32, rounded once on the way out.
//
// A lane owns the dimension pairs (8j + i, D/2 + 8j + i), i < 8, of a head: two
// 16-byte loads in bf16, and the rotation needs no exchange between lanes.  D/16
// lanes hold a head, so a warp takes 4 (D = 128) or 8 heads of one row at a
// time; the row's cosines and sines are computed once per warp and shared by its
// heads through shared memory.
#pragma once

#include "common.cuh"
#include "kv4.cuh"
#include "simt.cuh"

namespace tg {

constexpr int kRopeWarps = 8;

struct QkRopeParams {
  const void* q;
  const void* k;
  int64_t ldq, ldk;
  int64_t m;
  int hq, hkv;
  const int32_t* pos;
  const float* wq;   // null: ones
  const float* wk;
  int qk_norm;
  float eps;
  void* q_out;       // forward: rotated rows; backward: input gradients
  void* k_out;
  int64_t ldqo, ldko;
  const float* dq;   // backward: upstream gradients, contiguous rows
  const float* dk;
  float* part;       // backward: [blocks][2][D] partial norm-weight gradients, or null
  int split;         // warps that share one row: 1, or one for each of its passes
};

// A pass: the warp's 4 (D = 128) or 8 heads of q, or of k; a row is its passes of q, then of k.
template <int D>
struct RopePasses {
  static constexpr int kLanes = D / 16, kHeads = 32 / kLanes;  // lanes of a head, heads of a pass
  int of_q, all;
  __host__ __device__ RopePasses(int hq, int hkv)
      : of_q((hq + kHeads - 1) / kHeads), all(of_q + (hkv + kHeads - 1) / kHeads) {}
};

// cos and sin of the row's D/2 angles into the warp's table
template <int D>
__device__ __forceinline__ void rope_table(float2* cs, int32_t pos, const RopeTable& tab) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int e = 0; e < D / 64; ++e) {
    const double ang = static_cast<double>(pos) * tab.inv_freq[e * 32 + lane];
    const double turns = rint(ang * 0.15915494309189535);  // 1 / (2 pi)
    const float red = static_cast<float>(fma(-turns, 6.283185307179586, ang));
    float s, c;
    sincosf(red, &s, &c);
    cs[e * 32 + lane] = make_float2(c, s);
  }
}

template <int D>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = D / 32; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// eight values as they lie in memory, loaded ahead of their use
template <typename T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) w[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const { load8(reinterpret_cast<const T*>(w), x); }
};

__device__ __forceinline__ void weights8(const float* w, float (&x)[8]) {
  if (w) {
    x[0] = w[0], x[1] = w[1], x[2] = w[2], x[3] = w[3], x[4] = w[4], x[5] = w[5], x[6] = w[6], x[7] = w[7];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 1.0f;
  }
}

// The first loads of a row are on their way while its angles are formed, and as many passes
// as registers allow at a time, since a pass alone keeps 1 KB of a warp's loads in flight.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kRopeWarps, 2) k_qk_rope_fwd(const QkRopeParams p,
                                                                    const __grid_constant__ RopeTable tab) {
  constexpr int LH = RopePasses<D>::kLanes, HW = RopePasses<D>::kHeads, CH = sizeof(T) == 2 ? 3 : 2;
  __shared__ float2 s_cs[kRopeWarps][D / 2];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane % LH, sub = lane / LH;
  const RopePasses<D> passes(p.hq, p.hkv);
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kRopeWarps + warp, row = item / p.split;
  if (row >= p.m) return;  // warp-uniform
  const int step = p.split == 1 ? 1 : passes.all;
  const int32_t pos = p.pos[row];
  const T* q = static_cast<const T*>(p.q) + row * p.ldq + 8 * j;
  const T* k = static_cast<const T*>(p.k) + row * p.ldk + 8 * j;
  T* qo = static_cast<T*>(p.q_out) + row * p.ldqo + 8 * j;
  T* ko = static_cast<T*>(p.k_out) + row * p.ldko + 8 * j;
  float c[8], s[8], wa[8], wb[8];
  bool angles = false;
  int weights = -1;  // whose weights are loaded: 0 q, 1 k
  for (int i0 = static_cast<int>(item - row * p.split); i0 < passes.all; i0 += CH * step) {
    Raw8<T> xa[CH], xb[CH];
#pragma unroll
    for (int u = 0; u < CH; ++u) {
      const int i = i0 + u * step;
      const bool isk = i >= passes.of_q;
      const int h = (isk ? i - passes.of_q : i) * HW + sub;
      xa[u].zero();
      xb[u].zero();
      if (i < passes.all && h < (isk ? p.hkv : p.hq)) {
        const T* x = (isk ? k : q) + static_cast<int64_t>(h) * D;
        xa[u].load(x);
        xb[u].load(x + D / 2);
      }
    }
    if (!angles) {
      angles = true;
      rope_table<D>(s_cs[warp], pos, tab);
      __syncwarp();
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 v = s_cs[warp][8 * j + e];
        c[e] = v.x;
        s[e] = v.y;
      }
    }
#pragma unroll
    for (int u = 0; u < CH; ++u) {
      const int i = i0 + u * step;
      if (i >= passes.all) break;
      const bool isk = i >= passes.of_q;
      const int h = (isk ? i - passes.of_q : i) * HW + sub;
      float a[8], b[8];
      xa[u].get(a);
      xb[u].get(b);
      if (p.qk_norm) {
        if (weights != isk) {
          weights = isk;
          const float* w = isk ? p.wk : p.wq;
          weights8(w ? w + 8 * j : nullptr, wa);
          weights8(w ? w + D / 2 + 8 * j : nullptr, wb);
        }
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += a[e] * a[e] + b[e] * b[e];
        const float r = 1.0f / sqrtf(head_sum<D>(ss) / static_cast<float>(D) + p.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          a[e] *= r * wa[e];
          b[e] *= r * wb[e];
        }
      }
      if (h < (isk ? p.hkv : p.hq)) {
        float ya[8], yb[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ya[e] = a[e] * c[e] - b[e] * s[e];
          yb[e] = b[e] * c[e] + a[e] * s[e];
        }
        T* y = (isk ? ko : qo) + static_cast<int64_t>(h) * D;
        store8(y, ya);
        store8(y + D / 2, yb);
      }
    }
  }
}

// Gradients: the warps stride over the rows (or, for few rows, over their passes) and keep
// their lanes' share of both norm-weight gradients in registers over all of them; the next
// pass is loaded before the current one is worked on.  The block adds its warps' shares in
// warp order, k_qk_rope_bwd_final the blocks' in block order, so reruns are bit-identical.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kRopeWarps, 2) k_qk_rope_bwd(const QkRopeParams p,
                                                                    const __grid_constant__ RopeTable tab) {
  constexpr int LH = RopePasses<D>::kLanes, HW = RopePasses<D>::kHeads;
  __shared__ float2 s_cs[kRopeWarps][D / 2];
  __shared__ float s_dw[kRopeWarps][2 * D];
  __shared__ __align__(16) float s_w[2][D];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane % LH, sub = lane / LH;
  const RopePasses<D> passes(p.hq, p.hkv);
  for (int i = threadIdx.x; i < 2 * D; i += 32 * kRopeWarps) {
    const float* w = i < D ? p.wq : p.wk;
    s_w[i / D][i % D] = w && p.qk_norm ? w[i % D] : 1.0f;
  }
  __syncthreads();
  float dwa[2][8] = {}, dwb[2][8] = {};  // [q, k][dimension]
  const int each = p.split == 1 ? passes.all : 1;  // passes of an item
  const int64_t items = p.m * p.split, stride = static_cast<int64_t>(gridDim.x) * kRopeWarps;
  Raw8<T> xa, xb;
  Raw8<float> ya, yb;
  // pass i of a row: its place, and its loads
  auto load = [&](int64_t row, int i) {
    const bool isk = i >= passes.of_q;
    const int h = (isk ? i - passes.of_q : i) * HW + sub, heads = isk ? p.hkv : p.hq;
    xa.zero(), xb.zero(), ya.zero(), yb.zero();
    if (h < heads) {
      const float* dy = (isk ? p.dk : p.dq) + (row * heads + h) * D + 8 * j;
      ya.load(dy);
      yb.load(dy + D / 2);
      if (p.qk_norm) {
        const T* x = (isk ? static_cast<const T*>(p.k) + row * p.ldk : static_cast<const T*>(p.q) + row * p.ldq) +
                     static_cast<int64_t>(h) * D + 8 * j;
        xa.load(x);
        xb.load(x + D / 2);
      }
    }
  };
  int64_t item = static_cast<int64_t>(blockIdx.x) * kRopeWarps + warp;
  if (item < items) load(item / p.split, static_cast<int>(item % p.split));
  for (; item < items; item += stride) {
    const int64_t row = item / p.split;
    const int first = static_cast<int>(item - row * p.split);
    __syncwarp();
    rope_table<D>(s_cs[warp], p.pos[row], tab);
    __syncwarp();
    for (int i = first; i < first + each; ++i) {
      const bool isk = i >= passes.of_q;
      const int h = (isk ? i - passes.of_q : i) * HW + sub;
      const Raw8<T> cxa = xa, cxb = xb;
      const Raw8<float> cya = ya, cyb = yb;
      if (i + 1 < first + each) load(row, i + 1);
      else if (item + stride < items) load((item + stride) / p.split, static_cast<int>((item + stride) % p.split));
      float a[8], b[8], ga[8], gb[8];
      cya.get(a);
      cyb.get(b);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 cs = s_cs[warp][8 * j + e];
        ga[e] = a[e] * cs.x + b[e] * cs.y;
        gb[e] = b[e] * cs.x - a[e] * cs.y;
      }
      if (p.qk_norm) {
        cxa.get(a);
        cxb.get(b);
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += a[e] * a[e] + b[e] * b[e];
        const float r = 1.0f / sqrtf(head_sum<D>(ss) / static_cast<float>(D) + p.eps);
        float wa[8], wb[8], dot = 0.0f;
        load8(&s_w[isk][8 * j], wa);
        load8(&s_w[isk][D / 2 + 8 * j], wb);
        auto take = [&](float (&da)[8], float (&db)[8]) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            da[e] += ga[e] * a[e] * r;
            db[e] += gb[e] * b[e] * r;
          }
        };
        if (isk) take(dwa[1], dwb[1]);  // warp-uniform
        else take(dwa[0], dwb[0]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ga[e] *= wa[e];
          gb[e] *= wb[e];
          dot += ga[e] * a[e] + gb[e] * b[e];
        }
        const float t = head_sum<D>(dot) / static_cast<float>(D) * r * r;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ga[e] = r * (ga[e] - a[e] * t);
          gb[e] = r * (gb[e] - b[e] * t);
        }
      }
      if (h < (isk ? p.hkv : p.hq)) {
        T* dx = (isk ? static_cast<T*>(p.k_out) + row * p.ldko : static_cast<T*>(p.q_out) + row * p.ldqo) +
                static_cast<int64_t>(h) * D + 8 * j;
        store8(dx, ga);
        store8(dx + D / 2, gb);
      }
    }
  }
  if (!p.part) return;
  // the warp's heads, then the block's warps
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float a = dwa[t][e], b = dwb[t][e];
#pragma unroll
      for (int o = LH; o < 32; o <<= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
      }
      if (sub == 0) {
        s_dw[warp][t * D + 8 * j + e] = a;
        s_dw[warp][t * D + D / 2 + 8 * j + e] = b;
      }
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += 32 * kRopeWarps) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kRopeWarps; ++w) v += s_dw[w][i];
    p.part[static_cast<int64_t>(blockIdx.x) * 2 * D + i] = v;
  }
}

// dw_q, dw_k [D] from the blocks' partials; one block of 4 * D threads per tensor:
// thread (c, d) adds the blocks b = c mod 4 in order, then the four sums are added.
__global__ void __launch_bounds__(512) k_qk_rope_bwd_final(const float* part, int blocks, int d, float* dwq, float* dwk) {
  __shared__ float s_sum[512];
  pdl_wait();
  pdl_launch_dependents();
  float* out = blockIdx.x ? dwk : dwq;
  const int c = threadIdx.x / d, i = threadIdx.x % d;
  float v = 0.0f;
  for (int b = c; b < blocks; b += 4) v += part[(static_cast<int64_t>(b) * 2 + blockIdx.x) * d + i];
  s_sum[threadIdx.x] = v;
  __syncthreads();
  if (c == 0 && out) out[i] = (s_sum[i] + s_sum[d + i]) + (s_sum[2 * d + i] + s_sum[3 * d + i]);
}

}  // namespace tg

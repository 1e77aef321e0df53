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
  int split;         // forward: warps that share one row
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

template <typename T, int D>
__global__ void __launch_bounds__(32 * kRopeWarps) k_qk_rope_fwd(const QkRopeParams p,
                                                                  const __grid_constant__ RopeTable tab) {
  __shared__ float2 s_cs[kRopeWarps][D / 2];
  pdl_wait();
  pdl_launch_dependents();
  constexpr int LH = D / 16, HW = 32 / LH;  // lanes per head, heads per warp pass
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane % LH, sub = lane / LH;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kRopeWarps + warp;
  const int64_t row = item / p.split;
  if (row >= p.m) return;  // warp-uniform
  rope_table<D>(s_cs[warp], p.pos[row], tab);
  __syncwarp();
  float c[8], s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float2 v = s_cs[warp][8 * j + e];
    c[e] = v.x;
    s[e] = v.y;
  }
  const int heads = p.hq + p.hkv;
  const T* q = static_cast<const T*>(p.q) + row * p.ldq;
  const T* k = static_cast<const T*>(p.k) + row * p.ldk;
  T* qo = static_cast<T*>(p.q_out) + row * p.ldqo;
  T* ko = static_cast<T*>(p.k_out) + row * p.ldko;
  for (int h0 = static_cast<int>(item - row * p.split) * HW; h0 < heads; h0 += p.split * HW) {
    const int h = h0 + sub;
    const bool in = h < heads, isq = h < p.hq;
    float a[8] = {}, b[8] = {};
    if (in) {
      const T* x = isq ? q + static_cast<int64_t>(h) * D : k + static_cast<int64_t>(h - p.hq) * D;
      load8(x + 8 * j, a);
      load8(x + D / 2 + 8 * j, b);
    }
    if (p.qk_norm) {
      float ss = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += a[e] * a[e] + b[e] * b[e];
      const float r = 1.0f / sqrtf(head_sum<D>(ss) / static_cast<float>(D) + p.eps);
      const float* w = isq ? p.wq : p.wk;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        a[e] *= r * (w ? w[8 * j + e] : 1.0f);
        b[e] *= r * (w ? w[D / 2 + 8 * j + e] : 1.0f);
      }
    }
    if (in) {
      float ya[8], yb[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ya[e] = a[e] * c[e] - b[e] * s[e];
        yb[e] = b[e] * c[e] + a[e] * s[e];
      }
      T* y = isq ? qo + static_cast<int64_t>(h) * D : ko + static_cast<int64_t>(h - p.hq) * D;
      store8(y + 8 * j, ya);
      store8(y + D / 2 + 8 * j, yb);
    }
  }
}

// Gradients: a warp takes whole rows, block-strided, and keeps its lanes' share
// of both norm-weight gradients in registers over all of them; the block adds
// its warps' shares in warp order, k_qk_rope_bwd_final the blocks' in block
// order, so reruns are bit-identical.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kRopeWarps) k_qk_rope_bwd(const QkRopeParams p,
                                                                 const __grid_constant__ RopeTable tab) {
  __shared__ float2 s_cs[kRopeWarps][D / 2];
  __shared__ float s_dw[kRopeWarps][2 * D];
  pdl_wait();
  pdl_launch_dependents();
  constexpr int LH = D / 16, HW = 32 / LH;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane % LH, sub = lane / LH;
  const int heads = p.hq + p.hkv;
  float dwa[2][8] = {}, dwb[2][8] = {};  // [q, k][dimension]
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRopeWarps + warp; row < p.m;
       row += static_cast<int64_t>(gridDim.x) * kRopeWarps) {
    __syncwarp();
    rope_table<D>(s_cs[warp], p.pos[row], tab);
    __syncwarp();
    for (int h0 = 0; h0 < heads; h0 += HW) {
      const int h = h0 + sub;
      const bool in = h < heads, isq = h < p.hq;
      float xa[8] = {}, xb[8] = {}, ga[8] = {}, gb[8] = {};
      if (in) {
        const float* dy = isq ? p.dq + (row * p.hq + h) * D : p.dk + (row * p.hkv + (h - p.hq)) * D;
        float ya[8], yb[8];
        load8(dy + 8 * j, ya);
        load8(dy + D / 2 + 8 * j, yb);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 cs = s_cs[warp][8 * j + e];
          ga[e] = ya[e] * cs.x + yb[e] * cs.y;
          gb[e] = yb[e] * cs.x - ya[e] * cs.y;
        }
        if (p.qk_norm) {
          const T* x = isq ? static_cast<const T*>(p.q) + row * p.ldq + static_cast<int64_t>(h) * D
                           : static_cast<const T*>(p.k) + row * p.ldk + static_cast<int64_t>(h - p.hq) * D;
          load8(x + 8 * j, xa);
          load8(x + D / 2 + 8 * j, xb);
        }
      }
      if (p.qk_norm) {
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += xa[e] * xa[e] + xb[e] * xb[e];
        const float r = 1.0f / sqrtf(head_sum<D>(ss) / static_cast<float>(D) + p.eps);
        const float* w = isq ? p.wq : p.wk;
        float dot = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float na = ga[e] * xa[e] * r, nb = gb[e] * xb[e] * r;
          dwa[0][e] += isq ? na : 0.0f;
          dwb[0][e] += isq ? nb : 0.0f;
          dwa[1][e] += isq ? 0.0f : na;
          dwb[1][e] += isq ? 0.0f : nb;
          ga[e] *= w ? w[8 * j + e] : 1.0f;
          gb[e] *= w ? w[D / 2 + 8 * j + e] : 1.0f;
          dot += ga[e] * xa[e] + gb[e] * xb[e];
        }
        const float t = head_sum<D>(dot) / static_cast<float>(D) * r * r;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ga[e] = r * (ga[e] - xa[e] * t);
          gb[e] = r * (gb[e] - xb[e] * t);
        }
      }
      if (in) {
        T* dx = isq ? static_cast<T*>(p.q_out) + row * p.ldqo + static_cast<int64_t>(h) * D
                    : static_cast<T*>(p.k_out) + row * p.ldko + static_cast<int64_t>(h - p.hq) * D;
        store8(dx + 8 * j, ga);
        store8(dx + D / 2 + 8 * j, gb);
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

// Decode attention over the paged 4-bit KV cache: for each request the new
// token's query heads over its cached rows,
//     l_c = temp_h ratio_r sm_scale (q_h . k_c) + gain_h bias_c,  out_h = sum_c softmax_c(l) v_c,
// with k_c and v_c the values the 4-bit rows stand for.  A key whose bias is
// -infinity is left out altogether, whatever its row holds; a request without
// keys gets zeros (lse -infinity).
#pragma once

#include "common.cuh"
#include "kv4.cuh"

namespace tg {

constexpr int kKv4MaxGroup = 8;
constexpr int kKv4Chunk = 128;  // keys per pass of the block

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
};

// One block per (request, KV head): a thread per key for the logits, then a
// thread per dimension for P.V, 128 keys at a time.
template <typename T, int D>
__global__ void __launch_bounds__(128) k_kv4_decode_simple(const Kv4DecodeParams p) {
  __shared__ float s_q[kKv4MaxGroup][D];
  __shared__ float s_p[kKv4MaxGroup][kKv4Chunk];
  __shared__ int64_t s_row[kKv4Chunk];
  pdl_wait();
  pdl_launch_dependents();
  const int r = blockIdx.x / p.c.hkv, kvh = blockIdx.x % p.c.hkv, h0 = kvh * p.group, tid = threadIdx.x;
  const T* q = static_cast<const T*>(p.q) + r * p.ldq + static_cast<int64_t>(h0) * D;
  for (int i = tid; i < p.group * D; i += 128) s_q[i / D][i % D] = to_f32(q[i]);
  int len = p.lens[r];
  if (len < 0 || len > static_cast<int64_t>(p.max_pages) * p.c.page_rows) {
    if (tid == 0) raise_error(kErrKvPage, 1);
    len = 0;
  }
  float mrun[kKv4MaxGroup], lrun[kKv4MaxGroup], o[kKv4MaxGroup];
  for (int u = 0; u < kKv4MaxGroup; ++u) mrun[u] = -INFINITY, lrun[u] = o[u] = 0.0f;
  const float ratio = p.ratio ? p.ratio[r] : 1.0f;
  for (int c0 = 0; c0 < len; c0 += kKv4Chunk) {
    __syncthreads();
    const int key = c0 + tid;
    int64_t row = -1;
    float bias = 0.0f;
    if (key < len) {
      const int32_t page = p.tables[static_cast<int64_t>(r) * p.max_pages + (key >> p.c.page_shift)];
      if (page < 0 || page >= p.c.num_pages) raise_error(kErrKvPage, 2);
      else {
        const int32_t slot = (page << p.c.page_shift) + (key & (p.c.page_rows - 1));
        row = kv4_row(p.c, slot, kvh);
        if (p.c.bias) bias = p.c.bias[slot];
        if (bias == -INFINITY) row = -1;
      }
    }
    s_row[tid] = row;
    float x[kKv4MaxGroup];
    for (int u = 0; u < kKv4MaxGroup; ++u) x[u] = 0.0f;
    if (row >= 0) {
      for (int g = 0; g < D / 32; ++g) {
        const float s = __bfloat162float(p.c.k_scales[row * (D / 32) + g]);
        float part[kKv4MaxGroup];
        for (int u = 0; u < kKv4MaxGroup; ++u) part[u] = 0.0f;
        for (int rr = 0; rr < 8; ++rr) {
          const uint32_t w = *reinterpret_cast<const uint32_t*>(p.c.k_codes + row * (D / 2) +
                                                                kv4_word<D>(rr, g >> 1, static_cast<int32_t>(row))) >>
                             (16 * (g & 1));
          for (int e = 0; e < 4; ++e) {
            const float kv = e2m1_value(w >> (4 * e) & 15u);
            for (int u = 0; u < p.group; ++u) part[u] += kv * s_q[u][32 * g + 4 * rr + e];
          }
        }
        for (int u = 0; u < p.group; ++u) x[u] += s * part[u];
      }
    }
    for (int u = 0; u < p.group; ++u) {
      const float a = p.temp[h0 + u] * ratio * p.scale_log2;
      s_p[u][tid] = row >= 0 ? a * x[u] + p.gain[h0 + u] * bias * 1.4426950408889634f : -INFINITY;
    }
    __syncthreads();
    for (int u = 0; u < p.group; ++u) {
      float top = mrun[u];
      for (int i = 0; i < kKv4Chunk; ++i) top = fmaxf(top, s_p[u][i]);
      const float use = top == -INFINITY ? 0.0f : top;
      const float alpha = exp2f(mrun[u] - use);
      mrun[u] = top;
      lrun[u] *= alpha;
      o[u] *= alpha;
      for (int i = 0; i < kKv4Chunk; ++i) {
        const int64_t vr = s_row[i];
        if (vr < 0) continue;
        const float w = exp2f(s_p[u][i] - use);
        lrun[u] += w;
        if (tid < D) {
          const int g = tid / 32, rr = tid % 32 / 4, e = tid % 4;
          const uint32_t word = *reinterpret_cast<const uint32_t*>(
              p.c.v_codes + vr * (D / 2) + kv4_word<D>(rr, g >> 1, static_cast<int32_t>(vr)));
          o[u] += w * (e2m1_value(word >> (16 * (g & 1) + 4 * e) & 15u) * __bfloat162float(p.c.v_scales[vr * (D / 32) + g]));
        }
      }
    }
  }
  for (int u = 0; u < p.group; ++u) {
    if (tid < D)
      static_cast<T*>(p.out)[r * p.ldo + static_cast<int64_t>(h0 + u) * D + tid] =
          from_f32<T>(lrun[u] == 0.0f ? 0.0f : o[u] / lrun[u]);
    if (tid == 0 && p.lse)
      p.lse[static_cast<int64_t>(r) * p.hq + h0 + u] =
          lrun[u] == 0.0f ? -INFINITY : (mrun[u] + log2f(lrun[u])) * 0.6931471805599453f;
  }
}

}  // namespace tg

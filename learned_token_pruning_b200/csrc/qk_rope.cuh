// Per-head RMSNorm of q and k with the position rotation in the same pass, and
// its gradients.  With x a head row, r = 1 / sqrt(mean x^2 + eps), w the norm
// weight, R the rotate-half rotation by the angles pos * theta^(-2i/D):
//     y = R (x r w)
//     g = R^T dy,  dw = sum over rows and heads of g x r,
//     dx = r g w - x r^3 mean(g w x)
// The angle is formed in turns and reduced to half a turn in double (positions reach
// 2^31), sine and cosine of the remainder are taken in fp32; every other value and
// sum is fp32, rounded once on the way out.  Turns, because sincospif needs no
// reduction of its own: against sincosf of the remainder in radians the backward of
// 4160 rows (16 + 8 heads of 128, bf16) takes 25.4 us instead of 26.0 (fewer registers,
// nothing spilled), the forward of 8256 the same.
//
// A lane owns the dimension pairs (8j + i, D/2 + 8j + i), i < 8, of a head: two
// 16-byte loads in bf16, and the rotation needs no exchange between lanes.  D/16
// lanes hold a head, so a warp takes 4 (D = 128) or 8 heads of one row at a
// time; the row's cosines and sines are computed once per warp and shared by its
// heads through shared memory.
//
// Bound by memory in fp32 (8256 rows of 16 + 8 heads of 128: 37.5 us, 5.4 TB/s, 83 % of a copy's
// rate), nearly so in bf16 (21.1 us, 4.8 TB/s).  The backward of 2064 rows, bf16 with fp32
// gradients in, takes 16.3 us (3.1 TB/s), 4160 rows 25.4: some 340 instructions a pass at 16 warps
// an SM, whose waits for shared memory and shuffles are the largest; its last 3.7 us
// are the weight gradients' second kernel.  Tried there: four pairs to a lane and half the
// registers of a pass, 18.8 us; a ring of asynchronous copies in shared memory, 19.3 (forward
// 22.5); the loop unrolled over two register sets, 22.8 (spills).
#pragma once

#include "attn_bwd_tc.cuh"
#include "attn_tc.cuh"
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
  int split, per;    // parts a row is cut into, passes of one
};

// A pass: the warp's 4 (D = 128) or 8 heads of q, or of k; a row is its passes of q, then of k.
template <int D>
struct RopePasses {
  static constexpr int kLanes = D / 16, kHeads = 32 / kLanes;  // lanes of a head, heads of a pass
  int of_q, all;
  __host__ __device__ RopePasses(int hq, int hkv)
      : of_q((hq + kHeads - 1) / kHeads), all(of_q + (hkv + kHeads - 1) / kHeads) {}
};

// Where value d of a half head sits in the tables in shared memory: the first four of each
// lane's eight, then the second four, so that a 16-byte read meets every bank once (forward
// of 8256 rows 21.9 -> 21.1 us, backward of 2064 16.7 -> 16.3).
template <int D>
__device__ __forceinline__ int rope_slot(int d) {
  return (d & 4) * (D / 16) + (d >> 3) * 4 + (d & 3);
}

// A lane's frequencies, read once: an index that differs by lane is served from constant
// memory one lane at a time.
template <int D>
struct RopeFreqs {
  double f[D / 64];
  __device__ __forceinline__ RopeFreqs(const RopeTable& tab) {
#pragma unroll
    for (int e = 0; e < D / 64; ++e) f[e] = tab.inv_freq[e * 32 + (threadIdx.x & 31)] * 0.15915494309189535;  // turns
  }
  // cos and sin of the row's D/2 angles into the warp's tables
  __device__ __forceinline__ void table(float* cosines, float* sines, int32_t pos) const {
#pragma unroll
    for (int e = 0; e < D / 64; ++e) {
      const double at = pos;
      float s, c;
      sincospif(2.0f * static_cast<float>(fma(at, f[e], -rint(at * f[e]))), &s, &c);
      cosines[rope_slot<D>(e * 32 + (threadIdx.x & 31))] = c;
      sines[rope_slot<D>(e * 32 + (threadIdx.x & 31))] = s;
    }
  }
};

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
};

// Eight fp32 values as four register pairs: a packed operation does two of them.
struct F8 {
  uint64_t v[4];
  __device__ __forceinline__ void get(const Raw8<__nv_bfloat16>& r) {
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f2_pack(bf16_lo(w[i]), bf16_hi(w[i]));
  }
  __device__ __forceinline__ void get(const Raw8<float>& r) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[2 * i] = f2_pack(__uint_as_float(r.w[i].x), __uint_as_float(r.w[i].y));
      v[2 * i + 1] = f2_pack(__uint_as_float(r.w[i].z), __uint_as_float(r.w[i].w));
    }
  }
  template <int D>
  __device__ __forceinline__ void from(const float* p) {  // lane j's eight of a table of half a head, at p + 4 j
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + D / 4);
    v[0] = f2_pack(a.x, a.y), v[1] = f2_pack(a.z, a.w), v[2] = f2_pack(b.x, b.y), v[3] = f2_pack(b.z, b.w);
  }
  template <typename T>
  __device__ __forceinline__ void put(T* p) const {
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) f2_unpack(v[i], x[2 * i], x[2 * i + 1]);
    store8(p, x);
  }
};
// sum of x y over the head's lanes, both halves
template <int D>
__device__ __forceinline__ float head_dot(const F8& xa, const F8& ya, const F8& xb, const F8& yb) {
  uint64_t s = f2_mul(xa.v[0], ya.v[0]), t = f2_mul(xb.v[0], yb.v[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    s = f2_fma(xa.v[i], ya.v[i], s);
    t = f2_fma(xb.v[i], yb.v[i], t);
  }
  float lo, hi;
  f2_unpack(f2_add(s, t), lo, hi);
  return head_sum<D>(lo + hi);
}

template <int D>
__device__ __forceinline__ void norm_weights(const QkRopeParams& p, float (*s_w)[D]) {
  for (int i = threadIdx.x; i < 2 * D; i += 32 * kRopeWarps) {
    const float* w = i < D ? p.wq : p.wk;
    const int at = i % D;
    s_w[i / D][at / (D / 2) * (D / 2) + rope_slot<D>(at % (D / 2))] = w && p.qk_norm ? w[at] : 1.0f;
  }
  __syncthreads();
}

// A warp's walk over its passes: its items (rows, or parts of them) stride through the launch;
// `step` passes are taken at a time.
struct RopeWalk {
  int64_t item, items, stride, row;
  int pass, end, split, per, all;
  __device__ __forceinline__ RopeWalk(const QkRopeParams& p, int all_)
      : item(static_cast<int64_t>(blockIdx.x) * kRopeWarps + (threadIdx.x >> 5)), items(p.m * p.split),
        stride(static_cast<int64_t>(gridDim.x) * kRopeWarps), split(p.split), per(p.per), all(all_) {
    place();
  }
  __device__ __forceinline__ void place() {
    if (split == 1) {
      row = item;
      pass = 0;
      end = all;
    } else {  // few items then: 32 bits
      row = static_cast<uint32_t>(item) / static_cast<uint32_t>(split);
      pass = static_cast<int>(item - row * split) * per;
      end = min(pass + per, all);
    }
  }
  __device__ __forceinline__ bool more() const { return item < items; }
  __device__ __forceinline__ void next(int step) {
    pass += step;
    if (pass >= end) {
      item += stride;
      place();
    }
  }
};

// The next passes' loads, and the next row's position, are on their way while these are worked on.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kRopeWarps, 2) k_qk_rope_fwd(const QkRopeParams p,
                                                                    const __grid_constant__ RopeTable tab) {
  constexpr int LH = RopePasses<D>::kLanes, HW = RopePasses<D>::kHeads, CH = sizeof(T) == 2 ? 2 : 1;
  __shared__ __align__(16) float s_c[kRopeWarps][D / 2], s_s[kRopeWarps][D / 2];
  __shared__ __align__(16) float s_w[2][D];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane % LH, sub = lane / LH;
  const RopePasses<D> passes(p.hq, p.hkv);
  const RopeFreqs<D> freqs(tab);
  norm_weights<D>(p, s_w);
  RopeWalk ahead(p, passes.all), here(p, passes.all);
  Raw8<T> xa[CH], xb[CH];
  int32_t pos = 0;
  auto load = [&]() {
    const T* q = static_cast<const T*>(p.q) + ahead.row * p.ldq + sub * D + 8 * j;
    const T* k = static_cast<const T*>(p.k) + ahead.row * p.ldk + sub * D + 8 * j;
#pragma unroll
    for (int u = 0; u < CH; ++u) {
      const int i = ahead.pass + u;
      const bool isk = i >= passes.of_q;
      const int h0 = (isk ? i - passes.of_q : i) * HW;
      if (i < ahead.end && h0 + sub < (isk ? p.hkv : p.hq)) {
        const T* x = (isk ? k : q) + h0 * D;
        xa[u].load(x);
        xb[u].load(x + D / 2);
      }
    }
    pos = p.pos[ahead.row];
  };
#pragma unroll
  for (int u = 0; u < CH; ++u) xa[u].zero(), xb[u].zero();
  if (ahead.more()) load();
  F8 c, s, ns;
  int64_t angles_of = -1;
  while (here.more()) {
    Raw8<T> ca[CH], cb[CH];
#pragma unroll
    for (int u = 0; u < CH; ++u) ca[u] = xa[u], cb[u] = xb[u];
    if (angles_of != here.row) {
      angles_of = here.row;
      __syncwarp();
      freqs.table(s_c[warp], s_s[warp], pos);
      __syncwarp();
      c.template from<D>(&s_c[warp][4 * j]);
      s.template from<D>(&s_s[warp][4 * j]);
#pragma unroll
      for (int e = 0; e < 4; ++e) ns.v[e] = s.v[e] ^ 0x8000000080000000ull;
    }
    ahead.next(CH);
    if (ahead.more()) load();
#pragma unroll
    for (int u = 0; u < CH; ++u) {
      const int i = here.pass + u;
      if (i >= here.end) break;
      const bool isk = i >= passes.of_q;
      const int h = (isk ? i - passes.of_q : i) * HW + sub;
      F8 a, b, wa, wb;
      a.get(ca[u]);
      b.get(cb[u]);
      if (p.qk_norm) {
        const float n = rsqrtf(head_dot<D>(a, a, b, b) * (1.0f / D) + p.eps);  // 2 ulp
        const uint64_t n2 = f2_pack(n, n);
        wa.template from<D>(&s_w[isk][4 * j]);
        wb.template from<D>(&s_w[isk][D / 2 + 4 * j]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          a.v[e] = f2_mul(a.v[e], f2_mul(wa.v[e], n2));
          b.v[e] = f2_mul(b.v[e], f2_mul(wb.v[e], n2));
        }
      }
      if (h < (isk ? p.hkv : p.hq)) {
        T* y = (isk ? static_cast<T*>(p.k_out) + here.row * p.ldko : static_cast<T*>(p.q_out) + here.row * p.ldqo) +
               h * D + 8 * j;
        F8 ya, yb;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          ya.v[e] = f2_fma(b.v[e], ns.v[e], f2_mul(a.v[e], c.v[e]));
          yb.v[e] = f2_fma(a.v[e], s.v[e], f2_mul(b.v[e], c.v[e]));
        }
        ya.put(y);
        yb.put(y + D / 2);
      }
    }
    here.next(CH);
  }
}

// Gradients.  The lanes' share of both norm-weight gradients stays in registers over all of a
// warp's passes; the block adds its warps' shares in warp order, k_qk_rope_bwd_final the
// blocks' in block order, so reruns are bit-identical.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kRopeWarps, 2) k_qk_rope_bwd(const QkRopeParams p,
                                                                    const __grid_constant__ RopeTable tab) {
  constexpr int LH = RopePasses<D>::kLanes, HW = RopePasses<D>::kHeads;
  __shared__ __align__(16) float s_c[kRopeWarps][D / 2], s_s[kRopeWarps][D / 2];
  __shared__ float s_dw[kRopeWarps][2 * D];
  __shared__ __align__(16) float s_w[2][D];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane % LH, sub = lane / LH;
  const RopePasses<D> passes(p.hq, p.hkv);
  const RopeFreqs<D> freqs(tab);
  norm_weights<D>(p, s_w);
  RopeWalk ahead(p, passes.all), here(p, passes.all);
  F8 dwa[2], dwb[2];  // [q, k]
#pragma unroll
  for (int e = 0; e < 4; ++e) dwa[0].v[e] = dwa[1].v[e] = dwb[0].v[e] = dwb[1].v[e] = 0;
  Raw8<T> xa, xb;
  Raw8<float> ya, yb;
  int32_t pos = 0;
  auto load = [&]() {  // heads past the last are loaded as zeros: they add nothing to the sums
    const bool isk = ahead.pass >= passes.of_q;
    const int h = (isk ? ahead.pass - passes.of_q : ahead.pass) * HW + sub, heads = isk ? p.hkv : p.hq;
    xa.zero(), xb.zero(), ya.zero(), yb.zero();
    if (h < heads) {
      const float* dy = (isk ? p.dk : p.dq) + (ahead.row * heads + h) * D + 8 * j;
      ya.load(dy);
      yb.load(dy + D / 2);
      if (p.qk_norm) {
        const T* x = (isk ? static_cast<const T*>(p.k) + ahead.row * p.ldk : static_cast<const T*>(p.q) + ahead.row * p.ldq) +
                     h * D + 8 * j;
        xa.load(x);
        xb.load(x + D / 2);
      }
    }
    pos = p.pos[ahead.row];
  };
  if (ahead.more()) load();
  int64_t angles_of = -1;
  while (here.more()) {
    const Raw8<T> cxa = xa, cxb = xb;
    const Raw8<float> cya = ya, cyb = yb;
    if (angles_of != here.row) {
      angles_of = here.row;
      __syncwarp();
      freqs.table(s_c[warp], s_s[warp], pos);
      __syncwarp();
    }
    ahead.next(1);
    if (ahead.more()) load();
    const bool isk = here.pass >= passes.of_q;
    const int h = (isk ? here.pass - passes.of_q : here.pass) * HW + sub;
    F8 a, b, ga, gb, c, s;
    a.get(cya);
    b.get(cyb);
    c.template from<D>(&s_c[warp][4 * j]);
    s.template from<D>(&s_s[warp][4 * j]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      ga.v[e] = f2_fma(b.v[e], s.v[e], f2_mul(a.v[e], c.v[e]));
      gb.v[e] = f2_fma(a.v[e], s.v[e] ^ 0x8000000080000000ull, f2_mul(b.v[e], c.v[e]));
    }
    if (p.qk_norm) {
      a.get(cxa);
      b.get(cxb);
      const float n = rsqrtf(head_dot<D>(a, a, b, b) * (1.0f / D) + p.eps);  // 2 ulp
      const uint64_t n2 = f2_pack(n, n);
      auto take = [&](F8& da, F8& db) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          da.v[e] = f2_fma(f2_mul(ga.v[e], n2), a.v[e], da.v[e]);
          db.v[e] = f2_fma(f2_mul(gb.v[e], n2), b.v[e], db.v[e]);
        }
      };
      if (isk) take(dwa[1], dwb[1]);  // warp-uniform
      else take(dwa[0], dwb[0]);
      c.template from<D>(&s_w[isk][4 * j]);
      s.template from<D>(&s_w[isk][D / 2 + 4 * j]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        ga.v[e] = f2_mul(ga.v[e], c.v[e]);
        gb.v[e] = f2_mul(gb.v[e], s.v[e]);
      }
      const float t = -head_dot<D>(ga, a, gb, b) * (1.0f / D) * n * n;
      const uint64_t t2 = f2_pack(t, t);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        ga.v[e] = f2_mul(n2, f2_fma(a.v[e], t2, ga.v[e]));
        gb.v[e] = f2_mul(n2, f2_fma(b.v[e], t2, gb.v[e]));
      }
    }
    if (h < (isk ? p.hkv : p.hq)) {
      T* dx = (isk ? static_cast<T*>(p.k_out) + here.row * p.ldko : static_cast<T*>(p.q_out) + here.row * p.ldqo) +
              h * D + 8 * j;
      ga.put(dx);
      gb.put(dx + D / 2);
    }
    here.next(1);
  }
  if (!p.part) return;
  // the warp's heads, then the block's warps
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float v[4];
      f2_unpack(dwa[t].v[e], v[0], v[1]);
      f2_unpack(dwb[t].v[e], v[2], v[3]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int o = LH; o < 32; o <<= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        if (sub == 0) s_dw[warp][t * D + (i >> 1) * (D / 2) + 8 * j + 2 * e + (i & 1)] = v[i];
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

// dw_q, dw_k [D] from the blocks' partials: a block takes 32 dimensions of one of them, warp w
// adds the blocks b = w mod 32 in order, and the 32 sums are added in order.
__global__ void __launch_bounds__(1024) k_qk_rope_bwd_final(const float* part, int blocks, int d, float* dwq,
                                                            float* dwk) {
  __shared__ float s_sum[32][33];
  pdl_wait();
  pdl_launch_dependents();
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, i = blockIdx.y * 32 + lane;
  float* out = blockIdx.x ? dwk : dwq;
  const float* p = part + static_cast<int64_t>(blockIdx.x) * d + i;
  float v = 0.0f;
#pragma unroll 10
  for (int b = w; b < blocks; b += 32) v += p[static_cast<int64_t>(b) * 2 * d];
  s_sum[w][lane] = v;
  __syncthreads();
  if (w == 0 && out) {
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < 32; ++k) t += s_sum[k][lane];
    out[i] = t;
  }
}

}  // namespace tg

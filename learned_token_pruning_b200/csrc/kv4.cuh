// The paged 4-bit KV cache: page tables and slot maps built on the device, and
// rows moved in and out of the cache.
//
// A cache row of one KV head is D E2M1 codes (sign, 2 exponent bits, 1 mantissa
// bit: the values 0, .5, 1, 1.5, 2, 3, 4, 6) and one bf16 scale per 32
// dimensions: 4.5 bits a value.  Layout of a page (kv4 cache in tg.h):
//   codes  [page][head][row][D / 2] bytes,  scales [page][head][row][D / 32] bf16
// so that one head's rows of a page are one contiguous block, which a bulk copy
// takes as it is.  Inside a row the 16-bit unit of dimensions 32g + 4r .. + 3
// (low nibble first) sits at unit r * (D / 32) + g: the four units a decode lane
// needs, one per scale group, are neighbours.  At D = 128 a row is 64 bytes, and
// rows 2 and 3 of every four hold their 32-byte halves swapped, so that a warp
// reading 8 bytes of each of four neighbouring rows meets every bank once.
#pragma once

#include "attn_bwd_tc.cuh"
#include "attn_tc.cuh"
#include "common.cuh"

namespace tg {

// consistency checks of the paged cache (device error word, see common.cuh)
constexpr uint32_t kErrPageTable = 4;  // lengths, new rows, tables or the free list do not fit
constexpr uint32_t kErrKvSlot = 5;     // slot past the cache
constexpr uint32_t kErrKvPage = 6;     // page id or request length out of range

struct Kv4Cache {
  uint8_t* k_codes;
  uint8_t* v_codes;
  __nv_bfloat16* k_scales;
  __nv_bfloat16* v_scales;
  float* bias;        // [num_pages][page_rows] or null
  int64_t num_pages;
  int32_t page_rows;  // 16, 32, 64 or 128
  int32_t page_shift;
  int32_t hkv;
};

// index of the (page, head, row) triple of a slot
__device__ __forceinline__ int64_t kv4_row(const Kv4Cache& c, int32_t slot, int head) {
  const int64_t page = slot >> c.page_shift;
  return ((page * c.hkv + head) << c.page_shift) + (slot & (c.page_rows - 1));
}

// ---------------------------------------------------------------------------
// Page tables.  One cluster of CTAs: each scans all requests by itself (three
// prefix sums in shared memory: returned pages, taken pages, new rows) and then
// takes its share of the page moves and of the slots.  The cluster barriers
// order the reads of the old state before the writes of the new one, so the
// state may be updated in place.  Bound by latency: the two barriers and the
// dependent loads (length -> page -> slot).  Device time: one more row for 56 of 64
// requests 6.5 us, 129828 rows for 1000 requests (pages of 16, 0.6 MB) 12.4 us.
// ---------------------------------------------------------------------------
constexpr int kTabThreads = 512;
constexpr int kTabMaxReq = 4096;
constexpr int kTabTimes = 8;
constexpr int kTabPer = kTabMaxReq / kTabThreads;  // requests per thread at most

struct PageTableParams {
  const int32_t* lens;
  const int32_t* new_rows;
  const uint8_t* release;  // or null
  int32_t nreq;
  int32_t page_rows;
  uint32_t last_page;  // the last one with a slot of 31 bits
  int32_t* tables;
  int32_t max_pages;
  int32_t* free_pages;
  int32_t free_cap;
  const int32_t* n_free;
  int32_t* lens_out;
  int32_t* n_free_out;
  int32_t* slots;
  int32_t nslots;
  int32_t* row_start;  // null only where slots are by request
  bool by_request;     // one new row at most: slots[r] is request r's
};

__host__ __device__ constexpr size_t page_table_smem(int nreq) { return static_cast<size_t>(4 * nreq + 3) * 4; }

// largest r with start[r] <= i (start ascending, start[0] = 0, i < start[n]); the
// requests without items have start[r] == start[r + 1] and are never returned
__device__ __forceinline__ int find_request(const int32_t* start, int n, int32_t i) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= i) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The slot of row `row` of a page, -1 for a bad page id (reported) and for none (both -1).  Any ids
// and page sizes: up to the last page the product fits 32 bits, and past 2^31 - 1 it is negative.
__device__ __forceinline__ int32_t page_slot(const PageTableParams& p, int32_t id, int32_t row) {
  int32_t slot = static_cast<int32_t>(static_cast<uint32_t>(id) * p.page_rows + row);
  if (static_cast<uint32_t>(id) > p.last_page || slot < 0) {
    slot = -1;
    if (row >= 0) raise_error(kErrPageTable, 4);
  }
  return slot;
}

__device__ __forceinline__ void block_scan3(int64_t (&v)[3], int64_t (*s_warp)[3], int64_t (&before)[3],
                                            int64_t (&total)[3]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t inc[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    inc[k] = v[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, inc[k], o);
      if (lane >= o) inc[k] += up;
    }
    if (lane == 31) s_warp[warp][k] = inc[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    int64_t base = 0, all = 0;
    for (int w = 0; w < kTabThreads / 32; ++w) {
      if (w < warp) base += s_warp[w][k];
      all += s_warp[w][k];
    }
    before[k] = base + inc[k] - v[k];
    total[k] = all;
  }
}

__global__ void __launch_bounds__(kTabThreads) k_page_tables(const PageTableParams p) {
  extern __shared__ int32_t s_tab[];
  __shared__ int64_t s_warp[kTabThreads / 32][3];
  __shared__ int s_bad;
  int32_t* s_len = s_tab;                   // [nreq] rows held before this call's new ones
  int32_t* s_back = s_len + p.nreq;         // [nreq + 1] first returned page
  int32_t* s_take = s_back + p.nreq + 1;    // [nreq + 1] first taken page
  int32_t* s_rows = s_take + p.nreq + 1;    // [nreq + 1] first new row
  const int rank = static_cast<int>(cluster_ctarank()), size = static_cast<int>(gridDim.x);
  if (threadIdx.x == 0) s_bad = 0;
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();
  const int64_t P = p.page_rows, most = static_cast<int64_t>(p.max_pages) * P;
  const int per = (p.nreq + kTabThreads - 1) / kTabThreads;
  const int r0 = threadIdx.x * per;
  int32_t len[kTabPer], add[kTabPer], back[kTabPer], take[kTabPer];
  int64_t v[3] = {0, 0, 0};
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kTabPer; ++i) {
    len[i] = add[i] = back[i] = take[i] = 0;
    const int r = r0 + i;
    if (i < per && r < p.nreq) {
      int64_t l = p.lens[r];
      const int64_t n = p.new_rows[r];
      if (l < 0 || l > most || n < 0 || (p.by_request && n > 1)) bad = true;
      else {
        if (p.release && p.release[r]) {
          back[i] = static_cast<int32_t>((l + P - 1) / P);
          l = 0;
        }
        if (l + n > most) bad = true;
        else {
          len[i] = static_cast<int32_t>(l);
          add[i] = static_cast<int32_t>(n);
          take[i] = static_cast<int32_t>((l + n + P - 1) / P - (l + P - 1) / P);
        }
      }
    }
    v[0] += back[i];
    v[1] += take[i];
    v[2] += add[i];
  }
  if (bad) s_bad = 1;  // same value from every writer
  int64_t before[3], total[3];
  block_scan3(v, s_warp, before, total);  // its barrier also publishes s_bad
  const int64_t nf = *p.n_free;
  // one verdict from the same inputs in every CTA
  const bool refuse = s_bad || nf < 0 || nf + total[0] > p.free_cap || total[1] > nf + total[0] || total[2] > p.nslots;
#pragma unroll
  for (int i = 0; i < kTabPer; ++i) {
    const int r = r0 + i;
    if (i < per && r < p.nreq) {
      s_len[r] = len[i];
      s_back[r] = static_cast<int32_t>(before[0]);
      s_take[r] = static_cast<int32_t>(before[1]);
      s_rows[r] = static_cast<int32_t>(before[2]);
    }
    before[0] += back[i];
    before[1] += take[i];
    before[2] += add[i];
  }
  if (threadIdx.x == 0) {
    s_back[p.nreq] = static_cast<int32_t>(total[0]);
    s_take[p.nreq] = static_cast<int32_t>(total[1]);
    s_rows[p.nreq] = static_cast<int32_t>(total[2]);
  }
  __syncthreads();
  cluster_sync_all();  // every CTA has read the old lengths and free count
  const int t0 = rank * kTabThreads + threadIdx.x, step = size * kTabThreads;
  if (refuse) {
    if (t0 == 0) raise_error(kErrPageTable, s_bad ? 1u : (total[1] > nf + total[0] ? 2u : 3u));
    for (int i = t0; i < p.nslots; i += step) p.slots[i] = -1;
    for (int i = t0; p.row_start && i <= p.nreq; i += step) p.row_start[i] = 0;
    for (int i = t0; i < p.nreq && p.lens_out != p.lens; i += step) p.lens_out[i] = p.lens[i];
    if (t0 == 0) *p.n_free_out = static_cast<int32_t>(nf);
    return;
  }
  const int32_t nback = static_cast<int32_t>(total[0]), ntake = static_cast<int32_t>(total[1]);
  const int32_t nrows = static_cast<int32_t>(total[2]), top = static_cast<int32_t>(nf + total[0]);
  for (int i = t0; i < nback; i += step) {
    const int r = find_request(s_back, p.nreq, i);
    p.free_pages[nf + i] = p.tables[static_cast<int64_t>(r) * p.max_pages + (i - s_back[r])];
  }
  if (nback) cluster_sync_all();  // returned pages are listed before any page is taken
  for (int i = t0; i < ntake; i += step) {
    const int r = find_request(s_take, p.nreq, i);
    const int first = (s_len[r] + p.page_rows - 1) / p.page_rows;
    p.tables[static_cast<int64_t>(r) * p.max_pages + first + (i - s_take[r])] = __ldcg(p.free_pages + (top - 1 - i));
  }
  // the id of page `page` of request r: pages taken in this call are read off the free list
  // (another thread writes the table)
  auto page_id = [&](int r, int32_t page) {
    const int32_t held = (s_len[r] + p.page_rows - 1) / p.page_rows;
    return __ldcg(page < held ? p.tables + static_cast<int64_t>(r) * p.max_pages + page
                              : p.free_pages + (top - 1 - (s_take[r] + page - held)));
  };
  // A warp takes 32 neighbouring slots up to eight times in a row, as often as it takes to go
  // round once: one search for the first row's request, then short walks, and the page ids a
  // lane needs on their way together.  129828 slots of 1000 requests, 16 CTAs: eight times
  // 12.4 us, twice 15.5; one slot for each of 1000 requests, where a walk passes as many
  // requests as slots: 15.1 and 9.0.
  const int lane = threadIdx.x & 31;
  const int times = max(1, min(kTabTimes, (p.nslots + step - 1) / step));
  for (int r = t0; p.by_request && r < p.nreq; r += step) {
    const int32_t page = s_len[r] / p.page_rows;
    p.slots[r] = s_rows[r + 1] == s_rows[r] ? -1 : page_slot(p, page_id(r, page), s_len[r] - page * p.page_rows);
  }
  for (int c = t0 >> 5; !p.by_request && static_cast<int64_t>(c) * times * 32 < p.nslots; c += step >> 5) {
    const int i0 = c * times * 32 + lane;
    int r = i0 < nrows ? find_request(s_rows, p.nreq, i0) : 0;
    int32_t id[kTabTimes], off[kTabTimes];
#pragma unroll
    for (int k = 0; k < kTabTimes; ++k) {
      const int i = i0 + 32 * k;
      id[k] = -1;
      off[k] = -1;
      if (k < times && i < nrows) {
        while (s_rows[r + 1] <= i) ++r;
        const int32_t at = s_len[r] + (i - s_rows[r]);
        const int32_t page = at / p.page_rows;
        off[k] = at - page * p.page_rows;
        id[k] = page_id(r, page);
      }
    }
#pragma unroll
    for (int k = 0; k < kTabTimes; ++k) {
      const int i = i0 + 32 * k;
      const int32_t slot = page_slot(p, id[k], off[k]);
      if (k < times && i < p.nslots) p.slots[i] = slot;
    }
  }
  for (int i = t0; i <= p.nreq; i += step) {
    if (p.row_start) p.row_start[i] = s_rows[i];
    if (i < p.nreq) p.lens_out[i] = s_len[i] + (s_rows[i + 1] - s_rows[i]);
  }
  if (t0 == 0) *p.n_free_out = top - ntake;
}

// ---------------------------------------------------------------------------
// Rows in and out.  Four lanes share a group of 32 dimensions, eight dimensions
// (one 16-byte load in bf16) each.  8256 rows of 8 heads of 128, K and V, pages of 64: in 14.0 us
// (bf16, 43 MB, 3.1 TB/s, 47 % of a copy's rate; fp32, 77 MB, 17.5 us, 67 %), out 13.4 (bf16)
// and 17.4 (fp32); bf16 in and then fp32 out 30.1 us (121 MB, 61 %).  Bound by the instructions: 10.1 M
// warp instructions in (bf16) and 11.9 M out (fp32), issued in 70 and 74 % of the
// cycles, the logic pipe 64 % busy with both.  A decode step's rows are bound by the launch.
// ---------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(ww[i]);
    x[2 * i + 1] = bf16_hi(ww[i]);
  }
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]);
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                            pack_bf16x2(x[6], x[7]));
}
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&x)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// Nearest E2M1 code of x / s for s > 0, ties to the even code, by comparing |x|
// with the seven borders times s.  A border has at most 3 significant bits and s
// is bf16, so the products are exact and the code is the exact nearest one.
__device__ __forceinline__ uint32_t e2m1_code(float x, float s) {
  const float a = fabsf(x);
  uint32_t c = 0;
  c += a > 0.25f * s;
  c += a >= 0.75f * s;
  c += a > 1.25f * s;
  c += a >= 1.75f * s;
  c += a > 2.5f * s;
  c += a >= 3.5f * s;
  c += a > 5.0f * s;
  return c | (__float_as_uint(x) >> 28 & 8u);
}

// Eight E2M1 codes, nearest with ties to the even code, +-6 at most; x[0] in the low nibble.
__device__ __forceinline__ uint32_t e2m1_round8(const float (&x)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 c0, c1, c2, c3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 c1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 c3, %8, %7;\n\t"
      "mov.b32 %0, {c0, c1, c2, c3};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

// Eight codes of x / s, exactly the nearest ones; s > 0.
//   bf16: x times the approximate 1 / s (1 ulp) is off by less than 2^-22 of itself, and a
//   quotient of two bf16 numbers that is not a border between codes is 2^-11 of itself away
//   from one (a border has 3 significant bits), so rounding the product to 15 bits puts
//   quotients on a border exactly there and no other on the wrong side of one.
//   fp32: the product is taken once a little below and once a little above; where the
//   codes differ, a border lies between, and the comparisons decide.
// Scales below 2^-100, whose reciprocals may not be floats, take the comparisons too.
template <typename T>
__device__ __forceinline__ uint32_t e2m1_codes8(const float (&x)[8], float s) {
  float r, y[8], z[8];
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  uint32_t w, other;
  if constexpr (sizeof(T) == 2) {
    // y rounded to 15 bits as c - (c - y), c = (2^9 + 1) y: on the multiply-add pipe, in pairs
    const uint64_t r2 = f2_pack(r, r), big = f2_pack(513.0f, 513.0f), minus = f2_pack(-1.0f, -1.0f);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint64_t v = f2_mul(f2_pack(x[2 * e], x[2 * e + 1]), r2), c = f2_mul(v, big);
      f2_unpack(f2_fma(f2_fma(v, minus, c), minus, c), y[2 * e], y[2 * e + 1]);
    }
    w = other = e2m1_round8(y);
  } else {
    const float below = r * (1.0f - 9.5367431640625e-7f), above = r * (1.0f + 9.5367431640625e-7f);  // 2^-20
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = x[e] * below, z[e] = x[e] * above;
    w = e2m1_round8(y);
    other = e2m1_round8(z);
  }
  if (w != other || s < 7.888609052210118e-31f) {  // 2^-100
    w = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) w |= e2m1_code(x[e], s) << (4 * e);
  }
  return w;
}

// the values of the two codes in byte b of w
template <int B>
__device__ __forceinline__ float2 e2m1_values(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b0;\n\t}" : "=r"(h) : "r"(w >> (8 * B)));
  float2 f;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}" : "=f"(f.x), "=f"(f.y) : "r"(h));
  return f;
}

struct Kv4RowsParams {
  Kv4Cache c;
  const void* k;   // rows in (store) or out (load)
  const void* v;
  int64_t ldk, ldv;
  float* bias;     // row biases in (store) or out (load), or null
  const int32_t* slots;
  int64_t rows;
};

// byte offset in a row of the 32-bit word that holds units (r, 2gp) and (r, 2gp + 1)
template <int D>
__device__ __forceinline__ int kv4_word(int r, int gp, int32_t slot) {
  const int at = (r * (D / 64) + gp) * 4;
  return D == 128 ? at ^ ((slot & 2) << 4) : at;
}

// A thread takes the same eight values of K or V of one head (`li` of a row's) in IT rows: rows are
// dealt to the blocks IT * per_block at a time, blockIdx.y counts 256 items of a row each.
struct Kv4Place {
  int li, head, l, g, l4;  // item of the row, head, eighth of the head, scale group, eighth of the group
  bool is_v, mine;
  int64_t row0;
  int step;  // rows between this thread's
  template <int D, int IT>
  __device__ __forceinline__ static Kv4Place at(const Kv4RowsParams& p) {
    Kv4Place t;
    const int per_row = 2 * p.c.hkv * (D / 8), chunk = min(per_row, 256);
    const int sub = threadIdx.x / chunk;
    t.step = 256 / chunk;
    t.li = threadIdx.x - sub * chunk + 256 * blockIdx.y;
    t.mine = sub < t.step && t.li < per_row;  // eight neighbouring lanes alike: chunk and per_row are multiples of 16
    t.row0 = static_cast<int64_t>(blockIdx.x) * IT * t.step + sub;
    const int head2 = t.li / (D / 8);
    t.l = t.li % (D / 8);
    t.is_v = head2 >= p.c.hkv;
    t.head = t.is_v ? head2 - p.c.hkv : head2;
    t.g = t.l >> 2;
    t.l4 = t.l & 3;
    return t;
  }
};

// The largest magnitude of a lane's eight values, as fp32 bits: infinities and NaN come out on top.
__device__ __forceinline__ uint32_t top8(const uint4 (&w)[1]) {
  const uint32_t m = 0x7fff7fffu;
  return __vmaxu2(__vmaxu2(w[0].x & m, w[0].y & m), __vmaxu2(w[0].z & m, w[0].w & m));  // a pair of bf16
}
__device__ __forceinline__ uint32_t top8(const uint4 (&w)[2]) {
  const uint32_t m = 0x7fffffffu;
  const uint32_t a = max(max(w[0].x & m, w[0].y & m), max(w[0].z & m, w[0].w & m));
  return max(a, max(max(w[1].x & m, w[1].y & m), max(w[1].z & m, w[1].w & m)));
}

template <typename T, int D, int IT>
__global__ void __launch_bounds__(256) k_kv4_store(const Kv4RowsParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const Kv4Place t = Kv4Place::at<D, IT>(p);
  const T* src = static_cast<const T*>(t.is_v ? p.v : p.k) + t.head * D + t.l * 8;
  const int64_t ld = t.is_v ? p.ldv : p.ldk;
  uint8_t* codes = t.is_v ? p.c.v_codes : p.c.k_codes;
  __nv_bfloat16* scales = (t.is_v ? p.c.v_scales : p.c.k_scales) + t.g;
  const int64_t slots = p.c.num_pages * p.c.page_rows;
  constexpr int kW = sizeof(T) / 2;
  int32_t slot[IT];
  uint4 raw[IT][kW];
#pragma unroll
  for (int u = 0; u < IT; ++u) {
    const int64_t row = t.row0 + u * t.step;
    slot[u] = -1;
#pragma unroll
    for (int i = 0; i < kW; ++i) raw[u][i] = make_uint4(0, 0, 0, 0);
    if (t.mine && row < p.rows) {
      slot[u] = p.slots[row];
#pragma unroll
      for (int i = 0; i < kW; ++i) raw[u][i] = reinterpret_cast<const uint4*>(src + row * ld)[i];
    }
  }
#pragma unroll
  for (int u = 0; u < IT; ++u) {
    if (slot[u] >= slots) {
      if (t.li == 0) raise_error(kErrKvSlot, 1);
      slot[u] = -1;
    }
    // max / 6 rounded to bf16 by way of fp32, which must meet no false tie.  The product with 1/6
    // (2^-25 off) is less than a step from the quotient.  For a bf16 maximum it is on a tie where
    // the quotient is and 2^-12 away elsewhere.  For an fp32 maximum the remainder's sign
    // says which side of it the quotient lies on: a product above it goes a step down, and the last
    // bit is set where there is a remainder, so that only an exact quotient is on a tie (below the
    // smallest normal number an fp32 quotient rounded to nearest can fall on one).
    uint32_t top = top8(raw[u]);
    float sixth;
    if constexpr (kW == 1) {
      top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
      top = max(top << 16, top & 0xffff0000u);
      sixth = __uint_as_float(top) * (1.0f / 6.0f);
    } else {
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float largest = __uint_as_float(top);
      sixth = largest * (1.0f / 6.0f);
      const float rest = fmaf(sixth, -6.0f, largest);
      sixth = __uint_as_float((__float_as_uint(sixth) - (rest < 0.0f)) | (rest != 0.0f));
    }
    const bool finite = top < 0x7f800000u;
    const __nv_bfloat16 sb = __float2bfloat16_rn(finite ? sixth : __uint_as_float(0x7fffffffu));
    const float s = __bfloat162float(sb);
    float x[8];
    load8(reinterpret_cast<const T*>(raw[u]), x);
    const uint32_t w = finite && s > 0.0f ? e2m1_codes8<T>(x, s) : 0u;  // dimension 8l first
    // low half: unit (2 l4, g); high half: (2 l4 + 1, g).  The lane of the neighbouring
    // group has the same units of group g ^ 1: each keeps one and hands over the other.
    const uint32_t got = __shfl_xor_sync(0xffffffffu, t.g & 1 ? w & 0xffffu : w >> 16, 4);
    const uint32_t word = t.g & 1 ? got | (w & 0xffff0000u) : (w & 0xffffu) | got << 16;
    if (slot[u] < 0) continue;
    const int64_t at = kv4_row(p.c, slot[u], t.head);
    *reinterpret_cast<uint32_t*>(codes + at * (D / 2) + kv4_word<D>(2 * t.l4 + (t.g & 1), t.g >> 1, slot[u])) = word;
    if (t.l4 == 0) scales[at * (D / 32)] = sb;
    if (t.li == 0 && p.c.bias) p.c.bias[slot[u]] = p.bias ? p.bias[t.row0 + u * t.step] : 0.0f;
  }
}

template <typename T, int D, int IT>
__global__ void __launch_bounds__(256) k_kv4_load(const Kv4RowsParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const Kv4Place t = Kv4Place::at<D, IT>(p);
  T* dst = static_cast<T*>(const_cast<void*>(t.is_v ? p.v : p.k)) + t.head * D + t.l * 8;
  const int64_t ld = t.is_v ? p.ldv : p.ldk;
  const uint8_t* codes = t.is_v ? p.c.v_codes : p.c.k_codes;
  const __nv_bfloat16* scales = (t.is_v ? p.c.v_scales : p.c.k_scales) + t.g;
  const int64_t slots = p.c.num_pages * p.c.page_rows;
  int32_t slot[IT];
  uint32_t word[IT];
  float s[IT];
#pragma unroll
  for (int u = 0; u < IT; ++u) {
    const int64_t row = t.row0 + u * t.step;
    slot[u] = t.mine && row < p.rows ? p.slots[row] : -1;
  }
#pragma unroll
  for (int u = 0; u < IT; ++u) {
    if (slot[u] >= slots) {
      if (t.li == 0) raise_error(kErrKvSlot, 2);
      slot[u] = -1;
    }
    word[u] = 0;
    s[u] = 0.0f;
    if (slot[u] >= 0) {
      const int64_t at = kv4_row(p.c, slot[u], t.head);
      word[u] = *reinterpret_cast<const uint32_t*>(codes + at * (D / 2) + kv4_word<D>(2 * t.l4 + (t.g & 1), t.g >> 1, slot[u]));
      s[u] = __bfloat162float(scales[at * (D / 32)]);
    }
  }
#pragma unroll
  for (int u = 0; u < IT; ++u) {
    const uint32_t got = __shfl_xor_sync(0xffffffffu, t.g & 1 ? word[u] & 0xffffu : word[u] >> 16, 4);
    const uint32_t w = t.g & 1 ? got | (word[u] & 0xffff0000u) : (word[u] & 0xffffu) | got << 16;
    const int64_t row = t.row0 + u * t.step;
    const float2 v[4] = {e2m1_values<0>(w), e2m1_values<1>(w), e2m1_values<2>(w), e2m1_values<3>(w)};
    float x[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = v[e].x * s[u];
      x[2 * e + 1] = v[e].y * s[u];
    }
    if constexpr (sizeof(T) == 4) {
      // 32 bytes a lane: the lanes of a pair trade halves, so that one store writes whole sectors
      const bool odd = t.l & 1;
      float give[4], own[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        give[e] = __shfl_xor_sync(0xffffffffu, odd ? x[e] : x[e + 4], 1);
        own[e] = odd ? x[e + 4] : x[e];
      }
      if (slot[u] < 0) continue;
      float* out = reinterpret_cast<float*>(dst + row * ld);
      *reinterpret_cast<float4*>(out + (odd ? -4 : 0)) = odd ? make_float4(give[0], give[1], give[2], give[3])
                                                             : make_float4(own[0], own[1], own[2], own[3]);
      *reinterpret_cast<float4*>(out + (odd ? 4 : 8)) = odd ? make_float4(own[0], own[1], own[2], own[3])
                                                            : make_float4(give[0], give[1], give[2], give[3]);
    } else {
      if (slot[u] < 0) continue;
      store8(dst + row * ld, x);
    }
    if (t.li == 0 && p.bias) p.bias[row] = p.c.bias ? p.c.bias[slot[u]] : 0.0f;
  }
}

}  // namespace tg

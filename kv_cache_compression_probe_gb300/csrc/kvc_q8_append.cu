// kvc_q8_append and kvc_q8_pack: rows into the 8-bit cache.
//
// A task is the keys, or the values, that go into one page of a unit: one warp's for up to 8
// tokens, a CTA's (8 warps) for more.  D / 16 lanes hold a row, 8 elements of each half a lane, so
// that a rotation's pairs meet in a lane and loads and stores are 16 and 8 bytes.  The largest magnitude of the new
// rows and the page's old scale give the new one; rows stay in registers until
// then (beyond 8 a warp they are read again).  Only when the scale grows are the page's old
// codes read and moved to it.
// Bound by latency: one token of 4096 (b,l,h) with 16384 query rows 8.9 us (with a CTA of 8 warps a page 28, most of them
// idle), a 2048-token chunk of 8 KV heads, 47 MB, 11.8 us (with 4 loads of 4 bytes a lane and row 26).
#include <algorithm>

#include "kvc_chunk_tc.cuh"
#include "kvc_q8.cuh"

namespace {

using kvc::Q8Args;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kFew = 8;                // tokens up to which a task is one warp's
constexpr int kQPasses = 2;            // query rows of a lane

struct Q8Append {
  Q8Args x;
  const float* cos_tab;                // null: no rotation
  const float* sin_tab;
  const void* q;                       // null: no queries
  const void* k_new;
  const void* v_new;
  const float* pos_new;
  void* q_out;
  const int32_t* cap_lh;
  int32_t* len_out;
  int64_t n_half, page_ctas, tasks;
  int per_unit;                        // pages of a unit that a call can touch
};

// Lane i of a row's D / 16: elements 8i .. 8i + 7 of each half.
template <typename T, int D>
__device__ __forceinline__ void load_row(const T* row, int i, float (&v)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const T* p = row + h * (D / 2) + 8 * i;
    if constexpr (sizeof(T) == 2) {
      const uint4 w = *reinterpret_cast<const uint4*>(p);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[8 * h + 2 * k] = __uint_as_float(u[k] << 16);
        v[8 * h + 2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
      }
    } else {
      kvcd::load4(p, v + 8 * h);
      kvcd::load4(p + 4, v + 8 * h + 4);
    }
  }
}

// The rotation by table row e; every product and sum is rounded by itself, so that the codes
// can be reproduced bit for bit.
template <int D>
__device__ __forceinline__ void load_angles(const Q8Append& a, int64_t e, int i, float (&c)[8], float (&s)[8]) {
  const int64_t at = e * (D / 2) + 8 * i;
#pragma unroll
  for (int k = 0; k < 8; k += 4) {
    kvcd::VecLoad<float, 4>::ld(a.cos_tab + at + k, c + k);
    kvcd::VecLoad<float, 4>::ld(a.sin_tab + at + k, s + k);
  }
}
__device__ __forceinline__ void rotate(float (&v)[16], const float (&c)[8], const float (&s)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float x = v[k], y = v[8 + k];
    v[k] = __fsub_rn(__fmul_rn(x, c[k]), __fmul_rn(y, s[k]));
    v[8 + k] = __fadd_rn(__fmul_rn(y, c[k]), __fmul_rn(x, s[k]));
  }
}

// Table row of a position, or -1 outside the table (the last of n tokens included).
__device__ __forceinline__ int64_t table_row(float pos, int n, int64_t n_half) {
  if (!(pos >= 0.f && pos < 8388608.f)) return -1;
  const int64_t e = (int64_t)(2.f * pos);
  return e + 2 * (int64_t)(n - 1) < n_half ? e : -1;
}

// Bounds of four features, a byte each.
struct Bounds4 {
  uint32_t lo, hi;
};
constexpr uint32_t kNoLo = 0x7f7f7f7fu, kNoHi = 0x81818181u;      // 127, -127
__device__ __forceinline__ void join(Bounds4& a, uint32_t lo, uint32_t hi) {
  a.lo = __vmins4(a.lo, lo);
  a.hi = __vmaxs4(a.hi, hi);
}
// Codes as signed bytes in the order of their values.
__device__ __forceinline__ uint32_t in_order(uint32_t codes) {
  const uint32_t s = codes & 0x80808080u;
  return codes ^ (s - (s >> 7));
}
// rint(value / 4) of four codes in that order.
__device__ __forceinline__ uint32_t bounds_of(uint32_t ordered) {
  const uint32_t c = in_order(ordered);                // its own inverse
  float v[4];
  kvcd::e4m3_f32((uint16_t)c, v[0], v[1]);
  kvcd::e4m3_f32((uint16_t)(c >> 16), v[2], v[3]);
  uint32_t w = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) w |= (uint32_t)(kvcd::bound_of(v[k]) & 255) << (8 * k);
  return w;
}

template <int D>
struct TaskSmem {
  float top[kWarps];
  Bounds4 b[kWarps][D / 16][4];
};

// A page's part of a task, by kW warps (w: this one's number among them).  page_of() checks the unit's
// pages and gives the task's, or -1; it comes after the first rows' loads, which need not wait
// for the page table.
template <typename T, int D, int kW, bool kKeys, class Page>
__device__ __forceinline__ void append_page(const Q8Append& a, int64_t u, int old, int t0, int count, int64_t e0, int w,
                                            TaskSmem<D>& sm, const Page& page_of) {
  constexpr int kL = D / 16, kG = 32 / kL, kStep = kW * kG, kHold = kW > 1 && kG < 8 ? 2 : 1;
  const Q8Args& x = a.x;
  const int lane = threadIdx.x & 31, i = lane % kL, r0 = w * kG + lane / kL;   // first row of this lane
  const T* rows = static_cast<const T*>(kKeys ? a.k_new : a.v_new) + (u * x.T + t0) * D;
  const bool turn = kKeys && a.cos_tab, bounds = kKeys && x.bounds;
  auto row = [&](int r, float (&v)[16]) {
    load_row<T, D>(rows + (int64_t)r * D, i, v);
    if (turn) {
      float c[8], s[8];
      load_angles<D>(a, e0 + 2 * (int64_t)(t0 + r), i, c, s);
      rotate(v, c, s);
    }
  };
  float held[kHold][16], top = 0.f;
#pragma unroll
  for (int k = 0; k < kHold; ++k)
    if (r0 + k * kStep < count) row(r0 + k * kStep, held[k]);
  const int64_t page = page_of();
  if (page < 0) return;
  float* scale = (kKeys ? x.k_scale : x.v_scale) + page;
  const int x_old = old > 0 ? kvcd::scale_exp(*scale) : kvc::kQ8MinExp;
#pragma unroll
  for (int k = 0; k < kHold; ++k)
    if (r0 + k * kStep < count)
#pragma unroll
      for (int f = 0; f < 16; ++f) top = fmaxf(top, fabsf(held[k][f]));
  for (int r = r0 + kHold * kStep; r < count; r += kStep) {
    float v[16];
    row(r, v);
#pragma unroll
    for (int f = 0; f < 16; ++f) top = fmaxf(top, fabsf(v[f]));
  }
  top = kvcd::warp_max(top);
  if constexpr (kW > 1) {
    if (lane == 0) sm.top[w] = top;
    __syncthreads();                                   // and every thread has read the old scale
#pragma unroll
    for (int k = 0; k < kW; ++k) top = fmaxf(top, sm.top[k]);
  }
  const int xs = max(x_old, kvcd::scale_for(top));
  const bool grow = old > 0 && xs > x_old;
  uint8_t* codes = (kKeys ? x.K : x.V) + (page << x.shift) * D + 8 * i;
  Bounds4 b[4];                                        // of this lane's features, codes in order
#pragma unroll
  for (int k = 0; k < 4; ++k) b[k] = Bounds4{kNoLo, kNoHi};
  if (grow) {                                          // the old codes move to the new scale
    const float f = kvcd::pow2i(x_old - xs);
    for (int r = r0; r < old; r += kStep)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint2* p = reinterpret_cast<uint2*>(codes + r * D + h * (D / 2));
        const uint2 was = *p;
        uint32_t c[2] = {was.x, was.y};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float y[4];
          kvcd::e4m3_f32((uint16_t)c[k], y[0], y[1]);
          kvcd::e4m3_f32((uint16_t)(c[k] >> 16), y[2], y[3]);
          c[k] = kvcd::f32_e4m3x2(y[0] * f, y[1] * f) | (uint32_t)kvcd::f32_e4m3x2(y[2] * f, y[3] * f) << 16;
          if (bounds) join(b[2 * h + k], in_order(c[k]), in_order(c[k]));
        }
        *p = make_uint2(c[0], c[1]);
      }
  }
  const float f = kvcd::pow2i(-xs);
  auto put = [&](int r, const float (&v)[16]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t c[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float* y = v + 8 * h + 4 * k;
        c[k] = kvcd::f32_e4m3x2(y[0] * f, y[1] * f) | (uint32_t)kvcd::f32_e4m3x2(y[2] * f, y[3] * f) << 16;
        if (bounds) join(b[2 * h + k], in_order(c[k]), in_order(c[k]));
      }
      *reinterpret_cast<uint2*>(codes + (old + r) * D + h * (D / 2)) = make_uint2(c[0], c[1]);
    }
  };
#pragma unroll
  for (int k = 0; k < kHold; ++k)
    if (r0 + k * kStep < count) put(r0 + k * kStep, held[k]);
  for (int r = r0 + kHold * kStep; r < count; r += kStep) {
    float v[16];
    row(r, v);
    put(r, v);
  }
  if (w == 0 && lane == 0) *scale = kvcd::pow2i(xs);
  if (kKeys && x.logm)
    for (int r = w * 32 + lane; r < count; r += 32 * kW) x.logm[(page << x.shift) + old + r] = 0.f;
  if constexpr (kKeys) {
    if (!bounds) return;
    const bool one = kW == 1 && count == 1 && !grow;   // a single row, which the first lanes hold: lo is hi
    if (!one)
#pragma unroll
      for (int o = kL; o < 32; o <<= 1)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          join(b[k], __shfl_xor_sync(KVC_FULL_MASK, b[k].lo, o), __shfl_xor_sync(KVC_FULL_MASK, b[k].hi, o));
    if constexpr (kW > 1) {
      if (lane < kL)
#pragma unroll
        for (int k = 0; k < 4; ++k) sm.b[w][lane][k] = b[k];
      __syncthreads();
      if (w > 0) return;
      for (int v = 1; v < kWarps; ++v)
#pragma unroll
        for (int k = 0; k < 4; ++k) join(b[k], sm.b[v][i][k].lo, sm.b[v][i][k].hi);
    }
    if (lane >= kL) return;
    int8_t* to = x.bounds + page * 2 * D + 8 * i;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint2* lo = reinterpret_cast<uint2*>(to + h * (D / 2));
      uint2* hi = reinterpret_cast<uint2*>(to + D + h * (D / 2));
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        b[2 * h + k].lo = bounds_of(b[2 * h + k].lo);
        b[2 * h + k].hi = one ? b[2 * h + k].lo : bounds_of(b[2 * h + k].hi);
      }
      if (old > 0 && !grow) {
        const uint2 l = *lo, m = *hi;
        join(b[2 * h], l.x, m.x);
        join(b[2 * h + 1], l.y, m.y);
      }
      *lo = make_uint2(b[2 * h].lo, b[2 * h + 1].lo);
      *hi = make_uint2(b[2 * h].hi, b[2 * h + 1].hi);
    }
  }
}

// Query rows: a lane has the same 8 + 8 elements of kQPasses rows.
template <typename T, int D>
__device__ __forceinline__ void rotate_queries(const Q8Append& a, int64_t warp) {
  constexpr int kL = D / 16, kG = 32 / kL;
  const Q8Args& x = a.x;
  const int lane = threadIdx.x & 31, i = lane % kL;
  const int64_t r0 = warp * kG * kQPasses + lane / kL;
  const uint32_t total = (uint32_t)(x.units * x.G * x.T), per_b = (uint32_t)(x.per_seq * x.G) * x.T;   // rows, below 2^32
  float v[kQPasses][16];
  int64_t e[kQPasses];
#pragma unroll
  for (int k = 0; k < kQPasses; ++k) {
    e[k] = -1;
    if (r0 + k * kG >= total) continue;
    const uint32_t r = (uint32_t)(r0 + k * kG);
    const int b = (int)(r / per_b), t = (int)(r % (uint32_t)x.T);
    const int n = x.n_new ? __ldg(x.n_new + b) : x.T;
    if (n > x.T || t >= n) continue;
    e[k] = a.cos_tab ? table_row(__ldg(a.pos_new + b), n, a.n_half) : 0;
    if (e[k] < 0) continue;
    e[k] += 2 * (int64_t)t;
    load_row<T, D>(static_cast<const T*>(a.q) + (int64_t)r * D, i, v[k]);
  }
#pragma unroll
  for (int k = 0; k < kQPasses; ++k) {
    if (e[k] < 0) continue;
    if (a.cos_tab) {
      float c[8], s[8];
      load_angles<D>(a, e[k], i, c, s);
      rotate(v[k], c, s);
    }
    T* to = static_cast<T*>(a.q_out) + (r0 + k * kG) * D + 8 * i;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if constexpr (sizeof(T) == 2) {
        uint32_t y[4];
#pragma unroll
        for (int f = 0; f < 4; ++f) y[f] = kvctc::bf16x2(v[k][8 * h + 2 * f], v[k][8 * h + 2 * f + 1]);
        *reinterpret_cast<uint4*>(to + h * (D / 2)) = make_uint4(y[0], y[1], y[2], y[3]);
      } else {
#pragma unroll
        for (int f = 0; f < 8; f += 4)
          *reinterpret_cast<float4*>(to + h * (D / 2) + f) =
              make_float4(v[k][8 * h + f], v[k][8 * h + f + 1], v[k][8 * h + f + 2], v[k][8 * h + f + 3]);
      }
  }
}

template <typename T, int D, int kW>
__global__ void __launch_bounds__(kThreads, kW > 1 ? 3 : 4) q8_append_kernel(const __grid_constant__ Q8Append a) {
  __shared__ TaskSmem<D> sm;                           // kW > 1: a CTA is one task
  const Q8Args& x = a.x;
  kvcd::pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x >= a.page_ctas) {
    rotate_queries<T, D>(a, (blockIdx.x - a.page_ctas) * kWarps + warp);
    kvcd::pdl_trigger();
    return;
  }
  const uint32_t task = blockIdx.x * (uint32_t)(kWarps / kW) + warp / kW;
  if (task >= a.tasks) return;
  const uint32_t u = (task >> 1) / (uint32_t)a.per_unit;
  const int j = (int)((task >> 1) - u * (uint32_t)a.per_unit);
  const int b = (int)(u / (uint32_t)x.per_seq);
  const int64_t gu = kvcd::q8_unit_global(x, u);
  const int len = x.len_lh[gu], n = x.n_new ? __ldg(x.n_new + b) : x.T, cap = __ldg(a.cap_lh + gu);
  const int64_t e0 = a.cos_tab ? table_row(__ldg(a.pos_new + b), n, a.n_half) : 0;
  int bad = KVC_OK;
  if (len < 0 || n < 0 || n > x.T || (n > 0 && e0 < 0)) bad = KVC_EDEVICE;
  else if ((int64_t)len + n > cap) bad = KVC_ECAPACITY;
  else if ((int64_t)len + n > (int64_t)x.max_pages << x.shift) bad = KVC_EDEVICE;
  const int32_t* tab = x.table + gu * x.max_pages;
  const int first = len >> x.shift, last = n > 0 ? (len + n - 1) >> x.shift : first - 1;
  // Every warp looks at all the pages that the unit's tokens touch; the first one reports.
  auto page_of = [&]() -> int64_t {
    bool ok = true;
    int mine = 0;
    if (bad == KVC_OK)
      for (int i = first + lane; i <= last; i += 32) {
        const int page = __ldg(tab + i);
        ok &= (unsigned)page < (unsigned)x.pages;
        if (i == first + j) mine = page;
      }
    if (!__all_sync(KVC_FULL_MASK, ok) && bad == KVC_OK) bad = KVC_EDEVICE;
    if (j == 0 && (task & 1) == 0 && warp % kW == 0 && lane == 0) {
      if (bad != KVC_OK) kvcd::record_error(x.err, bad);
      a.len_out[gu] = bad == KVC_OK ? len + n : len;
    }
    return bad == KVC_OK ? __shfl_sync(KVC_FULL_MASK, mine, j & 31) : -1;
  };
  if (bad == KVC_OK && first + j <= last) {
    const int begin = (first + j) << x.shift;
    const int old = max(0, len - begin), t0 = begin + old - len;
    const int count = min(1 << x.shift, len + n - begin) - old;
    if (task & 1) append_page<T, D, kW, false>(a, u, old, t0, count, e0, warp % kW, sm, page_of);
    else append_page<T, D, kW, true>(a, u, old, t0, count, e0, warp % kW, sm, page_of);
  } else if (j == 0) {
    page_of();
  }
  kvcd::pdl_trigger();
}

// ---------------------------------------------------------------- pack
__device__ __forceinline__ void half_sync(int half) { asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory"); }

struct PageSmem {
  float top[2][4];
  int lo[128], hi[128];
};

// The page's bounds from shared memory, four bytes a thread.
template <int D>
__device__ __forceinline__ void store_bounds(int8_t* out, int i, const PageSmem& sm) {
  if (i < D / 2) {
    const int* from = i < D / 4 ? sm.lo + 4 * i : sm.hi + 4 * (i - D / 4);
    const uint32_t w = (uint32_t)(from[0] & 255) | (uint32_t)(from[1] & 255) << 8 | (uint32_t)(from[2] & 255) << 16 |
                       (uint32_t)(from[3] & 255) << 24;
    reinterpret_cast<uint32_t*>(out)[i] = w;
  }
}

struct Q8Pack {
  Q8Args x;
  const void* Kp;
  const void* Vp;
  const float* logm;
  const int64_t* off_lh;
  const int32_t* cap_lh;
  int32_t* len_out;
  int64_t rows;
};

// One CTA per (unit, page of its table): rows off + j R .. of the packed cache.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) q8_pack_kernel(const __grid_constant__ Q8Pack a) {
  __shared__ PageSmem sm;
  constexpr int kC = D / 8;                            // threads of a row, eight elements each
  const Q8Args& x = a.x;
  kvcd::pdl_trigger();
  kvcd::pdl_wait();
  const int64_t u = blockIdx.x / x.max_pages;
  const int j = (int)(blockIdx.x - u * x.max_pages);
  const int64_t gu = kvcd::q8_unit_global(x, u), off = a.off_lh[gu];
  const int len = x.len_lh[gu], cap = a.cap_lh[gu], R = 1 << x.shift;
  const int32_t* tab = x.table + gu * x.max_pages;
  int bad = KVC_OK;
  if (!kvc::rows_fit(off, len, a.rows)) bad = KVC_EDEVICE;
  else if (len > cap) bad = KVC_ECAPACITY;
  else if (len > (int64_t)x.max_pages << x.shift) bad = KVC_EDEVICE;
  bool ok = true;
  const int need = bad == KVC_OK ? (int)(((int64_t)len + R - 1) >> x.shift) : 0;
  for (int i = threadIdx.x; i < need; i += kThreads) ok &= (unsigned)__ldg(tab + i) < (unsigned)x.pages;
  if (!__syncthreads_and(ok)) bad = KVC_EDEVICE;
  if (j == 0 && threadIdx.x == 0) {
    if (bad != KVC_OK) kvcd::record_error(x.err, bad);
    a.len_out[gu] = bad == KVC_OK ? len : 0;
  }
  if (bad != KVC_OK || j >= need) return;
  const int half = threadIdx.x >> 7, i = threadIdx.x & 127, c = i % kC;
  const int count = min(R, len - (j << x.shift));
  const int64_t page = __ldg(tab + j), from = off + ((int64_t)j << x.shift);
  const T* rows = static_cast<const T*>(half ? a.Vp : a.Kp) + from * D + c * 8;
  float top = 0.f, v[8];
  for (int r = i / kC; r < count; r += 128 / kC) {
    kvcd::load4(rows + (int64_t)r * D, v);
    kvcd::load4(rows + (int64_t)r * D + 4, v + 4);
#pragma unroll
    for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(v[k]));
  }
  top = kvcd::warp_max(top);
  if ((i & 31) == 0) sm.top[half][i >> 5] = top;
  if (half == 0 && i < D) { sm.lo[i] = 127; sm.hi[i] = -127; }
  half_sync(half);
  const float* tops = sm.top[half];
  const int xs = kvcd::scale_for(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])));
  const float f = kvcd::pow2i(-xs);
  const bool bounds = half == 0 && x.bounds;
  int lo[8], hi[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) { lo[k] = 127; hi[k] = -127; }
  uint8_t* codes = (half ? x.V : x.K) + (page << x.shift) * D + c * 8;
  for (int r = i / kC; r < count; r += 128 / kC) {
    kvcd::load4(rows + (int64_t)r * D, v);
    kvcd::load4(rows + (int64_t)r * D + 4, v + 4);
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint16_t code = kvcd::f32_e4m3x2(v[2 * k] * f, v[2 * k + 1] * f);
      w[k >> 1] = k & 1 ? w[k >> 1] | (uint32_t)code << 16 : code;
      if (bounds) {
        float y[2];
        kvcd::e4m3_f32(code, y[0], y[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          lo[2 * k + h] = min(lo[2 * k + h], kvcd::bound_of(y[h]));
          hi[2 * k + h] = max(hi[2 * k + h], kvcd::bound_of(y[h]));
        }
      }
    }
    *reinterpret_cast<uint2*>(codes + r * D) = make_uint2(w[0], w[1]);
  }
  if (bounds && i / kC < count)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      atomicMin(&sm.lo[c * 8 + k], lo[k]);
      atomicMax(&sm.hi[c * 8 + k], hi[k]);
    }
  if (i == 0) (half ? x.v_scale : x.k_scale)[page] = kvcd::pow2i(xs);
  if (half == 1 && x.logm)
    for (int r = i; r < count; r += 128) x.logm[(page << x.shift) + r] = a.logm[from + r];
  half_sync(half);
  if (bounds) store_bounds<D>(x.bounds + page * 2 * D, i, sm);
}

}  // namespace

namespace kvc {

int q8_check(const kvc_params* p, const kvc_chunk* c, const kvc_q8* x) {
  const int st = chunk_check(p, c);
  if (st != KVC_OK) return st;
  if (c->page_rows < 16 || c->page_rows > 128) return KVC_EINVAL;
  if (c->softcap != 0.f || c->window != 0.f || c->slopes) return KVC_EINVAL;
  if (c->max_pages > (1 << 27) / c->page_rows) return KVC_EINVAL;      // entries of a (b,l,h) fit 27 bits
  if (!x || !x->K || !x->V || !x->k_scale || !x->v_scale) return KVC_EINVAL;
  if (q8_misaligned(x->K, 16) || q8_misaligned(x->V, 16) || q8_misaligned(x->bounds, 16)) return KVC_EINVAL;
  return KVC_OK;
}

void q8_fill(Q8Args& a, const kvc_params* p, const kvc_chunk* c, const kvc_q8* x) {
  ChunkArgs k = {};
  chunk_fill(k, p, c);
  a.K = x->K;
  a.V = x->V;
  a.k_scale = x->k_scale;
  a.v_scale = x->v_scale;
  a.bounds = x->bounds;
  a.logm = x->logm;
  a.table = c->page_table;
  a.n_new = c->n_new;
  a.units = k.units;
  a.lh_span = k.lh_span;
  a.lh_gap = k.lh_gap;
  a.lh_base = k.lh_base;
  a.T = k.T;
  a.H = k.H;
  a.G = k.G;
  a.per_seq = k.per_seq;
  a.max_pages = k.max_pages;
  a.shift = k.page_shift;
  a.pages = (int)(p->packed_rows >> k.page_shift);
  a.err = err_word();
}

}  // namespace kvc

extern "C" int kvc_q8_append(const kvc_params* p, const kvc_chunk* c, const kvc_q8* x, const float* rope_cos,
                             const float* rope_sin, int64_t n_half, const void* q, const void* k_new,
                             const void* v_new, const float* pos_new, void* q_out, const int32_t* len_lh,
                             const int32_t* cap_lh, int32_t* len_out, void* stream) {
  const int st = kvc::q8_check(p, c, x);
  if (st != KVC_OK) return st;
  if (!k_new || !v_new || !len_lh || !cap_lh || !len_out || len_out == len_lh) return KVC_EINVAL;
  if ((q != nullptr) != (q_out != nullptr) || (rope_cos != nullptr) != (rope_sin != nullptr)) return KVC_EINVAL;
  if (rope_cos && (!pos_new || n_half < 1)) return KVC_EINVAL;
  if (kvc::q8_misaligned(q, 16) || kvc::q8_misaligned(k_new, 16) || kvc::q8_misaligned(v_new, 16) ||
      kvc::q8_misaligned(q_out, 16) || kvc::q8_misaligned(rope_cos, 16) || kvc::q8_misaligned(rope_sin, 16))
    return KVC_EINVAL;
  Q8Append a = {};
  kvc::q8_fill(a.x, p, c, x);
  if (!a.x.err) return KVC_ECUDA;
  a.x.len_lh = len_lh;
  a.cos_tab = rope_cos;
  a.sin_tab = rope_sin;
  a.n_half = n_half;
  a.q = q;
  a.q_out = q_out;
  a.k_new = k_new;
  a.v_new = v_new;
  a.pos_new = pos_new;
  a.cap_lh = cap_lh;
  a.len_out = len_out;
  const int R = c->page_rows;
  const bool few = c->T <= kFew;
  a.per_unit = std::min((c->T + R - 2) / R + 1, c->max_pages);
  a.tasks = 2 * a.x.units * a.per_unit;
  a.page_ctas = few ? (a.tasks + kWarps - 1) / kWarps : a.tasks;
  const int64_t rows = q ? a.x.units * a.x.G * a.x.T : 0, per = kWarps * kQPasses * (512 / p->d);
  const int64_t grid = a.page_ctas + (rows + per - 1) / per;
  if (grid >= (1LL << 31) || rows >= (1LL << 32) - 4096 || a.tasks >= (1LL << 32)) return KVC_EINVAL;
  using B = __nv_bfloat16;
  auto kernel = p->dtype == KVC_BF16 ? (p->d == 128 ? (few ? q8_append_kernel<B, 128, 1> : q8_append_kernel<B, 128, kWarps>)
                                                    : (few ? q8_append_kernel<B, 64, 1> : q8_append_kernel<B, 64, kWarps>))
                                     : (p->d == 128 ? (few ? q8_append_kernel<float, 128, 1> : q8_append_kernel<float, 128, kWarps>)
                                                    : (few ? q8_append_kernel<float, 64, 1> : q8_append_kernel<float, 64, kWarps>));
  kvc::count_launch();
  return kvc::cuda_status(kvc::chunk_launch(kernel, dim3((unsigned)grid), dim3(kThreads), 0,
                                            static_cast<cudaStream_t>(stream), a));
}

extern "C" int kvc_q8_pack(const kvc_params* p, const kvc_chunk* c, const kvc_q8* x, const void* Kp, const void* Vp,
                           const float* logm, int64_t rows, const int32_t* len_lh, const int64_t* off_lh,
                           const int32_t* cap_lh, int32_t* len_out, void* stream) {
  const int st = kvc::q8_check(p, c, x);
  if (st != KVC_OK) return st;
  if (!Kp || !Vp || !len_lh || !off_lh || !cap_lh || !len_out || len_out == len_lh || rows < 1) return KVC_EINVAL;
  if ((logm != nullptr) != (x->logm != nullptr)) return KVC_EINVAL;
  if (kvc::q8_misaligned(Kp, 16) || kvc::q8_misaligned(Vp, 16)) return KVC_EINVAL;
  Q8Pack a = {};
  kvc::q8_fill(a.x, p, c, x);
  if (!a.x.err) return KVC_ECUDA;
  a.x.len_lh = len_lh;
  a.Kp = Kp;
  a.Vp = Vp;
  a.logm = logm;
  a.rows = rows;
  a.off_lh = off_lh;
  a.cap_lh = cap_lh;
  a.len_out = len_out;
  const int64_t grid = a.x.units * c->max_pages;
  if (grid >= (1LL << 31)) return KVC_EINVAL;
  auto kernel = p->dtype == KVC_BF16 ? (p->d == 128 ? q8_pack_kernel<__nv_bfloat16, 128> : q8_pack_kernel<__nv_bfloat16, 64>)
                                     : (p->d == 128 ? q8_pack_kernel<float, 128> : q8_pack_kernel<float, 64>);
  kvc::count_launch();
  return kvc::cuda_status(kvc::chunk_launch(kernel, dim3((unsigned)grid), dim3(kThreads), 0,
                                            static_cast<cudaStream_t>(stream), a));
}

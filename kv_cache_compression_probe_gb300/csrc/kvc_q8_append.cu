// kvc_q8_append and kvc_q8_pack: rows into the 8-bit cache.
//
// One CTA per (unit, page that the call writes): four warps for the keys and four for the
// values.  The page's new rows are read twice (the second time from L1): once for their
// largest magnitude, which with the page's old scale gives the new one, and once for the
// codes.  Only when the scale grows are the page's old codes read and moved to it.
#include <algorithm>

#include "kvc_q8.cuh"

namespace {

using kvc::Q8Args;

constexpr int kThreads = 256;
constexpr int kQRows = 4;              // query rows of a warp

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
  int64_t n_half, page_ctas;
  int per_unit;                        // CTAs of a unit
};

// A row of D elements over a warp: lane i has elements i*kP .. of the first half in v[0 .. kP)
// and the same of the second half in v[kP ..), which the rotation pairs.
template <typename T, int D>
__device__ __forceinline__ void load_row(const T* row, int lane, float (&v)[D / 32]) {
  constexpr int kP = D / 64;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const T* p = row + h * (D / 2) + lane * kP;
    if constexpr (kP == 2) {
      kvcd::VecLoad<T, 2>::ld(p, v + h * kP);
    } else {
      v[h] = kvcd::to_f(*p);
    }
  }
}

// The rotation by table row e; every product and sum is rounded by itself, so that the codes
// can be reproduced bit for bit.
template <int D>
__device__ __forceinline__ void rotate(float (&v)[D / 32], const float* cos_tab, const float* sin_tab, int64_t e,
                                       int lane) {
  constexpr int kP = D / 64;
#pragma unroll
  for (int i = 0; i < kP; ++i) {
    const float c = __ldg(cos_tab + e * (D / 2) + lane * kP + i), s = __ldg(sin_tab + e * (D / 2) + lane * kP + i);
    const float a = v[i], b = v[kP + i];
    v[i] = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    v[kP + i] = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  }
}

// Table row of a position, or -1 outside the table (the last of n tokens included).
__device__ __forceinline__ int64_t table_row(float pos, int n, int64_t n_half) {
  if (!(pos >= 0.f && pos < 8388608.f)) return -1;
  const int64_t e = (int64_t)(2.f * pos);
  return e + 2 * (int64_t)(n - 1) < n_half ? e : -1;
}

__device__ __forceinline__ void half_sync(int half) { asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory"); }

struct PageSmem {
  float top[2][4];
  int lo[128], hi[128];
};

// Moves a page's first `rows` codes to a scale 2^up times as large, and (kBounds) adds them to
// the bounds.  By the 128 threads of a half.
template <int D, bool kBounds>
__device__ __forceinline__ void rescale(uint8_t* page, int rows, int up, int i, PageSmem& sm) {
  constexpr int kC = D / 16;
  const float f = kvcd::pow2i(-up);
  const int c = i % kC;
  int lo[16], hi[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) { lo[k] = 127; hi[k] = -127; }
  for (int r = i / kC; r < rows; r += 128 / kC) {
    uint4* p = reinterpret_cast<uint4*>(page + r * D + c * 16);
    uint4 w = *p;
    uint32_t* u = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int sh = (k & 1) * 16;
      float a, b;
      kvcd::e4m3_f32((uint16_t)(u[k >> 1] >> sh), a, b);
      const uint16_t code = kvcd::f32_e4m3x2(a * f, b * f);
      u[k >> 1] = (u[k >> 1] & ~(0xffffu << sh)) | ((uint32_t)code << sh);
      if (kBounds) {
        kvcd::e4m3_f32(code, a, b);
        const int x = kvcd::bound_of(a), y = kvcd::bound_of(b);
        lo[2 * k] = min(lo[2 * k], x);
        hi[2 * k] = max(hi[2 * k], x);
        lo[2 * k + 1] = min(lo[2 * k + 1], y);
        hi[2 * k + 1] = max(hi[2 * k + 1], y);
      }
    }
    *p = w;
  }
  if (kBounds && i / kC < rows)
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      atomicMin(&sm.lo[c * 16 + k], lo[k]);
      atomicMax(&sm.hi[c * 16 + k], hi[k]);
    }
}

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

template <typename T, int D, bool kKeys>
__device__ __forceinline__ void append_page(const Q8Append& a, int64_t u, int64_t page, int old, int t0, int count,
                                            int64_t e0, PageSmem& sm) {
  constexpr int kP = D / 64;
  const Q8Args& x = a.x;
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) & 3, i = threadIdx.x & 127;
  const T* rows = static_cast<const T*>(kKeys ? a.k_new : a.v_new) + (u * x.T + t0) * D;
  const bool turn = kKeys && a.cos_tab, bounds = kKeys && x.bounds;
  float v[D / 32], top = 0.f;
  for (int r = w; r < count; r += 4) {
    load_row<T, D>(rows + (int64_t)r * D, lane, v);
    if (turn) rotate<D>(v, a.cos_tab, a.sin_tab, e0 + 2 * (int64_t)(t0 + r), lane);
#pragma unroll
    for (int k = 0; k < 2 * kP; ++k) top = fmaxf(top, fabsf(v[k]));
  }
  top = kvcd::warp_max(top);
  if (lane == 0) sm.top[kKeys ? 0 : 1][w] = top;
  float* scale = (kKeys ? x.k_scale : x.v_scale) + page;
  const int x_old = old > 0 ? kvcd::scale_exp(*scale) : kvc::kQ8MinExp;
  half_sync(!kKeys);
  const float* tops = sm.top[kKeys ? 0 : 1];
  const int xs = max(x_old, kvcd::scale_for(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]))));
  const bool grow = old > 0 && xs > x_old;
  uint8_t* codes = (kKeys ? x.K : x.V) + (page << x.shift) * D;
  if (bounds) {
    const int8_t* was = x.bounds + page * 2 * D;
    if (i < D) {
      sm.lo[i] = old > 0 && !grow ? was[i] : 127;
      sm.hi[i] = old > 0 && !grow ? was[D + i] : -127;
    }
    half_sync(!kKeys);
  }
  if (grow) {
    if (bounds) rescale<D, true>(codes, old, xs - x_old, i, sm);
    else rescale<D, false>(codes, old, xs - x_old, i, sm);
  }
  const float f = kvcd::pow2i(-xs);
  int lo[2 * kP], hi[2 * kP];
#pragma unroll
  for (int k = 0; k < 2 * kP; ++k) { lo[k] = 127; hi[k] = -127; }
  for (int r = w; r < count; r += 4) {
    if (count > 4) {                                   // else v holds this warp's only row
      load_row<T, D>(rows + (int64_t)r * D, lane, v);
      if (turn) rotate<D>(v, a.cos_tab, a.sin_tab, e0 + 2 * (int64_t)(t0 + r), lane);
    }
    uint8_t* to = codes + (old + r) * D + lane * kP;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float y[2];
      const uint16_t c = kvcd::f32_e4m3x2(v[h * kP] * f, kP == 2 ? v[h * kP + kP - 1] * f : 0.f);
      if constexpr (kP == 2) *reinterpret_cast<uint16_t*>(to + h * (D / 2)) = c;
      else to[h * (D / 2)] = (uint8_t)c;
      if (bounds) {
        kvcd::e4m3_f32(c, y[0], y[1]);
#pragma unroll
        for (int k = 0; k < kP; ++k) {
          lo[h * kP + k] = min(lo[h * kP + k], kvcd::bound_of(y[k]));
          hi[h * kP + k] = max(hi[h * kP + k], kvcd::bound_of(y[k]));
        }
      }
    }
  }
  if (bounds && w < count)
#pragma unroll
    for (int k = 0; k < 2 * kP; ++k) {
      const int at = (k / kP) * (D / 2) + lane * kP + k % kP;
      atomicMin(&sm.lo[at], lo[k]);
      atomicMax(&sm.hi[at], hi[k]);
    }
  half_sync(!kKeys);                                   // every thread has read the old scale and bounds
  if (i == 0) *scale = kvcd::pow2i(xs);
  if (bounds) store_bounds<D>(x.bounds + page * 2 * D, i, sm);
  if (kKeys && x.logm)
    for (int r = i; r < count; r += 128) x.logm[(page << x.shift) + old + r] = 0.f;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) q8_append_kernel(const __grid_constant__ Q8Append a) {
  __shared__ PageSmem sm;
  const Q8Args& x = a.x;
  kvcd::pdl_trigger();
  kvcd::pdl_wait();
  const int lane = threadIdx.x & 31;
  if (blockIdx.x >= a.page_ctas) {                     // query rows, a few per warp
    const int64_t total = x.units * x.G * x.T;
    const int64_t r0 = ((blockIdx.x - a.page_ctas) * (kThreads / 32) + (threadIdx.x >> 5)) * kQRows;
    float v[kQRows][D / 32];
    int64_t e[kQRows];
#pragma unroll
    for (int k = 0; k < kQRows; ++k) {
      const int64_t r = r0 + k;
      e[k] = -1;
      if (r >= total) continue;
      const int64_t u = r / ((int64_t)x.G * x.T);
      const int t = (int)(r % x.T), b = (int)(u / x.per_seq);
      const int n = x.n_new ? x.n_new[b] : x.T;
      if (n > x.T || t >= n) continue;
      e[k] = a.cos_tab ? table_row(a.pos_new[b], n, a.n_half) : 0;
      if (e[k] < 0) continue;
      e[k] += 2 * (int64_t)t;
      load_row<T, D>(static_cast<const T*>(a.q) + r * D, lane, v[k]);
    }
#pragma unroll
    for (int k = 0; k < kQRows; ++k) {
      if (e[k] < 0) continue;
      if (a.cos_tab) rotate<D>(v[k], a.cos_tab, a.sin_tab, e[k], lane);
      T* to = static_cast<T*>(a.q_out) + (r0 + k) * D;
      constexpr int kP = D / 64;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < kP; ++i) to[h * (D / 2) + lane * kP + i] = kvcd::from_f<T>(v[k][h * kP + i]);
    }
    return;
  }
  const int64_t u = blockIdx.x / a.per_unit;
  const int j = (int)(blockIdx.x - u * a.per_unit);
  const int b = (int)(u / x.per_seq);
  const int64_t gu = kvcd::q8_unit_global(x, u);
  const int len = x.len_lh[gu], n = x.n_new ? x.n_new[b] : x.T, cap = a.cap_lh[gu];
  const int64_t e0 = a.cos_tab ? table_row(a.pos_new[b], n, a.n_half) : 0;
  int bad = KVC_OK;
  if (len < 0 || n < 0 || n > x.T || (int64_t)len + n > (int64_t)x.max_pages << x.shift || (n > 0 && e0 < 0))
    bad = KVC_EDEVICE;
  else if ((int64_t)len + n > cap)
    bad = KVC_ECAPACITY;
  const int32_t* tab = x.table + gu * x.max_pages;
  const int first = len >> x.shift, last = n > 0 ? (len + n - 1) >> x.shift : first - 1;
  bool ok = true;
  if (bad == KVC_OK)
    for (int i = first + threadIdx.x; i <= last; i += kThreads) ok &= (unsigned)__ldg(tab + i) < (unsigned)x.pages;
  if (!__syncthreads_and(ok) && bad == KVC_OK) bad = KVC_EDEVICE;
  if (j == 0 && threadIdx.x == 0) {
    if (bad != KVC_OK) kvcd::record_error(x.err, bad);
    a.len_out[gu] = bad == KVC_OK ? len + n : len;
  }
  if (bad != KVC_OK || first + j > last) return;
  const int begin = (first + j) << x.shift;
  const int old = max(0, len - begin), t0 = begin + old - len;
  const int count = min(1 << x.shift, len + n - begin) - old;
  const int64_t page = __ldg(tab + first + j);
  if (threadIdx.x < 128) append_page<T, D, true>(a, u, page, old, t0, count, e0, sm);
  else append_page<T, D, false>(a, u, page, old, t0, count, e0, sm);
}

// ---------------------------------------------------------------- pack
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
  if (len < 0 || len > (int64_t)x.max_pages << x.shift || off < 0 || off + len > a.rows) bad = KVC_EDEVICE;
  else if (len > cap) bad = KVC_ECAPACITY;
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
    kvcd::VecLoad<T, 4>::ld(rows + (int64_t)r * D, v);
    kvcd::VecLoad<T, 4>::ld(rows + (int64_t)r * D + 4, v + 4);
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
    kvcd::VecLoad<T, 4>::ld(rows + (int64_t)r * D, v);
    kvcd::VecLoad<T, 4>::ld(rows + (int64_t)r * D + 4, v + 4);
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
  a.per_unit = std::min((c->T + R - 2) / R + 1, c->max_pages);
  a.page_ctas = a.x.units * a.per_unit;
  const int64_t rows = q ? a.x.units * a.x.G * a.x.T : 0, per = (kThreads / 32) * kQRows;
  const int64_t grid = a.page_ctas + (rows + per - 1) / per;
  if (grid >= (1LL << 31)) return KVC_EINVAL;
  auto kernel = p->dtype == KVC_BF16 ? (p->d == 128 ? q8_append_kernel<__nv_bfloat16, 128> : q8_append_kernel<__nv_bfloat16, 64>)
                                     : (p->d == 128 ? q8_append_kernel<float, 128> : q8_append_kernel<float, 64>);
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

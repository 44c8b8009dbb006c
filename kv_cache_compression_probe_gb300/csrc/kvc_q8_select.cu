// kvc_q8_select: the pages a token of a KV head attends over, by a cheap score.
//
// A page's keys lie between its bounds lo and hi, feature by feature, so that
//   q . k <= sum_f max(q_f lo_f, q_f hi_f) = sum_f q+_f hi_f + q-_f lo_f
// for every key k of it (q+ and q- the positive and negative parts).  With q and the bounds as
// 8-bit integers the sum is an integer below 2^24: exact, so a selection does not depend on the
// order of a sum, and equal scores are equal.
#include "kvc_q8.cuh"

namespace {

using kvc::Q8Args;

constexpr int kThreads = 256, kWarps = kThreads / 32;

struct Q8Select {
  Q8Args x;
  const void* q;
  int32_t* sel;
  int n_sel, first, recent;
};

struct SelectSmem {
  uint32_t pos[8][32], neg[8][32];     // q+ and q- of a head, four features a word
  float top[8];                        // the head's largest |q|
  int count[2][kWarps];
};

// Sum of v over the block; `turn` alternates between calls, so one barrier is enough.
__device__ __forceinline__ int block_sum(int v, SelectSmem& sm, int& turn) {
  v = __reduce_add_sync(KVC_FULL_MASK, v);
  turn ^= 1;
  if ((threadIdx.x & 31) == 0) sm.count[turn][threadIdx.x >> 5] = v;
  __syncthreads();
  int t = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) t += sm.count[turn][i];
  return t;
}

// One CTA per (unit, token).
template <typename T, int D, int G>
__global__ void __launch_bounds__(kThreads) q8_select_kernel(const __grid_constant__ Q8Select a) {
  extern __shared__ uint32_t keys[];                   // order codes of the scores, a page each
  __shared__ SelectSmem sm;
  const Q8Args& x = a.x;
  kvcd::pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t u = blockIdx.x / x.T;
  const int t = (int)(blockIdx.x - u * x.T);
  const int64_t gu = kvcd::q8_unit_global(x, u);
  const int len = x.len_lh[gu], n = x.len_new[gu] - len;
  if (len < 0 || n < 0 || n > x.T || (int64_t)len + n > (int64_t)x.max_pages << x.shift) {
    if (t == 0 && tid == 0) kvcd::record_error(x.err, KVC_EDEVICE);
    return;
  }
  if (t >= n) return;
  int32_t* out = a.sel + blockIdx.x * (int64_t)a.n_sel;
  const int nb = ((len + t) >> x.shift) + 1;           // pages the token sees, its own the last
  if (nb <= a.n_sel) {
    for (int i = tid; i < a.n_sel; i += kThreads) out[i] = i < nb ? i : -1;
    return;
  }
  if (warp < G) {                                      // a head's row in 8-bit integers
    const T* q = static_cast<const T*>(a.q) + ((u * G + warp) * x.T + t) * D;
    float v[4], top = 0.f;
    if (lane < D / 4) {
      kvcd::VecLoad<T, 4>::ld(q + 4 * lane, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, fabsf(v[i]));
    }
    top = kvcd::warp_max(top);
    const float inv = top > 0.f ? __fmul_rn(127.f, __frcp_rn(top)) : 0.f;
    uint32_t p = 0, m = 0;
    if (lane < D / 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = min(max(__float2int_rn(__fmul_rn(v[i], inv)), -127), 127);
        p |= (uint32_t)(max(c, 0) & 255) << (8 * i);
        m |= (uint32_t)(min(c, 0) & 255) << (8 * i);
      }
      sm.pos[warp][lane] = p;
      sm.neg[warp][lane] = m;
    }
    if (lane == 0) sm.top[warp] = top;
  }
  __syncthreads();
  const int32_t* tab = x.table + gu * x.max_pages;
  bool bad = false;
  for (int b = tid; b < nb; b += kThreads) {
    if (b < a.first || b > nb - 1 - a.recent) {
      keys[b] = 0xffffffffu;
      continue;
    }
    const int page = __ldg(tab + b);
    if ((unsigned)page >= (unsigned)x.pages) {
      bad = true;
      keys[b] = 0;
      continue;
    }
    const uint4* bd = reinterpret_cast<const uint4*>(x.bounds + (int64_t)page * 2 * D);
    int acc[G];
#pragma unroll
    for (int g = 0; g < G; ++g) acc[g] = 0;
#pragma unroll 4
    for (int c = 0; c < D / 16; ++c) {
      const uint4 lo = __ldg(bd + c), hi = __ldg(bd + D / 16 + c);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const uint4 p = *reinterpret_cast<const uint4*>(&sm.pos[g][4 * c]);
        const uint4 m = *reinterpret_cast<const uint4*>(&sm.neg[g][4 * c]);
        acc[g] = __dp4a((int)p.x, (int)hi.x, __dp4a((int)p.y, (int)hi.y, __dp4a((int)p.z, (int)hi.z, __dp4a((int)p.w, (int)hi.w, acc[g]))));
        acc[g] = __dp4a((int)m.x, (int)lo.x, __dp4a((int)m.y, (int)lo.y, __dp4a((int)m.z, (int)lo.z, __dp4a((int)m.w, (int)lo.w, acc[g]))));
      }
    }
    const float s = __ldg(x.k_scale + page);
    float best = -INFINITY;
#pragma unroll
    for (int g = 0; g < G; ++g) best = fmaxf(best, __fmul_rn(__fmul_rn((float)acc[g], s), sm.top[g]));
    keys[b] = kvcd::float_key(best + 0.f);             // -0 counts as 0
  }
  if (__syncthreads_or(bad) && tid == 0) kvcd::record_error(x.err, KVC_EDEVICE);
  // The largest code that at least n_sel pages reach, bit by bit.
  int turn = 0;
  uint32_t cut = 0;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t trial = cut | 1u << bit;
    int mine = 0;
    for (int b = tid; b < nb; b += kThreads) mine += keys[b] >= trial;
    if (block_sum(mine, sm, turn) >= a.n_sel) cut = trial;
  }
  // Pages above it, and of those equal the first ones; thread i looks at a run of pages.
  const int per = (nb + kThreads - 1) / kThreads, b0 = min(nb, tid * per), b1 = min(nb, b0 + per);
  int above = 0, equal = 0;
  for (int b = b0; b < b1; ++b) {
    above += keys[b] > cut;
    equal += keys[b] == cut;
  }
  const int quota = a.n_sel - block_sum(above, sm, turn);   // of the equal ones
  int s1 = above, s2 = equal;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v1 = __shfl_up_sync(KVC_FULL_MASK, s1, o), v2 = __shfl_up_sync(KVC_FULL_MASK, s2, o);
    if (lane >= o) { s1 += v1; s2 += v2; }
  }
  __syncthreads();
  if (lane == 31) { sm.count[0][warp] = s1; sm.count[1][warp] = s2; }
  __syncthreads();
  s1 -= above;
  s2 -= equal;
  for (int w = 0; w < warp; ++w) { s1 += sm.count[0][w]; s2 += sm.count[1][w]; }
  for (int b = b0; b < b1; ++b) {
    const bool gt = keys[b] > cut, eq = keys[b] == cut;
    if (gt || (eq && s2 < quota)) out[s1 + min(s2, quota)] = b;
    s1 += gt;
    s2 += eq;
  }
}

template <typename T, int D>
auto select_kernel(int G) {
  return G == 1 ? q8_select_kernel<T, D, 1> : G == 2 ? q8_select_kernel<T, D, 2>
       : G == 4 ? q8_select_kernel<T, D, 4> : q8_select_kernel<T, D, 8>;
}

constexpr int kMaxPages = 32768;       // their order codes fit a CTA's shared memory

}  // namespace

extern "C" int kvc_q8_select(const kvc_params* p, const kvc_chunk* c, const kvc_q8* x, const void* q,
                             const int32_t* len_lh, const int32_t* len_new, int32_t n_sel, int32_t first,
                             int32_t recent, int32_t* sel, void* stream) {
  const int st = kvc::q8_check(p, c, x);
  if (st != KVC_OK) return st;
  if (!q || !len_lh || !len_new || !sel || !x->bounds || kvc::q8_misaligned(q, 16)) return KVC_EINVAL;
  if (n_sel < 1 || n_sel > kMaxPages || first < 0 || recent < 1 || first > n_sel - recent) return KVC_EINVAL;
  if (c->max_pages > kMaxPages) return KVC_EINVAL;
  Q8Select a = {};
  kvc::q8_fill(a.x, p, c, x);
  if (!a.x.err) return KVC_ECUDA;
  a.x.len_lh = len_lh;
  a.x.len_new = len_new;
  a.q = q;
  a.sel = sel;
  a.n_sel = n_sel;
  a.first = first;
  a.recent = recent;
  const int64_t grid = a.x.units * c->T;
  if (grid >= (1LL << 31)) return KVC_EINVAL;
  const bool bf = p->dtype == KVC_BF16;
  auto kernel = p->d == 128 ? (bf ? select_kernel<__nv_bfloat16, 128>(p->G) : select_kernel<float, 128>(p->G))
                            : (bf ? select_kernel<__nv_bfloat16, 64>(p->G) : select_kernel<float, 64>(p->G));
  const size_t smem = (size_t)c->max_pages * sizeof(uint32_t);
  if (smem > (40u << 10)) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxPages * 4);
    if (e != cudaSuccess) return kvc::cuda_status(e);
  }
  kvc::count_launch();
  return kvc::cuda_status(kvc::chunk_launch(kernel, dim3((unsigned)grid), dim3(kThreads), smem,
                                            static_cast<cudaStream_t>(stream), a));
}

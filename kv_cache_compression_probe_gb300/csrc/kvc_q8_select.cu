// kvc_q8_select: the pages a token of a KV head attends over, by a cheap score.
//
// A page's keys lie between its bounds lo and hi, feature by feature, so that
//   q . k <= sum_f max(q_f lo_f, q_f hi_f) = sum_f q+_f hi_f + q-_f lo_f
// for every key k of it (q+ and q- the positive and negative parts).  With q and the bounds as
// 8-bit integers the sum is an integer below 2^24: exact, so a selection does not depend on the
// order of a sum, and equal scores are equal.
//
// The sums are products of the tensor cores, 16 pages x 8 query rows a time (rows: G heads of one
// or more tokens).  The integers go as fp16, which holds them exactly, and every partial sum is an integer
// below 2^24, which fp32 holds: exact as well, and 4 times as fast here as the 8-bit integer form (8 cycles a 16 x 8 x 16
// product and scheduler against 66 for 16 x 8 x 32).  A product's 16 inner positions may stand for any features, as long as
// both operands agree, so a lane takes whole 16-byte pieces of the bounds.  The scores' order codes stay in shared
// memory, where a warp per token (for a single token over many pages the whole CTA) looks for the n_sel-th largest by
// halving the range of codes; scores are spread over it, so about 10 steps are enough as a rule.
// Measured (d 128, G 4): one token over 256 caches of 512 pages 10.9 us (34 MB of bounds, 3 TB/s: a chain of loads, the
// scores, the search), 300 tokens over 8 caches of 512 pages 19.5 us (instructions: issue slots 48%).
#include <algorithm>

#include "kvc_q8.cuh"

namespace {

using kvc::Q8Args;

constexpr int kThreads = 256, kWarps = kThreads / 32;

constexpr int kWarpPages = 640;        // pages whose codes a warp keeps in registers; a single token over more is the whole CTA's
                                       // (512 pages: a warp 11.7 us, the CTA 13.8)

struct Q8Select {
  Q8Args x;
  const void* q;
  int32_t* sel;
  int n_sel, first, recent;
  int tt, tiles;                       // tokens of a CTA, CTAs of a unit
};

template <int D, int NT>
struct SelectSmem {
  uint2 q[NT][D / 8][32];              // the rows' q+ (first half) and q- as operands: a lane's words of a product
  float top[NT * 8];                   // the rows' largest |q|
  int count[2][kWarps];
  uint32_t ends[2];
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint2 b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y));
}
// Four signed bytes as fp16 pairs: with the sign bit turned over a byte is x + 128, the low bits of the fp16
// number 1024 + 128 + x.
__device__ __forceinline__ void bytes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  w ^= 0x80808080u;
  const uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
}

// Order code of a score: -0 counts as 0, and what is no number as the least, so that kAlways is the code of the
// pages that are always in alone (the search relies on there being n_sel of them at most).
constexpr uint32_t kAlways = 0xffffffffu;
__device__ __forceinline__ uint32_t order_of(float s) { return s == s ? kvcd::float_key(s + 0.f) : 0; }

// Sum of v over the block; `turn` alternates between calls, so one barrier is enough.
__device__ __forceinline__ int block_sum(int v, int (&count)[2][kWarps], int& turn) {
  v = __reduce_add_sync(KVC_FULL_MASK, v);
  turn ^= 1;
  if ((threadIdx.x & 31) == 0) count[turn][threadIdx.x >> 5] = v;
  __syncthreads();
  int t = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) t += count[turn][i];
  return t;
}

// The codes of a warp's pages, lane i those of pages i, i + 32, ..: in registers where they are at most 32 kRegs
// (0: in shared memory).  Pages beyond nb count as code 0.
template <int kRegs>
struct WarpKeys {
  uint32_t reg[kRegs];
  __device__ __forceinline__ WarpKeys(const uint32_t* keys, int nb) {
#pragma unroll
    for (int i = 0; i < kRegs; ++i) reg[i] = (int)(threadIdx.x & 31) + 32 * i < nb ? keys[(threadIdx.x & 31) + 32 * i] : 0;
  }
  template <class F>
  __device__ __forceinline__ void each(F f) const {
#pragma unroll
    for (int i = 0; i < kRegs; ++i) f((int)(threadIdx.x & 31) + 32 * i, reg[i]);
  }
};
template <>
struct WarpKeys<0> {
  const uint32_t* keys;
  int nb;
  __device__ __forceinline__ WarpKeys(const uint32_t* k, int n) : keys(k), nb(n) {}
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    for (int b = threadIdx.x & 31; b < (nb + 31 & ~31); b += 32) f(b, b < nb ? keys[b] : 0);
  }
};

// The n_sel pages of largest code, by one warp, in ascending order.
template <int kRegs>
__device__ __forceinline__ void pick_by_warp(const uint32_t* keys, int nb, int n_sel, int32_t* out) {
  const int lane = threadIdx.x & 31;
  const WarpKeys<kRegs> mine(keys, nb);
  uint32_t cut = 0xffffffffu, top = 0;                 // least and largest code of the pages that need not be in
  mine.each([&](int b, uint32_t key) {
    cut = min(cut, b < nb ? key : 0xffffffffu);
    top = max(top, key == kAlways ? 0 : key);
  });
  cut = __reduce_min_sync(KVC_FULL_MASK, cut);
  top = max(cut, __reduce_max_sync(KVC_FULL_MASK, top));
  while (cut < top) {                                  // cut: the largest code so far that n_sel pages reach; none above top is
    const uint32_t trial = cut + (top - cut + 1) / 2;
    int reach = 0;
    mine.each([&](int b, uint32_t key) { reach += key >= trial; });
    reach = __reduce_add_sync(KVC_FULL_MASK, reach);
    if (reach >= n_sel) cut = trial;
    else top = trial - 1;
    if (reach == n_sel) break;
  }
  int above = 0;
  mine.each([&](int b, uint32_t key) { above += b < nb && key > cut; });
  int quota = n_sel - __reduce_add_sync(KVC_FULL_MASK, above), at = 0;   // of those equal to it: the first ones
  const uint32_t before = (1u << lane) - 1;
  mine.each([&](int b, uint32_t key) {
    const uint32_t eq = __ballot_sync(KVC_FULL_MASK, b < nb && key == cut);
    const bool take = b < nb && (key > cut || (key == cut && __popc(eq & before) < quota));
    const uint32_t taken = __ballot_sync(KVC_FULL_MASK, take);
    if (take) out[at + __popc(taken & before)] = b;
    at += __popc(taken);
    quota -= min(quota, __popc(eq));
  });
}

// The same by the whole block; thread i looks at a run of pages.
__device__ __forceinline__ void pick_by_block(const uint32_t* keys, int nb, int n_sel, int32_t* out,
                                              int (&count)[2][kWarps], uint32_t (&ends)[2]) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int turn = 0;
  uint32_t cut = 0xffffffffu, top = 0;
  for (int b = tid; b < nb; b += kThreads) {
    const uint32_t key = keys[b];
    cut = min(cut, key);
    top = max(top, key == kAlways ? 0 : key);
  }
  if (tid == 0) { ends[0] = 0xffffffffu; ends[1] = 0; }
  __syncthreads();
  cut = __reduce_min_sync(KVC_FULL_MASK, cut);
  top = __reduce_max_sync(KVC_FULL_MASK, top);
  if (lane == 0) { atomicMin(&ends[0], cut); atomicMax(&ends[1], top); }
  __syncthreads();
  cut = ends[0];
  top = max(cut, ends[1]);
  while (cut < top) {
    const uint32_t trial = cut + (top - cut + 1) / 2;
    int mine = 0;
    for (int b = tid; b < nb; b += kThreads) mine += keys[b] >= trial;
    mine = block_sum(mine, count, turn);
    if (mine >= n_sel) cut = trial;
    else top = trial - 1;
    if (mine == n_sel) break;
  }
  const int per = (nb + kThreads - 1) / kThreads, b0 = min(nb, tid * per), b1 = min(nb, b0 + per);
  int above = 0, equal = 0;
  for (int b = b0; b < b1; ++b) {
    above += keys[b] > cut;
    equal += keys[b] == cut;
  }
  const int quota = n_sel - block_sum(above, count, turn);    // of the equal ones
  int s1 = above, s2 = equal;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v1 = __shfl_up_sync(KVC_FULL_MASK, s1, o), v2 = __shfl_up_sync(KVC_FULL_MASK, s2, o);
    if (lane >= o) { s1 += v1; s2 += v2; }
  }
  __syncthreads();
  if (lane == 31) { count[0][warp] = s1; count[1][warp] = s2; }
  __syncthreads();
  s1 -= above;
  s2 -= equal;
  for (int w = 0; w < warp; ++w) { s1 += count[0][w]; s2 += count[1][w]; }
  for (int b = b0; b < b1; ++b) {
    const bool gt = keys[b] > cut, eq = keys[b] == cut;
    if (gt || (eq && s2 < quota)) out[s1 + min(s2, quota)] = b;
    s1 += gt;
    s2 += eq;
  }
}

// One CTA per (unit, tt tokens); query row r is head r % G of token r / G.
template <typename T, int D, int G, int NT>
__global__ void __launch_bounds__(kThreads, 2) q8_select_kernel(const __grid_constant__ Q8Select a) {
  constexpr int kH = D / 64, kS = D / 16;              // 16-byte pieces of a row per lane, products for lo (and for hi)
  extern __shared__ uint32_t keys[];                   // [tt][max_pages] order codes of the scores
  __shared__ SelectSmem<D, NT> sm;
  const Q8Args& x = a.x;
  kvcd::pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int64_t u = blockIdx.x / a.tiles;
  const int t0 = (int)(blockIdx.x - u * a.tiles) * a.tt;
  const int64_t gu = kvcd::q8_unit_global(x, u);
  const int len = x.len_lh[gu], n = x.len_new[gu] - len;
  if (len < 0 || n < 0 || n > x.T || (int64_t)len + n > (int64_t)x.max_pages << x.shift) {
    if (t0 == 0 && tid == 0) kvcd::record_error(x.err, KVC_EDEVICE);
    return;
  }
  const int tokens = min(a.tt, n - t0);
  if (tokens <= 0) return;
  int32_t* out = a.sel + (u * x.T + t0) * a.n_sel;
  const int most = ((len + t0 + tokens - 1) >> x.shift) + 1;   // pages that the last token sees
  if (most > a.n_sel) {
    const int32_t* tab = x.table + gu * x.max_pages;
    // ---- the first pages' bounds are on their way while the rows become integers
    struct Fetched {
      uint4 lo[2][kH], hi[2][kH];
      float scale[2];
    };
    bool bad = false;
    auto fetch = [&](int p0) {
      Fetched f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int b = p0 + g + 8 * j;
        int page = b < most ? __ldg(tab + b) : 0;
        if ((unsigned)page >= (unsigned)x.pages) {
          bad = true;
          page = 0;
        }
        const uint4* p = reinterpret_cast<const uint4*>(x.bounds + (int64_t)page * 2 * D) + c;
#pragma unroll
        for (int h = 0; h < kH; ++h) {
          f.lo[j][h] = p[4 * h];
          f.hi[j][h] = p[D / 16 + 4 * h];
        }
        f.scale[j] = x.k_scale[page];
      }
      return f;
    };
    Fetched next = fetch(warp * 16);
    float v[NT][4];                                    // this warp's rows warp, warp + 8, ..
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int r = warp + j * kWarps, tok = r / G;
      v[j][0] = v[j][1] = v[j][2] = v[j][3] = 0.f;
      if (tok < tokens && lane < D / 4)
        kvcd::load4(static_cast<const T*>(a.q) + ((u * G + r % G) * x.T + t0 + tok) * D + 4 * lane, v[j]);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int r = warp + j * kWarps;
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, fabsf(v[j][i]));
      top = kvcd::warp_max(top);
      const float inv = top > 0.f ? __fmul_rn(127.f, __frcp_rn(top)) : 0.f;
      uint32_t p = 0, m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = min(max(__float2int_rn(__fmul_rn(v[j][i], inv)), -127), 127);
        p |= (uint32_t)(max(k, 0) & 255) << (8 * i);
        m |= (uint32_t)(min(k, 0) & 255) << (8 * i);
      }
      if (lane < D / 4) {                              // word `lane`: piece h, lane c of the operand, word i of it
        const int h = lane / 16, cc = (lane % 16) / 4, i = lane % 4;
        uint2 y;
        bytes_f16(p, y.x, y.y);
        sm.q[r / 8][4 * h + i][(r % 8) * 4 + cc] = y;
        bytes_f16(m, y.x, y.y);
        sm.q[r / 8][kS + 4 * h + i][(r % 8) * 4 + cc] = y;
      }
      if (lane == 0) sm.top[r] = top;
    }
    __syncthreads();
    for (int p0 = warp * 16; p0 < most; p0 += kWarps * 16) {
      const Fetched f = next;
      if (p0 + kWarps * 16 < most) next = fetch(p0 + kWarps * 16);
      float acc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
#pragma unroll
      for (int v = 0; v < 2; ++v)
#pragma unroll
        for (int h = 0; h < kH; ++h) {
          const uint4 r0 = v ? f.lo[0][h] : f.hi[0][h], r1 = v ? f.lo[1][h] : f.hi[1][h];
          const uint32_t wa[4] = {r0.x, r0.y, r0.z, r0.w}, wb[4] = {r1.x, r1.y, r1.z, r1.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t a0, a1, a2, a3;
            bytes_f16(wa[i], a0, a2);
            bytes_f16(wb[i], a1, a3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(acc[nt], a0, a1, a2, a3, sm.q[nt][v * kS + 4 * h + i][lane]);
          }
        }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int b = p0 + g + 8 * j;
          float s0 = __fmul_rn(__fmul_rn(acc[nt][2 * j], f.scale[j]), sm.top[nt * 8 + 2 * c]);
          float s1 = __fmul_rn(__fmul_rn(acc[nt][2 * j + 1], f.scale[j]), sm.top[nt * 8 + 2 * c + 1]);
          if (G > 1) s0 = fmaxf(s0, s1);
          if (G > 2) s0 = fmaxf(s0, __shfl_xor_sync(KVC_FULL_MASK, s0, 1));
          if (G > 4) s0 = fmaxf(s0, __shfl_xor_sync(KVC_FULL_MASK, s0, 2));
          auto put = [&](int tok, float s) {
            const int own = (len + t0 + tok) >> x.shift;
            if (tok < tokens && b <= own)
              keys[tok * x.max_pages + b] = b < a.first || b > own - a.recent ? kAlways : order_of(s);
          };
          const int tok = (nt * 8 + 2 * c) / G;
          if (G == 1) {
            put(tok, s0);
            put(tok + 1, s1);
          } else if (2 * c % G == 0) {
            put(tok, s0);
          }
        }
    }
    if (bad) kvcd::record_error(x.err, KVC_EDEVICE);
    __syncthreads();
  }
  if (tokens == 1 && most > max(a.n_sel, kWarpPages)) {
    pick_by_block(keys, most, a.n_sel, out, sm.count, sm.ends);
  } else {
    for (int tok = warp; tok < tokens; tok += kWarps) {
      const int nb = ((len + t0 + tok) >> x.shift) + 1;
      int32_t* to = out + tok * (int64_t)a.n_sel;
      const uint32_t* mine = keys + tok * x.max_pages;
      if (nb > a.n_sel && nb <= 256) pick_by_warp<8>(mine, nb, a.n_sel, to);
      else if (nb > a.n_sel && nb <= kWarpPages) pick_by_warp<kWarpPages / 32>(mine, nb, a.n_sel, to);
      else if (nb > a.n_sel) pick_by_warp<0>(mine, nb, a.n_sel, to);
      else
        for (int i = lane; i < a.n_sel; i += 32) to[i] = i < nb ? i : -1;
    }
  }
  kvcd::pdl_trigger();
}

template <typename T, int D, int NT>
auto select_kernel(int G) {
  return G == 1 ? q8_select_kernel<T, D, 1, NT> : G == 2 ? q8_select_kernel<T, D, 2, NT>
       : G == 4 ? q8_select_kernel<T, D, 4, NT> : q8_select_kernel<T, D, 8, NT>;
}
template <int NT>
auto select_kernel(const kvc_params* p) {
  const bool bf = p->dtype == KVC_BF16;
  return p->d == 128 ? (bf ? select_kernel<__nv_bfloat16, 128, NT>(p->G) : select_kernel<float, 128, NT>(p->G))
                     : (bf ? select_kernel<__nv_bfloat16, 64, NT>(p->G) : select_kernel<float, 64, NT>(p->G));
}

constexpr int kMaxPages = 32768;       // their order codes fit a CTA's shared memory
constexpr int kKeyBytes = 64 << 10;    // and what several tokens' codes may take of it

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
  // Tokens of a CTA: they share the reading of the bounds, and their codes share its memory.
  const int fit = kKeyBytes / (c->max_pages * (int)sizeof(uint32_t));
  const int nt = c->T * p->G > 8 && fit * p->G > 8 ? 4 : 1;
  a.tt = std::max(1, std::min({c->T, nt * 8 / p->G, fit}));
  a.tiles = (c->T + a.tt - 1) / a.tt;
  const int64_t grid = a.x.units * a.tiles;
  if (grid >= (1LL << 31)) return KVC_EINVAL;
  auto kernel = nt == 4 ? select_kernel<4>(p) : select_kernel<1>(p);
  const size_t smem = (size_t)a.tt * c->max_pages * sizeof(uint32_t);
  if (smem > (30u << 10)) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxPages * 4);
    if (e != cudaSuccess) return kvc::cuda_status(e);
  }
  kvc::count_launch();
  return kvc::cuda_status(kvc::chunk_launch(kernel, dim3((unsigned)grid), dim3(kThreads), smem,
                                            static_cast<cudaStream_t>(stream), a));
}

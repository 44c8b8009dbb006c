// kvc_mass_evict: per-(b,l,h) eviction by accumulated attention mass.
//
// One CTA per (b,l,h) finds the smallest key that stays (a radix select over
// the 32-bit order code of the mass; protected entries have the largest code)
// and lists the moves: evicted entries below the new length ("holes") take the
// staying entries at or above it, both in index order.  A second kernel moves
// the rows.  Moving only those rows, instead of compacting the cache, keeps the
// traffic at twice the moved rows; the row order stops following the positions,
// so protection goes by position and not by index.
#include <algorithm>

#include "kvc_chunk.cuh"
#include "kvc_internal.h"

namespace {

using kvc::ChunkArgs;

constexpr int kPlanThreads = 1024;
constexpr int kMoveRows = 32;          // row moves per CTA and turn

struct EvictArgs {
  ChunkArgs a;                         // mass, Kp, Vp, logm, pos, len_lh, off_lh, len_out, pages
  const int32_t* keep_lh;
  const float* pos_next;
  float recent;
  int max_len, cols;
  int2* moves;                         // [units, cols] (hole, mover) entry indices
  int32_t* n_moves;                    // [units]
  int vec;                             // 16-byte vectors of a K or V row
};

// Order code of a mass: larger mass, larger code; NaN below everything (0) and
// protected entries above everything.
__device__ __forceinline__ uint32_t mass_code(float m, bool is_protected) {
  if (is_protected) return 0xffffffffu;
  if (m != m) return 0u;
  return kvcd::float_key(m == 0.f ? 0.f : m);          // -0 is 0; codes 0x007fffff (-inf) .. 0xff800000 (inf)
}

// Exclusive prefix of `v` over the block; returns the total.
__device__ __forceinline__ int block_prefix(int v, int* s_warp, int& excl) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(KVC_FULL_MASK, incl, o);
    if (lane >= o) incl += x;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(KVC_FULL_MASK, w, o);
      if (lane >= o) w += x;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  excl = incl - v + (warp > 0 ? s_warp[warp - 1] : 0);
  return s_warp[31];
}

__global__ void __launch_bounds__(kPlanThreads) mass_plan_kernel(EvictArgs ea) {
  const ChunkArgs& a = ea.a;
  __shared__ uint32_t hist[256];
  __shared__ int s_warp[32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_rem, s_ok;
  kvcd::pdl_trigger();
  kvcd::pdl_wait();
  const int64_t u = blockIdx.x;
  const int64_t gu = kvcd::unit_global(a, u);
  const int tid = threadIdx.x;
  const int len = a.len_lh[gu];
  const int64_t off = a.page_table ? 0 : a.off_lh[gu];
  if (tid == 0) s_ok = len >= 0 && len <= ea.max_len && len <= a.packed_rows && off >= 0 &&
                       (a.page_table || off + len <= a.packed_rows);
  __syncthreads();
  bool ok = s_ok != 0;
  if (ok && a.page_table) {
    const int need = (int)(((int64_t)len + (1 << a.page_shift) - 1) >> a.page_shift);
    ok = need <= a.max_pages;
    if (ok) {
      const int32_t* tab = a.page_table + gu * a.max_pages;
      const int64_t pages = a.packed_rows >> a.page_shift;
      for (int i = tid; i < need; i += kPlanThreads) ok &= tab[i] >= 0 && tab[i] < pages;
    }
  }
  if (!__syncthreads_and(ok)) {
    if (tid == 0) {
      kvcd::record_error(a.err, KVC_EDEVICE);
      ea.n_moves[u] = 0;
      a.len_out[gu] = len;
    }
    return;
  }
  const kvcd::RowMap rows = kvcd::row_map(a, u, off);
  const float safe = ea.pos_next[u / a.per_seq] - ea.recent;
  auto code = [&](int e) {
    const int64_t row = rows(e);
    return mass_code(a.mass[row], a.pos[row] >= safe);
  };
  // every thread owns a contiguous range of entries, so index order is thread order
  const int per = (len + kPlanThreads - 1) / kPlanThreads;
  const int i0 = min(len, tid * per), i1 = min(len, i0 + per);
  int mine = 0, excl;
  for (int e = i0; e < i1; ++e) mine += code(e) == 0xffffffffu;
  const int n_protected = block_prefix(mine, s_warp, excl);
  const int B = min(len, max(max(0, ea.keep_lh[gu]), n_protected));
  if (tid == 0) { s_prefix = 0; s_rem = B; }
  // the B-th largest code, 8 bits at a time (not needed when all or none stay)
  for (int shift = 24; shift >= 0 && B > 0 && B < len; shift -= 8) {
    for (int i = tid; i < 256; i += kPlanThreads) hist[i] = 0;
    __syncthreads();
    const uint32_t pre = s_prefix, mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
    for (int e = tid; e < len; e += kPlanThreads) {
      const uint32_t k = code(e);
      if ((k & mask) == pre) atomicAdd(&hist[(k >> shift) & 255], 1u);
    }
    __syncthreads();
    if (tid < 32) {                                    // lane: digits 255-8l .. 248-8l, descending
      int cnt[8], sum = 0;
#pragma unroll
      for (int x = 0; x < 8; ++x) { cnt[x] = (int)hist[255 - 8 * tid - x]; sum += cnt[x]; }
      int incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(KVC_FULL_MASK, incl, o);
        if (tid >= o) incl += v;
      }
      const int rem0 = s_rem;
      const unsigned hit = __ballot_sync(KVC_FULL_MASK, incl >= rem0);
      if (tid == __ffs(hit) - 1) {
        int rem = rem0 - (incl - sum), x = 0;
        while (x < 7 && cnt[x] < rem) rem -= cnt[x++];
        s_prefix = pre | ((uint32_t)(255 - 8 * tid - x) << shift);
        s_rem = rem;
      }
    }
    __syncthreads();
  }
  __syncthreads();
  const uint32_t cut = s_prefix;
  const int rem = s_rem;                               // how many of the entries at the cut stay
  const bool all = B >= len, none = B == 0;
  int ties = 0;
  if (!all && !none)
    for (int e = i0; e < i1; ++e) ties += code(e) == cut;
  int tie0;
  block_prefix(ties, s_warp, tie0);
  // holes (evicted, below B) and movers (staying, at or above B) before this thread's range
  int nh = 0, nm = 0, tie = tie0;
  auto stays = [&](int e) {
    if (all || none) return all;
    const uint32_t k = code(e);
    return k > cut || (k == cut && tie++ < rem);
  };
  for (int e = i0; e < i1; ++e) {
    const bool s = stays(e);
    if (e < B) nh += !s; else nm += s;
  }
  int h0, m0;
  const int holes = block_prefix(nh, s_warp, h0);
  block_prefix(nm, s_warp, m0);
  int2* mv = ea.moves + u * ea.cols;
  tie = tie0;
  for (int e = i0; e < i1; ++e) {
    const bool s = stays(e);
    if (e < B && !s) mv[h0++].x = e;
    else if (e >= B && s) mv[m0++].y = e;
  }
  if (tid == 0) {
    ea.n_moves[u] = holes;
    a.len_out[gu] = B;
  }
}

__global__ void __launch_bounds__(256) mass_move_kernel(EvictArgs ea) {
  const ChunkArgs& a = ea.a;
  kvcd::pdl_trigger();
  kvcd::pdl_wait();
  const int64_t u = blockIdx.y;
  const int n = ea.n_moves[u];
  const int64_t off = a.page_table ? 0 : a.off_lh[kvcd::unit_global(a, u)];
  const kvcd::RowMap rows = kvcd::row_map(a, u, off);
  const int2* mv = ea.moves + u * ea.cols;
  const int vec = ea.vec;
  uint4* K = static_cast<uint4*>(a.Kp);
  uint4* V = static_cast<uint4*>(a.Vp);
  for (int j0 = blockIdx.x * kMoveRows; j0 < n; j0 += gridDim.x * kMoveRows) {
    const int cnt = min(kMoveRows, n - j0);
    for (int i = threadIdx.x; i < cnt * vec; i += blockDim.x) {
      const int2 m = mv[j0 + i / vec];
      const int64_t to = rows(m.x) * vec + i % vec, from = rows(m.y) * vec + i % vec;
      const uint4 k = K[from], v = V[from];
      K[to] = k;
      V[to] = v;
    }
    for (int i = threadIdx.x; i < cnt; i += blockDim.x) {
      const int2 m = mv[j0 + i];
      const int64_t to = rows(m.x), from = rows(m.y);
      a.logm[to] = a.logm[from];
      a.pos[to] = a.pos[from];
      a.mass[to] = a.mass[from];
    }
  }
}

struct EvictLayout {
  size_t moves, count, total;
};
EvictLayout evict_layout(const kvc_params* p, const kvc_chunk* c, int max_len) {
  const size_t units = (size_t)p->B * p->H * (c->layer_end - c->layer_begin);
  EvictLayout w;
  w.moves = 0;
  w.count = kvc::align256(units * ((size_t)max_len / 2 + 1) * sizeof(int2));
  w.total = w.count + kvc::align256(units * sizeof(int32_t));
  return w;
}

}  // namespace

extern "C" size_t kvc_mass_evict_workspace_bytes(const kvc_params* p, const kvc_chunk* c, int32_t max_len) {
  if (kvc::chunk_check(p, c) != KVC_OK || max_len < 1) return 0;
  return evict_layout(p, c, max_len).total;
}

extern "C" int kvc_mass_evict(const kvc_params* p, const kvc_chunk* c, float* mass, const int32_t* keep_lh,
                              int32_t recent, const float* pos_next, void* Kp, void* Vp, float* logm,
                              float* pos, const int32_t* len_lh, const int64_t* off_lh, int32_t* len_out,
                              int32_t max_len, void* workspace, size_t ws_bytes, void* stream) {
  int st = kvc::chunk_check(p, c);
  if (st != KVC_OK) return st;
  if (!mass || !keep_lh || !pos_next || !Kp || !Vp || !logm || !pos || !len_lh || !len_out || recent < 0 ||
      max_len < 1 || (!off_lh && c->page_rows == 0))
    return KVC_EINVAL;
  if ((reinterpret_cast<uintptr_t>(Kp) & 15) || (reinterpret_cast<uintptr_t>(Vp) & 15)) return KVC_EINVAL;
  EvictArgs ea = {};
  kvc::chunk_fill(ea.a, p, c);
  if (ea.a.units > 65535) return KVC_EINVAL;           // grid.y of the move kernel
  const EvictLayout w = evict_layout(p, c, max_len);
  if (!workspace || ws_bytes < w.total || (reinterpret_cast<uintptr_t>(workspace) & 255)) return KVC_EWORKSPACE;
  ea.a.err = kvc::err_word();
  const int sms = kvc::sm_count();
  if (!ea.a.err || sms <= 0) return KVC_ECUDA;
  char* ws = static_cast<char*>(workspace);
  ea.moves = reinterpret_cast<int2*>(ws + w.moves);
  ea.n_moves = reinterpret_cast<int32_t*>(ws + w.count);
  ea.a.mass = mass; ea.a.Kp = Kp; ea.a.Vp = Vp; ea.a.logm = logm; ea.a.pos = pos;
  ea.a.len_lh = len_lh; ea.a.off_lh = off_lh; ea.a.len_out = len_out;
  ea.keep_lh = keep_lh; ea.pos_next = pos_next; ea.recent = (float)recent;
  ea.max_len = max_len;
  ea.cols = max_len / 2 + 1;
  ea.vec = p->d * (p->dtype == KVC_BF16 ? 2 : 4) / 16;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = kvc::chunk_launch(mass_plan_kernel, dim3((unsigned)ea.a.units), dim3(kPlanThreads), 0, s, ea);
  if (e != cudaSuccess) return kvc::cuda_status(e);
  kvc::count_launch(2);
  // at most max_len / 2 moves per unit, usually few: about 8 CTAs per SM stride over them
  const int64_t need = (ea.cols + kMoveRows - 1) / kMoveRows;
  const int64_t x = std::max<int64_t>(1, std::min<int64_t>(need, (8LL * sms + ea.a.units - 1) / ea.a.units));
  e = kvc::chunk_launch(mass_move_kernel, dim3((unsigned)x, (unsigned)ea.a.units), dim3(256), 0, s, ea);
  return kvc::cuda_status(e);
}

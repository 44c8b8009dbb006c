// kvc_chunk_attn and kvc_chunk_mass: attention of a chunk of new tokens over the
// packed cache, and the attention weight every entry received from it.  This
// file holds the host entries, the prepare and combine kernels, and the fp32
// kernels.
//
// fp32 kernels: 256 threads hold a tile of 64 (or, for few rows, 16) query rows
// and 64 entries.  Query rows, entries' keys and values are staged in shared
// memory as fp32; thread (ty, tx) forms the scores of rows ty*R.. and entries
// tx + 16 j, so the 16 lanes of a row share its maximum and sum by shuffles.
// fp32 has no tensor-core form of full precision.  A tile is staged between two barriers, so loads
// and arithmetic take turns: 512 tokens over 3584 entries (8 KV heads, G 4, d 128) take 955 us, 34
// TFLOP/s with the FMA pipe 47% busy, and one token over 64 caches of 4096 entries 231 us, 1.2 TB/s.
// Small calls are bound by the launches (33 tokens over 512 entries, 2 KV heads, d 64: 19 us).
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "kvc_chunk_tc.cuh"
#include "kvc_internal.h"

namespace {

using kvc::ChunkArgs;
using kvc::ChunkSeg;
using kvc::ChunkUnit;

constexpr int kKeys = 64;              // entries per tile of the fp32 kernels
constexpr int kSimtThreads = 256;

// ---------------------------------------------------------------- prepare
// One warp per (unit, group of 8 new tokens; mass: one per unit): checks the unit, appends the group's
// keys and values (kAppend) and writes the unit's record.  The rows to append are
// fetched before anything is known about the unit, so that their latency and that
// of the checks overlap.
constexpr int kPrepTok = 8;
constexpr int kPrepWarps = 4;

template <typename T, int D, bool kAppend>
__global__ void __launch_bounds__(32 * kPrepWarps) chunk_prepare_kernel(ChunkArgs a, int groups) {
  constexpr int kVec = D * (int)sizeof(T) / 16;        // 16-byte vectors of a row
  constexpr int kPer = kPrepTok * kVec / 32;           // vectors of K (and of V) per lane
  kvcd::pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * kPrepWarps + (threadIdx.x >> 5);
  const int64_t u = w / groups;
  const int g = (int)(w - u * groups);
  kvcd::pdl_wait();
  if (u >= a.units) return;
  const int b = (int)(u / a.per_seq), t0 = g * kPrepTok;
  uint4 kx[kPer], vx[kPer];
  if (kAppend) {
    const uint4* kn = reinterpret_cast<const uint4*>(static_cast<const T*>(a.k_new) + u * a.T * D);
    const uint4* vn = reinterpret_cast<const uint4*>(static_cast<const T*>(a.v_new) + u * a.T * D);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int at = t0 * kVec + lane + 32 * i;
      if (at < a.T * kVec) { kx[i] = __ldg(kn + at); vx[i] = __ldg(vn + at); }
    }
  }
  const int64_t gu = kvcd::unit_global(a, u);
  const int len = a.len_lh[gu];
  const int n = a.n_new ? a.n_new[b] : a.T;
  const int64_t off = a.page_table ? 0 : a.off_lh[gu];
  const int cap = a.cap_lh ? a.cap_lh[gu] : INT_MAX;
  // Mass: the next (b,l,h)'s first row and entries.  A unit that attention skipped for want of
  // capacity would reach into them.
  int64_t next_off = -1;
  int next_has = 0;
  if (!kAppend && !a.page_table && gu + 1 < a.units / a.per_seq * (a.lh_span + a.lh_gap)) {
    next_off = a.off_lh[gu + 1];
    next_has = max(a.len_lh[gu + 1], a.n_new ? a.n_new[(gu + 1) / (a.lh_span + a.lh_gap)] : a.T);
  }
  const float pos0 = kAppend ? a.pos_new[b] : 0.f;
  int bad = KVC_OK;
  if (len < 0 || n < 0 || n > a.T || off < 0 || (int64_t)len + n > a.packed_rows) bad = KVC_EDEVICE;
  else if (!a.page_table && !kvc::rows_fit(off, (int64_t)len + n, a.packed_rows)) bad = KVC_EDEVICE;
  else if ((int64_t)len + n > cap) bad = KVC_ECAPACITY;
  else if (next_off > off && off + len + n > next_off && next_has > 0) bad = KVC_ECAPACITY;
  else if (a.page_table) {
    const int need = (int)(((int64_t)len + n + (1 << a.page_shift) - 1) >> a.page_shift);
    if (need > a.max_pages) {
      bad = KVC_EDEVICE;
    } else {
      const int32_t* tab = a.page_table + gu * a.max_pages;
      const int64_t pages = a.packed_rows >> a.page_shift;
      bool ok = true;
#pragma unroll 4
      for (int i = lane; i < need; i += 32) {
        const int page = __ldg(tab + i);
        ok &= page >= 0 && page < pages;
      }
      if (!__all_sync(KVC_FULL_MASK, ok)) bad = KVC_EDEVICE;
    }
  }
  if (g == 0 && lane == 0) {
    if (bad != KVC_OK) kvcd::record_error(a.err, bad);
    kvcd::store_unit(a, u, bad == KVC_OK ? len : 0, bad == KVC_OK ? n : 0, off);
  }
  if (!kAppend || bad != KVC_OK) return;
  const kvcd::RowMap rows = kvcd::row_map(a, u, off);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int at = lane + 32 * i, t = t0 + at / kVec;
    if (t < n) {
      const int64_t row = rows(len + t) * kVec + at % kVec;
      static_cast<uint4*>(a.Kp)[row] = kx[i];
      static_cast<uint4*>(a.Vp)[row] = vx[i];
    }
  }
  if (lane < kPrepTok && t0 + lane < n) {
    const int64_t row = rows(len + t0 + lane);
    a.logm[row] = 0.f;
    a.pos[row] = pos0 + (float)(t0 + lane);
  }
}

// ---------------------------------------------------------------- window
// One CTA per unit of a call with a window: the first 128-entry tile that holds an
// entry inside the first token's window (the widest).  Tiles before it are seen by
// no token: attention leaves them out, and the mass of their entries only decays.
// In a cache in position order these are all the tiles outside the window.
constexpr int kWinThreads = 1024;
__global__ void __launch_bounds__(kWinThreads) chunk_window_kernel(ChunkArgs a) {
  __shared__ int s_first;
  kvcd::pdl_trigger();
  if (threadIdx.x == 0) s_first = INT_MAX;
  __syncthreads();
  kvcd::pdl_wait();
  const int64_t u = blockIdx.x;
  const int4 v = __ldcg(a.rec + u);                     // the prepare kernel's record
  const int len = v.x;
  const kvcd::RowMap rows = kvcd::row_map(a, u, ((int64_t)(uint32_t)v.z) | ((int64_t)v.w << 32));
  const float pos0 = a.pos_new[u / a.per_seq];
  int mine = len;                                       // the chunk's own entries are always live
  for (int e0 = threadIdx.x; e0 < len && mine == len; e0 += 8 * kWinThreads) {
    float p[8];                                         // eight loads in flight
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = e0 + i * kWinThreads;
      p[i] = e < len ? a.pos[rows(e)] : -INFINITY;
    }
#pragma unroll
    for (int i = 7; i >= 0; --i)
      if (p[i] - pos0 > -a.window) mine = e0 + i * kWinThreads;
  }
  mine = __reduce_min_sync(KVC_FULL_MASK, mine);
  if ((threadIdx.x & 31) == 0) atomicMin(&s_first, mine);
  __syncthreads();
  const int first = s_first & ~127;
  if (threadIdx.x == 0) a.first[u] = first;
  if (a.mass)
    for (int e = threadIdx.x; e < min(len, first); e += kWinThreads) a.mass[rows(e)] *= a.decay;
}

// ---------------------------------------------------------------- fp32 score tile
template <int D, int MR>
struct SimtSmem {
  float q[MR][D + 4];
  float k[kKeys][D + 4];               // then the numerators [MR][kKeys + 4]
  float v[kKeys][D];
  float lm[kKeys], rel[kKeys];
  kvcd::LocateSmem loc;
};

// `count` rows of a [.., D] array in shared memory, row r from row(r); the rest of the kRows zeroed.
template <int D, int kRows, int kStride, class RowFn>
__device__ __forceinline__ void stage_rows(float* dst, const float* src, int count, RowFn row) {
  constexpr int kVec = D / 4;
  for (int i = threadIdx.x; i < kRows * kVec; i += kSimtThreads) {
    const int r = i / kVec, v = i % kVec;
    *reinterpret_cast<float4*>(dst + r * kStride + v * 4) =
        r < count ? *reinterpret_cast<const float4*>(src + row(r) * D + v * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
}

// Products of this thread's R rows and 4 entries (tx + 16 j).
template <int D, int R>
__device__ __forceinline__ void score_tile(const float* q, const float* k, int ty, int tx, float (&s)[R][4]) {
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
  for (int f = 0; f < D; f += 4) {
    float4 kv[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4*>(k + (tx + 16 * j) * (D + 4) + f);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float4 qv = *reinterpret_cast<const float4*>(q + (ty * R + i) * (D + 4) + f);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        s[i][j] = fmaf(qv.x, kv[j].x, fmaf(qv.y, kv[j].y, fmaf(qv.z, kv[j].z, fmaf(qv.w, kv[j].w, s[i][j]))));
    }
  }
}

// Base-2 score from the raw product; sees: whether the row may look at all.
__device__ __forceinline__ float score_of(const ChunkArgs& a, float dot, float lm2, float rel,
                                          float slope2, int t, bool sees) {
  float x = dot * a.scale;
  if (a.softcap > 0.f) x = a.softcap * tanhf(x / a.softcap);
  x = fmaf(x, kvcd::kLog2eC, lm2);
  if (a.slopes) x = fmaf(slope2, rel - (float)t, x);   // pos_e - pos_token
  if (a.window > 0.f && !(rel > (float)t - a.window)) sees = false;
  return sees ? x : -INFINITY;
}

// ln m (base 2) and position relative to the chunk's first token of a tile's
// entries.
__device__ __forceinline__ void stage_bias(const ChunkArgs& a, float* lm, float* rel, int e0, int count,
                                           const kvcd::RowMap& rows, float pos0) {
  for (int c = threadIdx.x; c < kKeys; c += kSimtThreads) {
    lm[c] = c < count ? a.logm[rows(e0 + c)] * kvcd::kLog2eC : 0.f;
    rel[c] = c < count && (a.slopes || a.window > 0.f) ? a.pos[rows(e0 + c)] - pos0 : 0.f;
  }
}

// ---------------------------------------------------------------- fp32 attention
template <int D, int MR>
__global__ void __launch_bounds__(kSimtThreads, 2) chunk_attn_simt_kernel(ChunkArgs a) {
  constexpr int R = MR / 16, C = D / 64;               // rows and 4-feature groups per thread
  extern __shared__ __align__(16) unsigned char simt_raw[];
  auto& sm = *reinterpret_cast<SimtSmem<D, MR>*>(simt_raw);
  float* P = &sm.k[0][0];
  kvcd::pdl_trigger();
  kvcd::pdl_wait();
  const kvcd::AttnCost<kKeys> cost{a};
  const kvcd::Piece piece = kvcd::locate_piece<kSimtThreads>(cost, sm.loc);
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  if (tid == 0) a.seg[blockIdx.x] = ChunkSeg{piece.item, piece.item >= 0 && piece.lo > piece.start};
  if (a.len_out)
    for (int64_t u = (int64_t)blockIdx.x * kSimtThreads + tid; u < a.units; u += (int64_t)gridDim.x * kSimtThreads) {
      const ChunkUnit r = kvcd::load_unit(a, u);
      const int64_t gu = kvcd::unit_global(a, u);
      a.len_out[gu] = r.n > 0 ? r.len + r.n : a.len_lh[gu];
    }
  for (kvcd::Walk<kvcd::AttnCost<kKeys>> w(cost, piece); w.next();) {
    const int64_t u = w.item / a.rp;
    const int t0 = (int)(w.item - u * a.rp) * a.tpb;
    const int h = (int)(u % a.H);
    const float pos0 = a.pos_new[u / a.per_seq];
    const kvcd::RowMap rows = kvcd::row_map(a, u, w.r.off);
    const int used = a.G * a.tt;                       // rows of the block in use
    __syncthreads();
    stage_rows<D, MR, D + 4>(&sm.q[0][0], static_cast<const float*>(a.q), used, [&](int r) {
      return (u * a.G + r / a.tt) * a.T + min(a.T - 1, t0 + r % a.tt);
    });
    int tok[R], lim[R];
    float slope2[R], m[R], l[R], o[R][C][4];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int r = ty * R + i;
      tok[i] = t0 + r % a.tt;
      const bool live = r < used && tok[i] < w.r.n;
      lim[i] = live ? w.r.len + tok[i] + 1 : 0;
      slope2[i] = a.slopes && live ? a.slopes[h * a.G + r / a.tt] * kvcd::kLog2eC : 0.f;
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][c][e] = 0.f;
    }
    const int total = w.r.len + w.r.n;
    for (int tile = w.tb; tile < w.te; ++tile) {
      const int e0 = w.r.first + tile * kKeys, cnt = min(kKeys, total - e0);
      __syncthreads();
      auto row = [&](int r) { return rows(e0 + r); };
      stage_rows<D, kKeys, D + 4>(&sm.k[0][0], static_cast<const float*>(a.Kp), cnt, row);
      stage_rows<D, kKeys, D>(&sm.v[0][0], static_cast<const float*>(a.Vp), cnt, row);
      stage_bias(a, sm.lm, sm.rel, e0, cnt, rows, pos0);
      __syncthreads();
      float s[R][4];
      score_tile<D, R>(&sm.q[0][0], &sm.k[0][0], ty, tx, s);
      __syncthreads();                                 // the keys' place holds the numerators next
#pragma unroll
      for (int i = 0; i < R; ++i) {
        float mx = m[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = tx + 16 * j;
          s[i][j] = score_of(a, s[i][j], sm.lm[c], sm.rel[c], slope2[i], tok[i], e0 + c < lim[i]);
          mx = fmaxf(mx, s[i][j]);
        }
#pragma unroll
        for (int x = 8; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(KVC_FULL_MASK, mx, x));
        const float base = mx == -INFINITY ? 0.f : mx;
        const float f = exp2f(m[i] - base);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = exp2f(s[i][j] - base);
          sum += p;
          P[(ty * R + i) * (kKeys + 4) + tx + 16 * j] = p;
        }
#pragma unroll
        for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(KVC_FULL_MASK, sum, x);
        l[i] = fmaf(l[i], f, sum);
        m[i] = mx;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][c][e] *= f;
      }
      __syncwarp();                                    // a row's numerators come from its own warp
#pragma unroll 2
      for (int kk = 0; kk < kKeys; kk += 4) {
        float p[R][4];
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const float4 v = *reinterpret_cast<const float4*>(P + (ty * R + i) * (kKeys + 4) + kk);
          p[i][0] = v.x; p[i][1] = v.y; p[i][2] = v.z; p[i][3] = v.w;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const float4 v = *reinterpret_cast<const float4*>(&sm.v[kk + e][c * 64 + tx * 4]);
#pragma unroll
            for (int i = 0; i < R; ++i) {
              o[i][c][0] = fmaf(p[i][e], v.x, o[i][c][0]);
              o[i][c][1] = fmaf(p[i][e], v.y, o[i][c][1]);
              o[i][c][2] = fmaf(p[i][e], v.z, o[i][c][2]);
              o[i][c][3] = fmaf(p[i][e], v.w, o[i][c][3]);
            }
          }
      }
    }
    const bool whole = w.whole();
    const int64_t slot = (int64_t)blockIdx.x * 2 + (w.tb == 0 ? 1 : 0);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int r = ty * R + i;
      if (lim[i] == 0) continue;
      if (whole) {
        const float inv = l[i] > 0.f ? 1.f / l[i] : 0.f;
        const int64_t orow = (u * a.G + r / a.tt) * a.T + tok[i];
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            static_cast<float*>(a.out)[orow * D + c * 64 + tx * 4 + e] = o[i][c][e] * inv;
        if (a.lse && tx == 0) a.lse[orow] = l[i] > 0.f ? m[i] + log2f(l[i]) : -INFINITY;
      } else {
        const int64_t prow = slot * MR + r;
#pragma unroll
        for (int c = 0; c < C; ++c)
          *reinterpret_cast<float4*>(a.part + prow * D + c * 64 + tx * 4) =
              make_float4(o[i][c][0], o[i][c][1], o[i][c][2], o[i][c][3]);
        if (tx == 0) { a.part_ml[prow * 2] = m[i]; a.part_ml[prow * 2 + 1] = l[i]; }
      }
    }
  }
}

// ---------------------------------------------------------------- combine
// Block x joins the partial results of the item that the cut before CTA x
// splits, if that is the item's first cut: the head piece lies in slot 2(x-1)+1,
// the following pieces in slots 2x, 2(x+1), ...  blockIdx.y takes a group of
// rows, a warp a row.  Bound by latency, so several pieces are fetched at a time before
// anything is known about them: four where rows are few and pieces many, two in the
// large row blocks, whose items are seldom cut twice (their bytes count: 128 KB a piece).
template <typename T, int D, int kRowsBlock>
__global__ void __launch_bounds__(256) chunk_combine_kernel(const __grid_constant__ ChunkArgs a, int grid) {
  kvcd::pdl_trigger();
  kvcd::pdl_wait();
  const int x = blockIdx.x + 1, lane = threadIdx.x & 31;
  constexpr int C = D / 32, kFetch = kRowsBlock > 128 ? 2 : 4;
  const int r = blockIdx.y * 8 + (threadIdx.x >> 5);
  const ChunkSeg before = a.seg[x - 1], s = a.seg[x];
  if (!s.mid || (before.mid && before.item == s.item)) return;
  const int u = (int)((unsigned)s.item / (unsigned)a.rp);
  const int t0 = ((int)s.item - u * a.rp) * a.tpb;
  const int tile = kRowsBlock > 128 ? r >> 7 : 0, rt = kRowsBlock > 128 ? r & 127 : r;
  const int g = rt / a.tt, t = t0 + tile * a.tt + rt % a.tt;
  if (g >= a.G || t >= a.T || tile * a.tt >= a.tpb) return;
  const int n = __ldcg(a.rec + u).y;                    // new tokens (on its way with the pieces)
  float M = -INFINITY, l = 0.f, o[C];
#pragma unroll
  for (int c = 0; c < C; ++c) o[c] = 0.f;
  bool more = true;                                     // pieces x .. follow the head, as long as they start inside the item
  for (int y0 = x - 1; more; y0 += kFetch) {
    float2 ml[kFetch];
    float pv[kFetch][C];
    bool in[kFetch];
#pragma unroll
    for (int i = 0; i < kFetch; ++i) {
      const int y = y0 + i;
      const ChunkSeg p = y < grid ? a.seg[y] : ChunkSeg{-1, 0};
      in[i] = y == x - 1 || (p.mid && p.item == s.item);
      const int64_t prow = ((int64_t)min(y, grid - 1) * 2 + (y == x - 1 ? 1 : 0)) * kRowsBlock + r;
      ml[i] = *reinterpret_cast<const float2*>(a.part_ml + prow * 2);
      const float* po = a.part + prow * D + lane * C;
      if constexpr (C == 4) {
        const float4 v = *reinterpret_cast<const float4*>(po);
        pv[i][0] = v.x; pv[i][1] = v.y; pv[i][2] = v.z; pv[i][3] = v.w;
      } else {
        const float2 v = *reinterpret_cast<const float2*>(po);
        pv[i][0] = v.x; pv[i][1] = v.y;
      }
    }
#pragma unroll
    for (int i = 0; i < kFetch; ++i) {
      more = more && in[i];
      if (!more || ml[i].x == -INFINITY) continue;       // not the item's, or it saw nothing
      const float Mn = fmaxf(M, ml[i].x);
      const float f0 = exp2f(M - Mn), f1 = exp2f(ml[i].x - Mn);
      l = fmaf(l, f0, ml[i].y * f1);
#pragma unroll
      for (int c = 0; c < C; ++c) o[c] = fmaf(o[c], f0, pv[i][c] * f1);
      M = Mn;
    }
  }
  if (t >= n) return;
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const int64_t orow = ((int64_t)u * a.G + g) * a.T + t;
  T* op = static_cast<T*>(a.out) + orow * D + lane * C;
#pragma unroll
  for (int c = 0; c < C; ++c) op[c] = kvcd::from_f<T>(o[c] * inv);
  if (a.lse && lane == 0) a.lse[orow] = l > 0.f ? M + log2f(l) : -INFINITY;
}

// ---------------------------------------------------------------- fp32 mass
// The tile's keys stay in shared memory while the query rows pass.
template <int D>
__global__ void __launch_bounds__(kSimtThreads, 2) chunk_mass_simt_kernel(ChunkArgs a) {
  constexpr int MR = 64, R = 4;
  extern __shared__ __align__(16) unsigned char simt_raw[];
  auto& sm = *reinterpret_cast<SimtSmem<D, MR>*>(simt_raw);
  float* red = &sm.v[0][0];                            // [16][kKeys] column sums by row group
  kvcd::pdl_trigger();
  kvcd::pdl_wait();
  const kvcd::MassCost<kKeys> cost{a};
  const kvcd::Piece piece = kvcd::locate_piece<kSimtThreads>(cost, sm.loc);
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  if (tid == 0) a.seg[blockIdx.x] = kvcd::mass_seg(cost, piece);
  for (kvcd::MassWalk<kKeys> w(cost, piece); w.next();) {
    const int64_t u = w.u;
    const int e0 = w.r.first + w.tile * kKeys;
    const int h = (int)(u % a.H);
    const float pos0 = a.pos_new[u / a.per_seq];
    const kvcd::RowMap rows = kvcd::row_map(a, u, w.r.off);
    const int cnt = min(kKeys, w.r.len + w.r.n - e0);
    const int used = a.G * a.tt;
    __syncthreads();
    stage_rows<D, kKeys, D + 4>(&sm.k[0][0], static_cast<const float*>(a.Kp), cnt, [&](int r) { return rows(e0 + r); });
    stage_bias(a, sm.lm, sm.rel, e0, cnt, rows, pos0);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int rt = w.tb; rt < w.te; ++rt) {
      const int t0 = rt * a.tt;
      __syncthreads();
      stage_rows<D, MR, D + 4>(&sm.q[0][0], static_cast<const float*>(a.q), used, [&](int r) {
        return (u * a.G + r / a.tt) * a.T + min(a.T - 1, t0 + r % a.tt);
      });
      __syncthreads();
      float s[R][4];
      score_tile<D, R>(&sm.q[0][0], &sm.k[0][0], ty, tx, s);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int r = ty * R + i, t = t0 + r % a.tt;
        if (r >= used || t >= w.r.n) continue;
        const int g = r / a.tt;
        const float lse = a.lse[(u * a.G + g) * a.T + t];
        if (lse == -INFINITY) continue;
        const float slope2 = a.slopes ? a.slopes[h * a.G + g] * kvcd::kLog2eC : 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = tx + 16 * j;
          acc[j] += exp2f(score_of(a, s[i][j], sm.lm[c], sm.rel[c], slope2, t,
                                   c < cnt && e0 + c <= w.r.len + t) - lse);
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) red[ty * kKeys + tx + 16 * j] = acc[j];
    __syncthreads();
    if (tid < cnt) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) sum += red[i * kKeys + tid];
      if (w.whole()) kvcd::mass_store(a, w.r, rows, e0 + tid, sum);
      else a.part[((int64_t)blockIdx.x * 2 + (w.tb == 0 ? 1 : 0)) * kKeys + tid] = sum;
    }
  }
}

// Joins the partial column sums of a key tile that a cut splits (as
// chunk_combine_kernel).
template <int kTile>
__global__ void __launch_bounds__(kTile) chunk_mass_combine_kernel(ChunkArgs a, int grid) {
  kvcd::pdl_trigger();
  kvcd::pdl_wait();
  const int x = blockIdx.x + 1;
  const ChunkSeg s = a.seg[x], before = a.seg[x - 1];
  if (!s.mid || (before.mid && before.item == s.item)) return;
  const int64_t u = s.item >> 32;
  const ChunkUnit r = kvcd::load_unit(a, u);
  const int e = r.first + (int)(s.item & 0xffffffff) * kTile + threadIdx.x;
  if (e >= r.len + r.n) return;
  float sum = a.part[((int64_t)(x - 1) * 2 + 1) * kTile + threadIdx.x];
  for (int y = x; y < grid && a.seg[y].mid && a.seg[y].item == s.item; ++y)
    sum += a.part[(int64_t)y * 2 * kTile + threadIdx.x];
  kvcd::mass_store(a, r, kvcd::row_map(a, u, r.off), e, sum);
}

// ---------------------------------------------------------------- host side
struct ChunkLayout {
  size_t rec, first, seg, part, ml, total;
};

// Partial results: two per CTA.  The bf16 kernels run one CTA per SM, with up to 256 rows (mass:
// 128 entries); the fp32 kernels two, with up to 64 rows (64 entries).
constexpr int kMaxRowsTc = 256, kCtasTc = 1, kMaxRowsSimt = 64, kCtasSimt = 2;

ChunkLayout chunk_layout(const kvc_params* p, size_t units) {
  const bool tc = p->dtype == KVC_BF16;
  const size_t ctas = (size_t)(tc ? kCtasTc : kCtasSimt) * std::max(kvc::sm_count(), 1);
  const size_t rows = ctas * 2 * (tc ? kMaxRowsTc : kMaxRowsSimt);
  ChunkLayout w;
  w.rec = 0;
  w.first = kvc::align256(units * sizeof(int4));
  w.seg = w.first + kvc::align256(units * sizeof(int32_t));
  w.part = w.seg + kvc::align256(ctas * sizeof(ChunkSeg));
  w.ml = w.part + kvc::align256(rows * p->d * sizeof(float));
  w.total = w.ml + kvc::align256(rows * 2 * sizeof(float));
  return w;
}
ChunkLayout chunk_layout(const kvc_params* p, const kvc_chunk* c) {
  return chunk_layout(p, (size_t)p->B * p->H * (c->layer_end - c->layer_begin));
}

bool misaligned16(const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15) != 0; }

template <typename T, int D>
cudaError_t launch_prepare(const ChunkArgs& a, cudaStream_t s) {
  const int groups = a.k_new ? (a.T + kPrepTok - 1) / kPrepTok : 1;
  const int64_t warps = a.units * groups;
  const dim3 grid((unsigned)((warps + kPrepWarps - 1) / kPrepWarps)), block(32 * kPrepWarps);
  kvc::count_launch();
  const cudaError_t e = a.k_new ? kvc::chunk_launch(chunk_prepare_kernel<T, D, true>, grid, block, 0, s, a, groups)
                                : kvc::chunk_launch(chunk_prepare_kernel<T, D, false>, grid, block, 0, s, a, groups);
  if (e != cudaSuccess || !(a.window > 0.f)) return e;
  kvc::count_launch();
  return kvc::chunk_launch(chunk_window_kernel, dim3((unsigned)a.units), dim3(kWinThreads), 0, s, a);
}

template <typename T, int D, int kRowsBlock>
cudaError_t launch_combine(const ChunkArgs& a, int grid, cudaStream_t s) {
  if (grid < 2) return cudaSuccess;
  kvc::count_launch();
  return kvc::chunk_launch(chunk_combine_kernel<T, D, kRowsBlock>, dim3(grid - 1, kRowsBlock / 8), dim3(256), 0, s, a,
                           grid);
}

template <int D, int MR>
cudaError_t launch_attn_simt(ChunkArgs& a, int sms, cudaStream_t s) {
  a.tt = std::min(MR / a.G, a.T);
  a.tpb = a.tt;
  a.rp = (a.T + a.tpb - 1) / a.tpb;
  const size_t smem = sizeof(SimtSmem<D, MR>);
  cudaError_t e = kvc::chunk_allow_smem<chunk_attn_simt_kernel<D, MR>>(smem);
  if (e != cudaSuccess) return e;
  const int grid = kCtasSimt * sms;
  e = kvc::chunk_launch(chunk_attn_simt_kernel<D, MR>, dim3(grid), dim3(kSimtThreads), smem, s, a);
  if (e != cudaSuccess) return e;
  kvc::count_launch();
  return launch_combine<float, D, MR>(a, grid, s);
}

// Attention and the joining of its pieces; the units' records and the entries are there.
template <int D>
cudaError_t launch_attn_prepared(ChunkArgs& a, int sms, int page_rows, cudaStream_t s) {
  const cudaError_t e = kvc::chunk_attn_tc_launch(a, D, sms, page_rows, s);
  if (e != cudaSuccess) return e;
  return a.T > a.tt ? launch_combine<__nv_bfloat16, D, 256>(a, sms, s) : launch_combine<__nv_bfloat16, D, 128>(a, sms, s);
}

template <int D>
cudaError_t launch_attn_bf16(ChunkArgs& a, int sms, int page_rows, cudaStream_t s) {
  const cudaError_t e = launch_prepare<__nv_bfloat16, D>(a, s);
  return e != cudaSuccess ? e : launch_attn_prepared<D>(a, sms, page_rows, s);
}

template <int D>
cudaError_t launch_attn_f32(ChunkArgs& a, int sms, cudaStream_t s) {
  cudaError_t e = launch_prepare<float, D>(a, s);
  if (e != cudaSuccess) return e;
  if (a.G * a.T <= 16) return launch_attn_simt<D, 16>(a, sms, s);
  return launch_attn_simt<D, 64>(a, sms, s);
}

template <int kTile>
cudaError_t launch_mass_combine(const ChunkArgs& a, int grid, cudaStream_t s) {
  if (grid < 2) return cudaSuccess;
  kvc::count_launch();
  return kvc::chunk_launch(chunk_mass_combine_kernel<kTile>, dim3(grid - 1), dim3(kTile), 0, s, a, grid);
}

template <int D>
cudaError_t launch_mass_bf16(ChunkArgs& a, int sms, int page_rows, cudaStream_t s) {
  cudaError_t e = launch_prepare<__nv_bfloat16, D>(a, s);
  if (e == cudaSuccess) e = kvc::chunk_mass_tc_launch(a, D, sms, page_rows, s);
  if (e != cudaSuccess) return e;
  return launch_mass_combine<128>(a, sms, s);
}

template <int D>
cudaError_t launch_mass_f32(ChunkArgs& a, int sms, cudaStream_t s) {
  cudaError_t e = launch_prepare<float, D>(a, s);
  if (e != cudaSuccess) return e;
  a.tt = std::min(64 / a.G, a.T);
  const size_t smem = sizeof(SimtSmem<D, 64>);
  e = kvc::chunk_allow_smem<chunk_mass_simt_kernel<D>>(smem);
  if (e != cudaSuccess) return e;
  const int grid = kCtasSimt * sms;
  e = kvc::chunk_launch(chunk_mass_simt_kernel<D>, dim3(grid), dim3(kSimtThreads), smem, s, a);
  if (e != cudaSuccess) return e;
  kvc::count_launch();
  return launch_mass_combine<kKeys>(a, grid, s);
}

}  // namespace

namespace kvc {

int chunk_check(const kvc_params* p, const kvc_chunk* c) {
  const int st = check_params(p);
  if (st != KVC_OK) return st;
  if (!c || c->T < 1 || c->T > 65536) return KVC_EINVAL;
  if (c->layer_begin < 0 || c->layer_begin >= c->layer_end || c->layer_end > p->L) return KVC_EINVAL;
  if (p->packed_rows < 1 || p->packed_rows >= (1LL << 31)) return KVC_EINVAL;
  if (c->page_rows != 0) {
    if (c->page_rows < 16 || c->page_rows > 1024 || (c->page_rows & (c->page_rows - 1))) return KVC_EINVAL;
    if (!c->page_table || c->max_pages < 1 || p->packed_rows < c->page_rows) return KVC_EINVAL;
  }
  if (!(c->softcap >= 0.f && c->softcap < INFINITY && c->window >= 0.f && c->window < INFINITY)) return KVC_EINVAL;
  // units times row blocks, and the prepare kernel's grid, stay below 2^31
  const int64_t units = (int64_t)p->B * p->H * (c->layer_end - c->layer_begin);
  if (units > (1 << 24) || units * ((c->T + 1) / 2) >= (1LL << 31)) return KVC_EINVAL;
  return KVC_OK;
}

void chunk_fill(ChunkArgs& a, const kvc_params* p, const kvc_chunk* c) {
  const int Lr = c->layer_end - c->layer_begin;
  a.page_table = c->page_rows ? c->page_table : nullptr;
  a.n_new = c->n_new;
  a.slopes = c->slopes;
  a.packed_rows = p->packed_rows;
  a.units = (int64_t)p->B * Lr * p->H;
  a.lh_span = (int64_t)Lr * p->H;
  a.lh_gap = (int64_t)(p->L - Lr) * p->H;
  a.lh_base = (int64_t)c->layer_begin * p->H;
  a.T = c->T;
  a.H = p->H;
  a.G = p->G;
  a.per_seq = Lr * p->H;
  a.max_pages = c->max_pages;
  a.page_shift = 0;
  while (c->page_rows >> (a.page_shift + 1)) ++a.page_shift;
  a.scale = 1.f / sqrtf((float)p->d);
  a.scale_log2 = a.scale * kvcd::kLog2eC;
  // Beyond these a cap has no effect on scores of any size that fp32 sums tell apart (above), or
  // leaves nothing of them (below); the reciprocal and the base-2 cap stay finite and normal.
  a.softcap = c->softcap > 0.f ? std::min(std::max(c->softcap, 0x1p-64f), 0x1p64f) : 0.f;
  // Distances are multiples of 1/2, so the next multiple of 1/2 is the same window, and the
  // kernels' differences of positions and windows are exact (token - 33.0000038 is not: it can round to
  // the position of an entry inside).  A float of 2^22 or more is a multiple of 1/2 itself.
  a.window = c->window < 0x1p22f ? 0.5f * ceilf(2.f * c->window) : c->window;
  a.wait_ns = wait_limit_ns();
  a.withhold = withhold_copies();
}

size_t chunk_rows_bytes(const kvc_params* p, int64_t units) { return chunk_layout(p, (size_t)units).total; }

void chunk_rows_workspace(ChunkArgs& a, const kvc_params* p, int64_t units, void* workspace) {
  const ChunkLayout w = chunk_layout(p, (size_t)units);
  char* ws = static_cast<char*>(workspace);
  a.rec = reinterpret_cast<int4*>(ws + w.rec);
  a.first = reinterpret_cast<int32_t*>(ws + w.first);
  a.seg = reinterpret_cast<ChunkSeg*>(ws + w.seg);
  a.part = reinterpret_cast<float*>(ws + w.part);
  a.part_ml = reinterpret_cast<float*>(ws + w.ml);
}

cudaError_t chunk_attn_rows(ChunkArgs& a, int d, int sms, cudaStream_t s) {
  return d == 128 ? launch_attn_prepared<128>(a, sms, 0, s) : launch_attn_prepared<64>(a, sms, 0, s);
}

static int chunk_workspace(ChunkArgs& a, const kvc_params* p, const kvc_chunk* c, void* workspace, size_t ws_bytes) {
  if (!workspace || ws_bytes < chunk_layout(p, c).total || (reinterpret_cast<uintptr_t>(workspace) & 255)) return KVC_EWORKSPACE;
  chunk_rows_workspace(a, p, (int64_t)p->B * p->H * (c->layer_end - c->layer_begin), workspace);
  return KVC_OK;
}

}  // namespace kvc

extern "C" size_t kvc_chunk_workspace_bytes(const kvc_params* p, const kvc_chunk* c) {
  if (kvc::chunk_check(p, c) != KVC_OK) return 0;
  return chunk_layout(p, c).total;
}

extern "C" int kvc_chunk_attn(const kvc_params* p, const kvc_chunk* c, const void* q, const void* k_new,
                              const void* v_new, const float* pos_new, void* Kp, void* Vp, float* logm,
                              float* pos, const int32_t* len_lh, const int32_t* cap_lh,
                              const int64_t* off_lh, void* out, float* lse, int32_t* len_out,
                              void* workspace, size_t ws_bytes, void* stream) {
  int st = kvc::chunk_check(p, c);
  if (st != KVC_OK) return st;
  if (!q || !k_new || !v_new || !pos_new || !Kp || !Vp || !logm || !pos || !len_lh || !cap_lh || !out ||
      (!off_lh && c->page_rows == 0))
    return KVC_EINVAL;
  if (misaligned16(q) || misaligned16(k_new) || misaligned16(v_new) || misaligned16(Kp) || misaligned16(Vp) ||
      (reinterpret_cast<uintptr_t>(out) & 31))
    return KVC_EINVAL;
  ChunkArgs a = {};
  kvc::chunk_fill(a, p, c);
  st = kvc::chunk_workspace(a, p, c, workspace, ws_bytes);
  if (st != KVC_OK) return st;
  a.err = kvc::err_word();
  const int sms = kvc::sm_count();
  if (!a.err || sms <= 0 || !kvc::chunk_tc_available()) return KVC_ECUDA;
  a.q = q; a.k_new = k_new; a.v_new = v_new; a.pos_new = pos_new;
  a.Kp = Kp; a.Vp = Vp; a.logm = logm; a.pos = pos;
  a.len_lh = len_lh; a.cap_lh = cap_lh; a.off_lh = off_lh;
  a.out = out; a.lse = lse; a.len_out = len_out;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (p->dtype == KVC_BF16)
    e = p->d == 128 ? launch_attn_bf16<128>(a, sms, c->page_rows, s) : launch_attn_bf16<64>(a, sms, c->page_rows, s);
  else
    e = p->d == 128 ? launch_attn_f32<128>(a, sms, s) : launch_attn_f32<64>(a, sms, s);
  return kvc::cuda_status(e);
}

extern "C" int kvc_chunk_mass(const kvc_params* p, const kvc_chunk* c, const void* q, const void* Kp,
                              const float* logm, const float* pos, const float* pos_new,
                              const int32_t* len_lh, const int64_t* off_lh, const float* lse, float decay,
                              float* mass, void* workspace, size_t ws_bytes, void* stream) {
  return kvc_chunk_mass_cap(p, c, q, Kp, logm, pos, pos_new, len_lh, nullptr, off_lh, lse, decay, mass, workspace,
                            ws_bytes, stream);
}

extern "C" int kvc_chunk_mass_cap(const kvc_params* p, const kvc_chunk* c, const void* q, const void* Kp,
                                  const float* logm, const float* pos, const float* pos_new,
                                  const int32_t* len_lh, const int32_t* cap_lh, const int64_t* off_lh,
                                  const float* lse, float decay, float* mass, void* workspace,
                                  size_t ws_bytes, void* stream) {
  int st = kvc::chunk_check(p, c);
  if (st != KVC_OK) return st;
  if (!q || !Kp || !logm || !pos || !pos_new || !len_lh || !lse || !mass || (!off_lh && c->page_rows == 0) ||
      !(decay >= 0.f && decay <= 1.f))
    return KVC_EINVAL;
  if (misaligned16(q) || misaligned16(Kp)) return KVC_EINVAL;
  ChunkArgs a = {};
  kvc::chunk_fill(a, p, c);
  st = kvc::chunk_workspace(a, p, c, workspace, ws_bytes);
  if (st != KVC_OK) return st;
  a.err = kvc::err_word();
  const int sms = kvc::sm_count();
  if (!a.err || sms <= 0 || !kvc::chunk_tc_available()) return KVC_ECUDA;
  a.q = q; a.Kp = const_cast<void*>(Kp); a.logm = const_cast<float*>(logm); a.pos = const_cast<float*>(pos);
  a.pos_new = pos_new; a.len_lh = len_lh; a.cap_lh = cap_lh; a.off_lh = off_lh; a.lse = const_cast<float*>(lse);
  a.decay = decay; a.mass = mass;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (p->dtype == KVC_BF16)
    e = p->d == 128 ? launch_mass_bf16<128>(a, sms, c->page_rows, s) : launch_mass_bf16<64>(a, sms, c->page_rows, s);
  else
    e = p->d == 128 ? launch_mass_f32<128>(a, sms, s) : launch_mass_f32<64>(a, sms, s);
  return kvc::cuda_status(e);
}

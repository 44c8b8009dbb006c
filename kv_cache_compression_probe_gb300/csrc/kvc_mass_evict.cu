// kvc_mass_evict: per-(b,l,h) eviction by accumulated attention mass.
//
// Plan: a CTA per (b,l,h), or a cluster of up to 8 when there are few and long ones,
// reads the masses and positions once, keeps a 32-bit order code per entry in shared
// memory (protected entries have the largest code) and finds the smallest code that
// stays by a radix select of 11 bits at a time; the CTAs of a cluster add their
// histograms through distributed shared memory.  Then it lists the moves: evicted
// entries below the new length ("holes") take the staying entries at or above it,
// both in index order.  Bound by latency: one read of 8 bytes an entry, then a dozen
// block-wide steps on shared memory.
// Measured, both kernels: 256 (b,l,h) of 3300..5100 entries 20 us, 64 of 5000..8192 with 34 MB
// to move 35 us.  Loads in batches of eight, one barrier per prefix, protected entries kept out
// of the histograms and a search that ends once a whole bin stays took 2 to 5 us off.
// Move: a second kernel copies the rows (5 TB/s for 34 MB moved).  Moving only those, instead of compacting
// the cache, keeps the traffic at twice the moved rows; the row order stops
// following the positions, so protection goes by position and not by index.
#include <cooperative_groups.h>

#include <algorithm>

#include "kvc_chunk.cuh"
#include "kvc_internal.h"

namespace {

using kvc::ChunkArgs;

namespace cg = cooperative_groups;

constexpr int kPlanThreads = 512;     // 256 (b,l,h) of 4200 entries: 256, 512, 1024 threads took 28, 20, 27 us
constexpr int kBins = 2048;
constexpr int kCluster = 8;            // CTAs of a cluster at most
constexpr int kMaxKeys = 50000;        // order codes of one CTA in shared memory (200 KB)
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

// Exclusive prefixes of N counts over the block, and their totals.  One barrier: every warp
// adds up the warps' sums itself, and calls alternate between two buffers.
template <int N>
__device__ __forceinline__ void block_prefix(const int (&v)[N], int (*s_warp)[32], int (&excl)[N], int (&total)[N]) {
  constexpr int kWarps = kPlanThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl[N];
#pragma unroll
  for (int c = 0; c < N; ++c) {
    incl[c] = v[c];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(KVC_FULL_MASK, incl[c], o);
      if (lane >= o) incl[c] += x;
    }
    if (lane == 31) s_warp[c][warp] = incl[c];
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < N; ++c) {
    int w = lane < kWarps ? s_warp[c][lane] : 0;
#pragma unroll
    for (int o = 1; o < kWarps; o <<= 1) {
      const int x = __shfl_up_sync(KVC_FULL_MASK, w, o);
      if (lane >= o) w += x;
    }
    const int before = __shfl_sync(KVC_FULL_MASK, w, max(warp - 1, 0));
    excl[c] = incl[c] - v[c] + (warp > 0 ? before : 0);
    total[c] = __shfl_sync(KVC_FULL_MASK, w, kWarps - 1);
  }
}

struct PlanSmem {
  uint32_t hist[2][kBins];             // passes alternate, so one barrier a pass is enough
  int warp[2][2][32];                  // sums of block_prefix: two buffers of two counts
  int ties, holes, movers, safe;       // this CTA's counts, read by the cluster
  uint32_t prefix;
  int rem, found;                      // entries of the bin that stay; whether that is all of it
};

// kKeys: the codes are in shared memory; else every pass forms them from global memory.
template <bool kKeys>
__global__ void __launch_bounds__(kPlanThreads) mass_plan_kernel(const __grid_constant__ EvictArgs ea) {
  const ChunkArgs& a = ea.a;
  extern __shared__ __align__(16) unsigned char plan_raw[];
  PlanSmem& sm = *reinterpret_cast<PlanSmem*>(plan_raw);
  uint32_t* keys = reinterpret_cast<uint32_t*>(plan_raw + sizeof(PlanSmem));
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), nr = (int)cluster.num_blocks();
  auto sync = [&]() {
    if (nr > 1) cluster.sync();
    else __syncthreads();
  };
  kvcd::pdl_trigger();
  kvcd::pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t u = blockIdx.x / nr;
  const int64_t gu = kvcd::unit_global(a, u);
  const int len = a.len_lh[gu], keep = ea.keep_lh[gu];
  const int64_t off = a.page_table ? 0 : a.off_lh[gu];
  const float safe_from = ea.pos_next[u / a.per_seq] - ea.recent;
  bool ok = len >= 0 && len <= ea.max_len && len <= a.packed_rows && off >= 0 &&
            (a.page_table || off + len <= a.packed_rows);
  if (ok && a.page_table) {
    const int need = (int)(((int64_t)len + (1 << a.page_shift) - 1) >> a.page_shift);
    ok = need <= a.max_pages;
    if (ok) {
      const int32_t* tab = a.page_table + gu * a.max_pages;
      const int64_t pages = a.packed_rows >> a.page_shift;
      for (int i = tid; i < need; i += kPlanThreads) ok &= __ldg(tab + i) >= 0 && __ldg(tab + i) < pages;
    }
  }
  if (tid == 0) sm.safe = sm.ties = sm.holes = sm.movers = 0;
  for (int i = tid; i < kBins; i += kPlanThreads) sm.hist[0][i] = 0;
  if (!__syncthreads_and(ok)) {                        // every CTA of the cluster sees the same
    if (tid == 0 && rank == 0) {
      kvcd::record_error(a.err, KVC_EDEVICE);
      ea.n_moves[u] = 0;
      a.len_out[gu] = len;
    }
    return;
  }
  const kvcd::RowMap rows = kvcd::row_map(a, u, off);
  const int share = (len + nr - 1) / nr;
  const int lo = min(len, rank * share), n = min(len, lo + share) - lo;   // this CTA's entries
  auto form = [&](int i) {
    const int64_t row = rows(lo + i);
    return mass_code(a.mass[row], a.pos[row] >= safe_from);
  };
  auto code = [&](int i) { return kKeys ? keys[i] : form(i); };
  int mine = 0;
  constexpr int kBatch = 8;                            // loads in flight per thread, times two
  for (int i0 = tid; i0 < n; i0 += kBatch * kPlanThreads) {
    float m[kBatch], p[kBatch];
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      const int64_t row = rows(lo + min(i0 + x * kPlanThreads, n - 1));
      m[x] = a.mass[row];
      p[x] = a.pos[row];
    }
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      const int i = i0 + x * kPlanThreads;
      if (i >= n) break;
      const uint32_t k = mass_code(m[x], p[x] >= safe_from);
      if (kKeys) keys[i] = k;
      mine += k == 0xffffffffu;
    }
  }
  mine = __reduce_add_sync(KVC_FULL_MASK, mine);
  if (lane == 0 && mine) atomicAdd(&sm.safe, mine);
  sync();
  auto total = [&](int PlanSmem::*m) {                 // a count over the cluster
    int t = 0;
    for (int r = 0; r < nr; ++r) t += cluster.map_shared_rank(&sm, r)->*m;
    return t;
  };
  auto before = [&](int PlanSmem::*m) {                // and over the CTAs before this one
    int t = 0;
    for (int r = 0; r < rank; ++r) t += cluster.map_shared_rank(&sm, r)->*m;
    return t;
  };
  const int safe = total(&PlanSmem::safe), B = min(len, max(max(0, keep), safe));
  const bool all = B >= len, none = B == 0;
  // The B-th largest code, 11 or 10 bits at a time.  The histograms leave the protected entries
  // out (they would all hit one bin), and the search ends as soon as a whole bin stays: then its
  // lower end cuts as well.  Nothing to look for when all, none or the protected ones stay.
  uint32_t cut = safe == B ? 0xffffffffu : 0u;
  int rem = safe == B ? B : B - safe;                  // how many of the entries at the cut stay
  bool found = all || none || safe == B;               // every entry at or above the cut stays
  int turn = 0;
  for (int pass = 0; pass < 3 && !found; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
    const uint32_t mask = pass == 0 ? 0u : 0xffffffffu << (shift + (pass == 1 ? 11 : 10));
    uint32_t* hist = sm.hist[pass & 1];
    for (int i = tid; i < n; i += kPlanThreads) {
      const uint32_t k = code(i);
      if ((k & mask) == cut && k != 0xffffffffu) atomicAdd(&hist[(k >> shift) & (bins - 1)], 1u);
    }
    sync();
    for (int i = tid; i < kBins; i += kPlanThreads) sm.hist[(pass + 1) & 1][i] = 0;
    // a thread holds kOwn bins, from the top down
    constexpr int kOwn = kBins / kPlanThreads;
    const int b0 = bins - 1 - kOwn * tid;
    int c[kOwn], sum = 0;
#pragma unroll
    for (int x = 0; x < kOwn; ++x) c[x] = 0;
    if (b0 > 0)
      for (int r = 0; r < nr; ++r) {
        const uint32_t* h = nr > 1 ? cluster.map_shared_rank(hist, r) : hist;
#pragma unroll
        for (int x = 0; x < kOwn; ++x) c[x] += (int)h[b0 - x];
      }
#pragma unroll
    for (int x = 0; x < kOwn; ++x) sum += c[x];
    int at;
    {
      int excl[1], all_bins[1];
      block_prefix<1>({sum}, sm.warp[turn], excl, all_bins);
      turn ^= 1;
      at = excl[0];
    }
    if (at < rem && rem <= at + sum) {                 // one thread: the counts reach rem here
#pragma unroll
      for (int x = 0; x < kOwn; ++x) {
        if (at < rem && rem <= at + c[x]) {
          sm.prefix = cut | ((uint32_t)(b0 - x) << shift);
          sm.rem = rem - at;
          sm.found = rem - at == c[x];
        }
        at += c[x];
      }
    }
    __syncthreads();
    cut = sm.prefix;
    rem = sm.rem;
    found = sm.found;
  }
  // contiguous ranges per thread (an odd count keeps them off each other's banks), so that
  // thread order is index order
  const int per = ((n + kPlanThreads - 1) / kPlanThreads) | 1;
  const int i0 = min(n, tid * per), i1 = min(n, i0 + per);
  int tie0 = 0;
  if (!found) {                                        // the first `rem` of the equal codes at the cut stay
    int ties[1] = {0}, excl[1], t[1];
    for (int i = i0; i < i1; ++i) ties[0] += code(i) == cut;
    block_prefix<1>(ties, sm.warp[turn], excl, t);
    turn ^= 1;
    if (tid == 0) sm.ties = t[0];
    sync();
    tie0 = excl[0] + before(&PlanSmem::ties);
  }
  int tie = tie0;
  auto stays = [&](int i) {
    if (all || none) return all;
    const uint32_t k = code(i);
    return k > cut || (k == cut && (found || tie++ < rem));
  };
  int count[2] = {0, 0}, at[2], sums[2];               // holes and movers
  for (int i = i0; i < i1; ++i) {
    const bool s = stays(i);
    if (lo + i < B) count[0] += !s;
    else count[1] += s;
  }
  block_prefix<2>(count, sm.warp[turn], at, sums);
  if (tid == 0) { sm.holes = sums[0]; sm.movers = sums[1]; }
  sync();
  int h0 = at[0] + before(&PlanSmem::holes), m0 = at[1] + before(&PlanSmem::movers);
  int2* mv = ea.moves + u * ea.cols;
  tie = tie0;
  if (count[0] + count[1] > 0)
    for (int i = i0; i < i1; ++i) {
      const bool s = stays(i);
      if (lo + i < B && !s) mv[h0++].x = lo + i;
      else if (lo + i >= B && s) mv[m0++].y = lo + i;
    }
  if (rank == 0 && tid == 0) {
    ea.n_moves[u] = total(&PlanSmem::holes);
    a.len_out[gu] = B;
  }
  if (nr > 1) cluster.sync();                          // nobody leaves while its counts are read
}

__global__ void __launch_bounds__(256) mass_move_kernel(const __grid_constant__ EvictArgs ea) {
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
  // A cluster of up to 8 per (b,l,h) while that leaves an SM to each CTA and more than 1024
  // entries a share.
  int nr = 1;
  while (nr < kCluster && ea.a.units * nr * 2 <= sms && max_len / (nr * 2) > 1024) nr *= 2;
  const int64_t share = ((int64_t)max_len + nr - 1) / nr;
  const bool in_smem = share <= kMaxKeys;
  const size_t smem = sizeof(PlanSmem) + (in_smem ? share * sizeof(uint32_t) : 0);
  cudaError_t e = in_smem ? kvc::chunk_allow_smem<mass_plan_kernel<true>>(sizeof(PlanSmem) + kMaxKeys * sizeof(uint32_t))
                          : cudaSuccess;
  if (e == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(ea.a.units * nr));
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = nr;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    e = in_smem ? cudaLaunchKernelEx(&cfg, mass_plan_kernel<true>, ea) : cudaLaunchKernelEx(&cfg, mass_plan_kernel<false>, ea);
  }
  if (e != cudaSuccess) return kvc::cuda_status(e);
  kvc::count_launch(2);
  // at most max_len / 2 moves per unit, usually few: about 8 CTAs per SM stride over them
  const int64_t need = (ea.cols + kMoveRows - 1) / kMoveRows;
  const int64_t x = std::max<int64_t>(1, std::min<int64_t>(need, (8LL * sms + ea.a.units - 1) / ea.a.units));
  e = kvc::chunk_launch(mass_move_kernel, dim3((unsigned)x, (unsigned)ea.a.units), dim3(256), 0, s, ea);
  return kvc::cuda_status(e);
}

// kvc_chunk_mass in bf16 on the tensor cores.
//
// Transposed products, S^T[128 entries x N query rows] = K Q^T: an entry is a
// TMEM lane, so the thread that owns it adds 2^(s - lse) over its columns with
// no exchange, and the sum stays in one register.  A key tile is loaded once and
// the query row tiles (128 rows: tt tokens x G heads; fewer, rounded up to 16,
// when the chunk is smaller) pass it.  Four groups of four warps take the steps
// in turn, each with its own TMEM buffer, which hides the latency of a step's
// chain; a key tile with several steps is joined through shared memory in group
// order.  Few rows: HBM is the bound (K is read once); many rows: the exponential
// unit (one exponential a score), just above the tensor cores' own time.  Then the
// product also carries -lse and ln m (an extra 16-wide step), so that a score costs a
// multiplication, an exponential and an addition: values read per score from shared
// memory would cost its full width.
// Measured (d 128, G 4): one token over 256 caches of 3200..5000 entries 51 us, 5.5
// TB/s; 1024 tokens over 7168 entries, 8 KV heads: 93 us, 2.7e12 scores a second.
// Warps: 0 copies (TMA; and the entries' ln m), 1 issues the products, 2 and 3 fetch
// the row statistics of alternate steps, 4..19 are the four groups.
#include <algorithm>

#include "kvc_chunk_tc.cuh"

namespace {

using kvc::ChunkArgs;
using kvc::ChunkUnit;
using namespace kvctc;

constexpr int kGroups = 4;
constexpr int kThreads = 128 + kGroups * 128;
constexpr int kCols = 512;             // a 128-column buffer per group

// What a kernel adds to the products: kPlain and the rest from shared memory, kExtra
// (several row tiles, no cap, bias or window) in the product itself.
enum Mode { kPlain, kExtra, kCapped, kPos, kCapPos };

// Key and query tiles in flight: keys stream past one row tile, or stay while row
// tiles stream past them.
constexpr int kTiles = 6;
// With one row tile of up to 64 rows the query rows come with the keys: four places of
// 64 rows in the query slots, one barrier and one release for both (a tile's keys take
// 1400 cycles of HBM, and the single thread that issues the products needed as long for
// its waits and commits).
constexpr uint32_t kFoldHalf = 64 * 128;   // of a 64-feature block
__device__ __forceinline__ int key_slots(bool several) { return several ? 2 : 4; }

template <int D>
struct MassSmem {
  static constexpr uint32_t kTileBytes = 128 * D * 2;
  alignas(1024) unsigned char tile[kTiles][kTileBytes];          // key slots, then query slots
  alignas(16) unsigned char ext_k[2][4096], ext_q[kGroups][4096];
  alignas(16) float nl[kGroups][128];                  // -lse of a row, -inf for rows that add nothing
  alignas(16) float slope[kGroups][128], tok[kGroups][128];
  float hand[kGroups][128];
  uint64_t k_full[4], k_empty[4], q_full[4], q_empty[4];
  uint64_t r_full[kGroups], r_empty[kGroups], s_full[kGroups], s_empty[kGroups];
  uint64_t hand_full, hand_empty, drain;
  kvcd::LocateSmem loc;
  uint32_t tmem;
  int abort;
};

// Sum over 16 columns of one entry's 2^(s - lse).  kEdge: some row adds nothing
// or does not see some entry of the tile.
template <bool kCap, bool kPos, bool kEdge>
__device__ __forceinline__ void add16(const ChunkArgs& a, const uint32_t (&s)[16], const float* nl, const float* slope,
                                      const float* tok, float lm, float rel, float first_tok, uint64_t& sum0,
                                      uint64_t& sum1) {
  const uint64_t sc = pk(a.scale_log2, a.scale_log2), lm2 = pk(lm, lm), rel2 = pk(rel, rel);
  const float cap_in = kCap ? a.scale / a.softcap : 0.f, cap_out = kCap ? a.softcap * kvcd::kLog2eC : 0.f;
#pragma unroll
  for (int c = 0; c < 16; c += 4) {
    const float4 n = *reinterpret_cast<const float4*>(nl + c);
    uint64_t x0 = add2(pk(n.x, n.y), lm2), x1 = add2(pk(n.z, n.w), lm2);
    if constexpr (kCap) {
      const uint64_t co = pk(cap_out, cap_out);
      x0 = fma2(pk(tanh_f(__uint_as_float(s[c]) * cap_in), tanh_f(__uint_as_float(s[c + 1]) * cap_in)), co, x0);
      x1 = fma2(pk(tanh_f(__uint_as_float(s[c + 2]) * cap_in), tanh_f(__uint_as_float(s[c + 3]) * cap_in)), co, x1);
    } else {
      x0 = fma2(pk(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sc, x0);
      x1 = fma2(pk(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])), sc, x1);
    }
    float4 t;
    if constexpr (kEdge) t = *reinterpret_cast<const float4*>(tok + c);
    if constexpr (kPos) {
      const float4 sl = *reinterpret_cast<const float4*>(slope + c);
      x0 = fma2(pk(sl.x, sl.y), rel2, x0);
      x1 = fma2(pk(sl.z, sl.w), rel2, x1);
    }
    float f[4];
    upk(x0, f[0], f[1]);
    upk(x1, f[2], f[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = kvcd::ex2(f[e]);
    if constexpr (kEdge) {
      const float nn[4] = {n.x, n.y, n.z, n.w}, tt[4] = {t.x, t.y, t.z, t.w};
      const float w = kPos && a.window > 0.f ? a.window : INFINITY;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        bool sees = nn[e] != -INFINITY && tt[e] >= first_tok;
        if constexpr (kPos) sees = sees && rel > tt[e] - w;
        f[e] = sees ? f[e] : 0.f;
      }
    }
    sum0 = add2(sum0, pk(f[0], f[1]));
    sum1 = add2(sum1, pk(f[2], f[3]));
  }
}

// Sum over 16 columns whose products are the whole score.  kEdge as in add16.
template <bool kEdge>
__device__ __forceinline__ void sum16(const ChunkArgs& a, const uint32_t (&s)[16], const float* tok, float first_tok,
                                      uint64_t& sum0, uint64_t& sum1) {
  const uint64_t sc = pk(a.scale_log2, a.scale_log2);
#pragma unroll
  for (int c = 0; c < 16; c += 4) {
    float f[4];
    upk(mul2(pk(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sc), f[0], f[1]);
    upk(mul2(pk(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])), sc), f[2], f[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = kvcd::ex2(f[e]);
    if constexpr (kEdge) {
      const float4 t = *reinterpret_cast<const float4*>(tok + c);
      f[0] = t.x >= first_tok ? f[0] : 0.f;
      f[1] = t.y >= first_tok ? f[1] : 0.f;
      f[2] = t.z >= first_tok ? f[2] : 0.f;
      f[3] = t.w >= first_tok ? f[3] : 0.f;
    }
    sum0 = add2(sum0, pk(f[0], f[1]));
    sum1 = add2(sum1, pk(f[2], f[3]));
  }
}

template <int D, int kMode>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_mass_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap qmap,
                         const __grid_constant__ ChunkArgs a) {
  using Smem = MassSmem<D>;
  constexpr int kBlocks = D / 64;
  constexpr uint32_t kFoldPlace = kBlocks * kFoldHalf;
  constexpr bool kCap = kMode == kCapped || kMode == kCapPos, kBias = kMode == kPos || kMode == kCapPos;
  extern __shared__ __align__(1024) unsigned char mass_raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(mass_raw) + 1023) & ~uintptr_t(1023));
  kvcd::pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      kvcd::mbar_init(&sm.k_full[i], kMode == kExtra ? 2 : 1);    // copy and extra columns
      kvcd::mbar_init(&sm.k_empty[i], 1);
      kvcd::mbar_init(&sm.q_full[i], 1);
      kvcd::mbar_init(&sm.q_empty[i], 1);
    }
    for (int i = 0; i < kGroups; ++i) {
      kvcd::mbar_init(&sm.r_full[i], 1);
      kvcd::mbar_init(&sm.r_empty[i], 4);
      kvcd::mbar_init(&sm.s_full[i], 1);
      kvcd::mbar_init(&sm.s_empty[i], 4);
    }
    kvcd::mbar_init(&sm.hand_full, 4 * kGroups);
    kvcd::mbar_init(&sm.hand_empty, 4);
    kvcd::mbar_init(&sm.drain, 1);
    sm.abort = 0;
    kvcd::fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(kvcd::smem_u32(&sm.tmem)),
                 "r"((uint32_t)kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  kvcd::pdl_wait();                                    // the prepare kernel's records
  const kvcd::MassCost<128> cost{a};
  const kvcd::Piece piece = kvcd::locate_piece<kThreads>(cost, sm.loc);
  if (tid == 0) a.seg[blockIdx.x] = kvcd::mass_seg(cost, piece);
  const uint32_t tmem = sm.tmem;
  volatile int* abort_flag = &sm.abort;
  const uint64_t ns = a.wait_ns;
  const int used = a.G * a.tt, cols = (used + 15) & ~15;         // rows of a row tile; columns of S^T
  const int kK = key_slots(a.T > a.tt), kQ = min(4, kTiles - kK);
  const bool fold = kMode != kExtra && a.T <= a.tt && used <= 64;
  int k_loads = 0, q_loads = 0;                        // copies issued (for the drain after a give-up)

  if (warp == 0) {
    // ------------------------------------------------------------ copies
    fence_proxy_async_all();
    int nk = 0, nq = 0;
    bool ok = true;
    float lm[4] = {0.f, 0.f, 0.f, 0.f};
    auto fetch_lm = [&](const kvcd::MassWalk<128>& w) {
      const kvcd::RowMap rows = kvcd::row_map(a, w.u, w.r.off);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = w.r.first + w.tile * 128 + lane + 32 * j;
        lm[j] = e < w.r.len + w.r.n ? __ldcg(a.logm + rows(e)) : 0.f;
      }
    };
    for (kvcd::MassWalk<128> w(cost, piece); ok && w.next(); ++nk) {
      const kvcd::RowMap rows = kvcd::row_map(a, w.u, w.r.off);
      const int e0 = w.r.first + w.tile * 128, boxes = tile_boxes(rows, e0, w.r.len + w.r.n);
      const int row = tile_row(rows, e0, w.r.len + w.r.n, lane);
      const int ks = nk % kK;
      if (nk >= kK) ok = warp_wait(&sm.k_empty[ks], (uint32_t)((nk / kK - 1) & 1), ns, abort_flag);
      if (!ok) break;
      if (fold && !a.withhold && lane == 0) {
        mbar_expect(&sm.k_full[ks], (uint32_t)(used * 128 * kBlocks));
#pragma unroll
        for (int h = 0; h < kBlocks; ++h)
          tma3d(kvcd::smem_u32(sm.tile[4]) + ks * kFoldPlace + h * kFoldHalf, &qmap, h * 64, w.tb * a.tt, (int)(w.u * a.G),
                &sm.k_full[ks]);
      }
      if (!a.withhold) {
        copy_tile<D>(rows, &kmap, kvcd::smem_u32(sm.tile[ks]), boxes, row, &sm.k_full[ks], lane);
        k_loads = nk + 1;
      }
      if (kMode == kExtra) {                           // the entries' columns: 1 1 1 l0 l1 l2
        if (nk == 0) fetch_lm(w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t l[3];
          split3(lm[j] / a.scale, l);
          ext_store(sm.ext_k[ks], lane + 32 * j, make_uint4(0x3f803f80, 0x3f80 | l[0] << 16, l[1] | l[2] << 16, 0),
                    make_uint4(0, 0, 0, 0));
        }
        kvcd::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) kvcd::mbar_arrive(&sm.k_full[ks]);
        kvcd::MassWalk<128> ahead = w;                 // the next item's, on their way meanwhile
        if (ahead.next()) fetch_lm(ahead);
      }
      for (int rt = w.tb; rt < w.te && !fold; ++rt, ++nq) {
        const int qs = nq % kQ;
        // (kExtra: kQ = kGroups, so a step's query slot is free when its products are there)
        if (nq >= kQ)
          ok = warp_wait(kMode == kExtra ? &sm.s_full[qs] : &sm.q_empty[qs], (uint32_t)((nq / kQ - 1) & 1), ns, abort_flag);
        if (!ok) break;
        if (lane == 0 && !a.withhold) {
          kvcd::mbar_arrive_expect_tx(&sm.q_full[qs], (uint32_t)(used * 128 * kBlocks));
#pragma unroll
          for (int h = 0; h < kBlocks; ++h)
            tma3d(kvcd::smem_u32(sm.tile[kK + qs]) + h * kHalf, &qmap, h * 64, rt * a.tt, (int)(w.u * a.G), &sm.q_full[qs]);
        }
        if (!a.withhold) q_loads = nq + 1;
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    // One thread.  kExtra: it waits for one barrier a step, r_full: the warp that writes the
    // row's extra columns has waited for the query tile, and for the group that read the
    // buffer last.  (Three waits and three commits a step took 1300 cycles against the
    // products' 580.)
    if (elect_one()) {
      int nk = 0, nq = 0;
      bool ok = true;
      const uint32_t lo = desc_lo(kvcd::smem_u32(sm.tile[0]), kLboK), id = idesc(cols, false);
      const uint32_t ek_lo = ext_lo(kvcd::smem_u32(sm.ext_k[0])), eq_lo = ext_lo(kvcd::smem_u32(sm.ext_q[0]));
      for (kvcd::MassWalk<128> w(cost, piece); ok && w.next(); ++nk) {
        const int ks = nk % kK;
        ok = wait_or_abort(&sm.k_full[ks], (uint32_t)((nk / kK) & 1), ns, abort_flag);
        for (int rt = w.tb; ok && rt < w.te; ++rt, ++nq) {
          const int qs = nq % kQ, sb = nq % kGroups;
          if (kMode == kExtra) {
            ok = wait_or_abort(&sm.r_full[sb], (uint32_t)((nq / kGroups) & 1), ns, abort_flag);
          } else {
            ok = fold || wait_or_abort(&sm.q_full[qs], (uint32_t)((nq / kQ) & 1), ns, abort_flag);
            if (ok && nq >= kGroups)
              ok = wait_or_abort(&sm.s_empty[sb], (uint32_t)((nq / kGroups - 1) & 1), ns, abort_flag);
          }
          if (!ok) break;
          fence_after();
          const uint32_t kb = lo + ks * (Smem::kTileBytes >> 4);
          const uint32_t qb = lo + (fold ? 4 * (Smem::kTileBytes >> 4) + ks * (kFoldPlace >> 4)
                                         : (kK + qs) * (Smem::kTileBytes >> 4));
          const uint32_t q_half = (fold ? kFoldHalf : kHalf) >> 4;
          const uint32_t d = tmem + sb * 128;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            mma_ss(d, desc(kb + (k >> 2) * (kHalf >> 4) + (k & 3) * 2), desc(qb + (k >> 2) * q_half + (k & 3) * 2), id, k > 0);
          }
          if (kMode == kExtra) mma_ss(d, ext_desc(ek_lo + ks * 256), ext_desc(eq_lo + sb * 256), id, 1);
          commit(&sm.s_full[sb]);
          if (kMode != kExtra && !fold) commit(&sm.q_empty[qs]);
          if (rt + 1 == w.te) commit(&sm.k_empty[ks]);
        }
      }
    }
    __syncwarp();
  } else if (warp < 4) {
    // ------------------------------------------------------------ row statistics
    int nq = 0;
    bool ok = true;
    int g[4], dt[4];                           // this lane's rows: head and token in the tile
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      g[j] = (lane + 32 * j) / a.tt;
      dt[j] = (lane + 32 * j) % a.tt;
    }
    for (kvcd::MassWalk<128> w(cost, piece); ok && w.next();) {
      // this warp's steps: every other one; their LSEs are fetched a step ahead
      auto lse_at = [&](int j, int rt) {
        const int t = rt * a.tt + dt[j];
        return g[j] < a.G && t < w.r.n ? __ldcg(a.lse + (w.u * a.G + g[j]) * a.T + t) : -INFINITY;
      };
      float next[4], slope[4];
      const int rt0 = w.tb + ((nq & 1) != (warp & 1));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        next[j] = rt0 < w.te ? lse_at(j, rt0) : 0.f;
        slope[j] = kBias && a.slopes && g[j] < a.G ? a.slopes[(w.u % a.H) * a.G + g[j]] * kvcd::kLog2eC : 0.f;
      }
      for (int rt = w.tb; ok && rt < w.te; ++rt, ++nq) {
        if ((nq & 1) != (warp & 1)) continue;
        float nl[4], sl[4], tk[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float lse = next[j];
          tk[j] = (float)dt[j];                        // tokens and positions count from the row tile's first
          sl[j] = slope[j];
          nl[j] = lse != -INFINITY ? -lse - sl[j] * tk[j] : -INFINITY;
          if (rt + 2 < w.te) next[j] = lse_at(j, rt + 2);
        }
        const int b = nq % kGroups;
        uint4 ext[4];                                  // n0 n1 n2 1 1 1 (-lse over the scale)
        if (kMode == kExtra) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t n[3];
            split3(nl[j] / a.scale_log2, n);
            ext[j] = make_uint4(n[0] | n[1] << 16, n[2] | 0x3f800000, 0x3f803f80, 0);
            if (rt * a.tt + dt[j] >= w.r.n) tk[j] = -INFINITY;   // a row past the tokens sees nothing
          }
          ok = warp_wait(&sm.q_full[nq % kQ], (uint32_t)((nq / kQ) & 1), ns, abort_flag);
          if (!ok) break;
        }
        if (nq >= kGroups) ok = warp_wait(&sm.r_empty[b], (uint32_t)((nq / kGroups - 1) & 1), ns, abort_flag);
        if (!ok) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = lane + 32 * j;
          sm.tok[b][r] = tk[j];
          if (kMode == kExtra) {
            ext_store(sm.ext_q[b], r, ext[j], make_uint4(0, 0, 0, 0));
          } else {
            sm.nl[b][r] = nl[j];
            if (kBias) sm.slope[b][r] = sl[j];
          }
        }
        if (kMode == kExtra) kvcd::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) kvcd::mbar_arrive(&sm.r_full[b]);
      }
    }
  } else {
    // ------------------------------------------------------------ weights of the entries
    const int grp = (warp - 4) >> 2, q4 = warp & 3;
    const int key = q4 * 32 + lane;
    const uint32_t ts = tmem + ((uint32_t)(q4 * 32) << 16) + grp * 128;
    int nq = 0;
    uint32_t phase = 0;
    uint32_t joins = 0;                                // key tiles joined so far
    for (kvcd::MassWalk<128> w(cost, piece); w.next();) {
      const int steps = w.te - w.tb;
      const int taker = (nq + steps - 1) % kGroups;    // the group of the last step writes the result
      const int mine = (grp - nq % kGroups + kGroups) % kGroups;   // this group's first step of the item
      const int e0 = w.r.first + w.tile * 128, e = e0 + key, total = w.r.len + w.r.n;
      float lm = 0.f, rel = 0.f, old = 0.f, acc = 0.f;
      int64_t row = 0;
      if (mine < steps || taker == grp) {
        if (e < total) {
          row = kvcd::row_map(a, w.u, w.r.off)(e);
          if (kMode != kExtra) lm = __ldcg(a.logm + row) * kvcd::kLog2eC;
          if (kBias) rel = __ldcg(a.pos + row) - a.pos_new[w.u / a.per_seq];
          if (taker == grp && e < w.r.len) old = a.mass[row];
        }
        uint64_t sum0 = 0, sum1 = 0;
        for (int i = mine; i < steps; i += kGroups) {
          const int t0 = (w.tb + i) * a.tt;
          if (kMode != kExtra) warp_join(&sm.r_full[grp], phase, ns, abort_flag);
          warp_join(&sm.s_full[grp], phase, ns, abort_flag);
          phase ^= 1;
          fence_after();
          const float first_tok = (float)(e - w.r.len - t0);  // tokens from this one on see the entry
          const float rel_t = rel - (float)t0;
          const bool edge = used < 128 || t0 + a.tt > w.r.n || e0 + 127 > w.r.len + t0 ||
                            (kBias && a.window > 0.f && __any_sync(KVC_FULL_MASK, e < total && !(rel_t > (float)a.tt - a.window)));
          if constexpr (kMode == kExtra) {             // 128 columns
            uint32_t s[2][16];
            tld16(ts, s[0]);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              wait_ld(s[q & 1]);
              if (q < 7) tld16(ts + (q + 1) * 16, s[(q + 1) & 1]);
              if (edge) sum16<true>(a, s[q & 1], sm.tok[grp] + q * 16, first_tok, sum0, sum1);
              else sum16<false>(a, s[q & 1], nullptr, 0.f, sum0, sum1);
            }
          } else {
            for (int c = 0; c < cols; c += 16) {
              uint32_t s[16];
              tld16(ts + c, s);
              wait_ld(s);
              const float *nl = sm.nl[grp] + c, *sl = sm.slope[grp] + c, *tk = sm.tok[grp] + c;
              if (edge) add16<kCap, kBias, true>(a, s, nl, sl, tk, lm, rel_t, first_tok, sum0, sum1);
              else add16<kCap, kBias, false>(a, s, nl, sl, tk, lm, rel_t, first_tok, sum0, sum1);
            }
          }
          fence_before();
          __syncwarp();
          if (lane == 0) {
            if (kMode != kExtra) kvcd::mbar_arrive(&sm.s_empty[grp]);
            kvcd::mbar_arrive(&sm.r_empty[grp]);
          }
        }
        float a0, a1;
        upk(add2(sum0, sum1), a0, a1);
        acc = a0 + a1;
      }
      if (steps > 1) {                                 // join the groups' sums in group order
        // every warp announces its sums of join j only after the sums of join j - 1 are read,
        // and the taker reads once all have, so neither barrier can run two phases ahead
        if (joins > 0) warp_wait(&sm.hand_empty, (joins - 1) & 1, ns, abort_flag);
        sm.hand[grp][key] = mine < steps ? acc : 0.f;
        __syncwarp();
        if (lane == 0) kvcd::mbar_arrive(&sm.hand_full);
        if (grp == taker) {
          warp_wait(&sm.hand_full, joins & 1, ns, abort_flag);
          acc = 0.f;
#pragma unroll
          for (int g = 0; g < kGroups; ++g) acc += sm.hand[g][key];
          __syncwarp();
          if (lane == 0) kvcd::mbar_arrive(&sm.hand_empty);
        }
        ++joins;
      }
      if (grp == taker && e < total) {
        if (w.whole()) a.mass[row] = e < w.r.len ? fmaf(a.decay, old, acc) : acc;
        else a.part[((int64_t)blockIdx.x * 2 + (w.tb == 0 ? 1 : 0)) * 128 + key] = acc;
      }
      nq += steps;
    }
  }

  fence_before();
  __syncthreads();
  if (*abort_flag) {                                   // a bounded wait gave up
    if (warp == 0 && lane == 0) {                      // copies still in flight land first
      for (int i = max(0, k_loads - kK); i < k_loads; ++i) kvcd::mbar_wait(&sm.k_full[i % kK], (uint32_t)((i / kK) & 1));
      for (int i = max(0, q_loads - kQ); i < q_loads; ++i) kvcd::mbar_wait(&sm.q_full[i % kQ], (uint32_t)((i / kQ) & 1));
    }
    if (warp == 1 && elect_one()) {                    // and every issued product ends
      commit(&sm.drain);
      kvcd::mbar_wait(&sm.drain, 0);
    }
    __syncthreads();
  }
  fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)kCols) : "memory");
  if (*abort_flag && tid == 0) kvcd::record_error(a.err, KVC_ETIMEOUT);
}

template <int D, int kMode>
cudaError_t launch(const CUtensorMap& km, const CUtensorMap& qm, const ChunkArgs& a, int sms, cudaStream_t s) {
  const size_t smem = sizeof(MassSmem<D>) + 1024;
  cudaError_t e = kvc::chunk_allow_smem<chunk_mass_tc_kernel<D, kMode>>(smem);
  if (e != cudaSuccess) return e;
  kvc::count_launch();
  return kvc::chunk_launch(chunk_mass_tc_kernel<D, kMode>, dim3(sms), dim3(kThreads), smem, s, km, qm, a);
}

template <int D>
cudaError_t launch_mods(const CUtensorMap& km, const CUtensorMap& qm, const ChunkArgs& a, int sms, cudaStream_t s) {
  const bool cap = a.softcap > 0.f, pos = a.slopes || a.window > 0.f;
  if (cap) return pos ? launch<D, kCapPos>(km, qm, a, sms, s) : launch<D, kCapped>(km, qm, a, sms, s);
  if (pos) return launch<D, kPos>(km, qm, a, sms, s);
  return a.T > a.tt ? launch<D, kExtra>(km, qm, a, sms, s) : launch<D, kPlain>(km, qm, a, sms, s);
}

}  // namespace

namespace kvc {

cudaError_t chunk_mass_tc_launch(ChunkArgs& a, int d, int sms, int page_rows, cudaStream_t s) {
  a.tt = std::min(128 / a.G, a.T);
  CUtensorMap km, qm;
  if (!chunk_encode_rows(&km, a.Kp, a.packed_rows, d, page_rows ? std::min(page_rows, 128) : 128) ||
      !chunk_encode_q(&qm, a.q, a.units * a.G, a.T, d, a.tt, a.G))
    return cudaErrorInvalidValue;
  return d == 128 ? launch_mods<128>(km, qm, a, sms, s) : launch_mods<64>(km, qm, a, sms, s);
}

}  // namespace kvc

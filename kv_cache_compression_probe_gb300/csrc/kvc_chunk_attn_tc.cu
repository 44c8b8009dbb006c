// kvc_chunk_attn in bf16 on the tensor cores.
//
// A query row tile is up to 128 rows: tt tokens x G heads of one (b,l,h), so the
// K and V of a KV head are read once for its whole group.  Per 128-entry tile
//   S[128 rows x 128 entries] = Q K^T    (tcgen05, both operands from shared memory)
//   P = 2^(s - m)                        (two threads per row, fp32)
//   O[128 rows x d] += P V               (P as the TMEM operand, V MN-major)
// with the reference m and the sum l of each row in registers.  m need not be
// the maximum, only near enough that nothing over- or underflows: fp32 and bf16
// have the same exponent range, so a reference off by up to 2^30 costs nothing (and
// leaves O room for values up to 2^64: 2^31 a tile, 2^24 tiles, 2^119 in all).
// It starts at 0, a tile takes one pass, and only a row whose maximum lies further
// away has its tile done again and O rescaled.  Tiles go from the newest entries to
// the oldest, so with a distance bias the first tile holds the largest scores.
//
// Two streams of S, P and O alternate, so that the tensor cores work on one
// while the softmax of the other runs:
//   kRowStreams  two row tiles over the same K and V tiles (many rows: the bound
//                is the tensor rate, or the softmax's issue slots);
//   else         one row tile over alternate K/V tiles, joined at the end (few
//                rows: the bound is HBM, and the two streams halve the latency
//                of a tile's chain).
// Warps: 0 copies (TMA), 1 issues the products, 2 and 3 fetch ln m and positions
// of alternate tiles (and 3 clears the V rows past the last entry), 4..11 and 12..19 are the softmax of the two streams.  The
// work is cut as kvc_chunk.cuh says; persistent, one CTA per SM (512 TMEM
// columns: S, S, O, O; P lies in S's place).
// Measured (d 128, G 4): 2048 tokens over 16K entries, 8 KV heads: 371 us, 1390
// TFLOP/s; one token over 256 caches of 3200..5000 entries: 95 us, 5.7 TB/s.
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "kvc_chunk_tc.cuh"

namespace {

using kvc::ChunkArgs;
using kvc::ChunkSeg;
using kvc::ChunkUnit;
using namespace kvctc;

constexpr int kThreads = 640;
constexpr int kBias = 4;               // bias tiles in flight
constexpr float kFar = 0x1p30f;        // half a tile's sum of numerators may be this large or (at first) its inverse
constexpr float kCoarse = 0x1p26f;     // references beyond have steps of 8 and more
constexpr float kLeap = 16.f;          // and then its largest of 64 is above the reference by 24 at least
constexpr int kCols = 512;             // TMEM columns

template <int D>
struct AttnSmem {
  static constexpr int kStages = D == 128 ? 4 : 8;     // K or V tiles in flight: 128 KB
  static constexpr uint32_t kTileBytes = 128 * D * 2;
  alignas(1024) unsigned char q[2][kTileBytes];
  alignas(1024) unsigned char ring[kStages][kTileBytes];
  alignas(16) unsigned char ext_k[kBias][4096];        // the extra step's entry columns, or (capped) base-2 ln m
  alignas(16) unsigned char ext_q[2][4096];            // and row factors
  alignas(16) float rel[kBias][128];                   // position - the row block's first
  float rel_min[kBias];                                // least position of the tile's entries
  int extra[kBias];                                    // the tile needs the extra step
  float xtop[2][2][128], xl[2][2][128];                // what the two halves of a row tell each other
  float m1[128], l1[128];                              // stream 1's statistics (entry streams)
  uint64_t full[kStages], empty[kStages], q_full[2], q_empty[2], bias_full[kBias], bias_empty[kBias];
  uint64_t s_full[2], p_full[2], o_done[2], j_full, j_free, tail_here, cleared, drain;
  kvcd::LocateSmem loc;
  uint32_t tmem;
  int abort;
};

// Where a load or product stands in the ring.
struct Ring {
  int slot, phase;
  __device__ __forceinline__ Ring() : slot(0), phase(0) {}
  template <int N> __device__ __forceinline__ void step() {
    if (++slot == N) { slot = 0; phase ^= 1; }
  }
};

// What a kernel does with the products, by what the call asks for.
//   kSums   ln m and the distance bias are part of the product: an extra 16-wide step
//           of Q K^T adds them (ext_key, ext_row)
//   kWindow the same, and entries beyond the window are left out
//   kCapped the tanh comes between the product and ln m, which is added per score from
//           shared memory
//   kCapPos the same with a distance bias or a window
//   kCapLarge a cap above kShortCap, with or without bias and window
enum Mode { kSums, kWindow, kCapped, kCapPos, kCapLarge };

// Largest cap of the short form cap - 2 cap / (1 + e^2y) of cap tanh(y).  It costs one
// exponential and one reciprocal, but cancels: the score is off by up to 4.5 * 2^-23 of the
// cap (2^-22 of e^2y from ex2, 2^-24 from the sum, 2^-23 from rcp, and two roundings of values
// the cap's size), 3.4e-5 at 64, whatever the score is.  Above, tanh_f costs a polynomial as well
// and is off by 9e-8 of the score.  Short form and tanh_f: drafts over pages 62 and 92 us, one
// token over 256 caches of 3200..5000 entries 126 and 206, 2048 tokens over 16K 666 and 1160.
constexpr float kShortCap = 64.f;

// What a thread needs to turn the products of its row into base-2 scores.
struct RowScore {
  float scale, cap_in, cap_out;        // s log2 e = scale product, or cap_out tanh(y), y = cap_in product
                                       // (short form: 2^(cap_in product) = e^2y)
  float slope, shift;                  // distance bias slope rel - shift
  float edge;                          // window: sees rel > edge
};

// What the base of a row's scores includes of the cap.
template <int kMode>
__device__ __forceinline__ float cap_base(const RowScore& r) {
  return kMode == kCapped || kMode == kCapPos ? r.cap_out : 0.f;
}

// Scores (plus `base`, both halves of a pair; base includes cap_base) of four entries c .. c + 3 of a tile.
// kMask: the row sees only the first `lim` entries, and of these those beyond the
// window's edge.  (A broadcast from shared memory costs its full width, 512 bytes a
// warp for four floats: per-entry values read here bounded the kernel, which is why
// the product carries them.)
template <int kMode, bool kMask>
__device__ __forceinline__ void scores4(const RowScore& r, const uint32_t* s, const float* lm, const float* rel, int c,
                                        uint64_t base, int lim, float (&f)[4]) {
  uint64_t x0 = base, x1 = base;
  float4 d;
  if constexpr (kMode >= kCapPos || (kMode == kWindow && kMask)) d = *reinterpret_cast<const float4*>(rel + c);
  if constexpr (kMode >= kCapped) {
    const float4 b = *reinterpret_cast<const float4*>(lm + c);
    const uint64_t ci = pk(r.cap_in, r.cap_in);
    x0 = add2(pk(b.x, b.y), base);
    x1 = add2(pk(b.z, b.w), base);
    if constexpr (kMode >= kCapPos) {
      const uint64_t sl = pk(r.slope, r.slope);
      x0 = fma2(sl, pk(d.x, d.y), x0);
      x1 = fma2(sl, pk(d.z, d.w), x1);
    }
    float e0, e1, e2, e3;
    upk(mul2(pk(__uint_as_float(s[0]), __uint_as_float(s[1])), ci), e0, e1);
    upk(mul2(pk(__uint_as_float(s[2]), __uint_as_float(s[3])), ci), e2, e3);
    if constexpr (kMode == kCapLarge) {
      const uint64_t co = pk(r.cap_out, r.cap_out);
      x0 = fma2(pk(tanh_f(e0), tanh_f(e1)), co, x0);
      x1 = fma2(pk(tanh_f(e2), tanh_f(e3)), co, x1);
    } else {                                           // cap tanh(y) = cap - 2 cap / (1 + e^2y)
      const uint64_t m2 = pk(-2.f * r.cap_out, -2.f * r.cap_out), one = pk(1.f, 1.f);
      upk(add2(pk(kvcd::ex2(e0), kvcd::ex2(e1)), one), e0, e1);
      upk(add2(pk(kvcd::ex2(e2), kvcd::ex2(e3)), one), e2, e3);
      x0 = fma2(pk(rcp(e0), rcp(e1)), m2, x0);
      x1 = fma2(pk(rcp(e2), rcp(e3)), m2, x1);
    }
  } else {
    const uint64_t sc = pk(r.scale, r.scale);
    x0 = fma2(pk(__uint_as_float(s[0]), __uint_as_float(s[1])), sc, x0);
    x1 = fma2(pk(__uint_as_float(s[2]), __uint_as_float(s[3])), sc, x1);
  }
  upk(x0, f[0], f[1]);
  upk(x1, f[2], f[3]);
  if constexpr (kMask) {
    if constexpr (kMode == kWindow || kMode >= kCapPos) {
      f[0] = d.x > r.edge ? f[0] : -INFINITY;
      f[1] = d.y > r.edge ? f[1] : -INFINITY;
      f[2] = d.z > r.edge ? f[2] : -INFINITY;
      f[3] = d.w > r.edge ? f[3] : -INFINITY;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = c + e < lim ? f[e] : -INFINITY;
  }
}

// Numerators 2^(s - base) of a row over 64 entries of a tile, packed as bf16 pairs;
// returns their sum in fp32, of the unrounded ones (the log-sum-exp goes on to the masses).  The
// product with V takes both operands of one type, and V is bf16; independent roundings of the
// numerators add as much error as that of the result (0.0023 instead of 0.0017 against 64 bits, for any
// number of entries).  A second bf16 part of P would cost the exponentials twice, because 64 numerators
// and their products do not fit this thread's 96 registers, and half as many products again.  The products come from TMEM in blocks of 16, the next
// block on its way while one is worked on.  kApart: the base is
// taken off scores already rounded, as score_max rounds them, so that the largest gives 1 even beyond
// kCoarse (nearer bases come off in the same step as elsewhere, and 0 after it).
template <int kMode, bool kMask, bool kApart = false>
__device__ __forceinline__ float numerators(const RowScore& r, uint32_t ts, const float* lm, const float* rel,
                                            float base, int lim, uint32_t (&p)[32]) {
  const float later = kApart && fabsf(base) > kCoarse ? base : 0.f;
  const float sh = cap_base<kMode>(r) - (base - later + r.shift);
  const uint64_t mb = pk(sh, sh);
  uint64_t s0 = 0, s1 = 0;
  uint32_t s[2][16];
  tld16(ts, s[0]);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    wait_ld(s[q & 1]);
    if (q < 3) tld16(ts + (q + 1) * 16, s[(q + 1) & 1]);
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
      float f[4];
      scores4<kMode, kMask>(r, s[q & 1] + e, lm, rel, q * 16 + e, mb, lim, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = kvcd::ex2(kApart ? f[i] - later : f[i]);
      s0 = add2(s0, pk(f[0], f[1]));
      s1 = add2(s1, pk(f[2], f[3]));
      p[q * 8 + e / 2] = bf16x2(f[0], f[1]);
      p[q * 8 + e / 2 + 1] = bf16x2(f[2], f[3]);
    }
  }
  float a0, a1;
  upk(add2(s0, s1), a0, a1);
  return a0 + a1;
}

// Largest score of a row over 64 entries (rare: kept small).
template <int kMode>
__device__ __forceinline__ float score_max(const RowScore& r, uint32_t ts, const float* lm, const float* rel, int lim) {
  float t = -INFINITY;
  const uint64_t mb = pk(cap_base<kMode>(r) - r.shift, cap_base<kMode>(r) - r.shift);
#pragma unroll 1
  for (int q = 0; q < 64; q += 16) {
    uint32_t s[16];
    tld16(ts + q, s);
    wait_ld(s);
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
      float f[4];
      scores4<kMode, true>(r, s + e, lm, rel, q + e, mb, lim, f);
      t = kvcd::fmax3(t, f[0], f[1]);
      t = kvcd::fmax3(t, f[2], f[3]);
    }
  }
  return t;
}

// The extra step.  Its 16 columns hold, per entry, ln m and the position split into
// bf16 parts (8 bits each, so three parts are the fp32 value) over sqrt(d)'s inverse,
// and per row the factors: 1 for the parts of ln m, the parts of the head's slope for
// those of the position.
// Columns: l0 l1 l2 | r0 r1 r2 r0 r1 | r0 r2 r1
__device__ __forceinline__ void ext_key(unsigned char* tile, int row, float lm, float rel) {
  uint32_t l[3], r[3];
  split3(lm, l);
  split3(rel, r);
  ext_store(tile, row, make_uint4(l[0] | l[1] << 16, l[2] | r[0] << 16, r[1] | r[2] << 16, r[0] | r[1] << 16),
            make_uint4(r[0] | r[2] << 16, r[1], 0, 0));
}
// Factors: 1 1 1 | s0 s0 s0 s1 s1 | s2 s1 s2
__device__ __forceinline__ void ext_row(unsigned char* tile, int row, float slope) {
  uint32_t p[3];
  split3(slope, p);
  constexpr uint32_t one = 0x3f80;
  ext_store(tile, row, make_uint4(one | one << 16, one | p[0] << 16, p[0] | p[0] << 16, p[1] | p[1] << 16),
            make_uint4(p[2] | p[1] << 16, p[2], 0, 0));
}

template <int D, bool kRowStreams, int kMode>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_attn_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                         const __grid_constant__ CUtensorMap qmap, const __grid_constant__ ChunkArgs a) {
  using Smem = AttnSmem<D>;
  constexpr int kStages = Smem::kStages;
  constexpr int kBlocks = D / 64;
  extern __shared__ __align__(1024) unsigned char attn_raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(attn_raw) + 1023) & ~uintptr_t(1023));
  kvcd::pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) { kvcd::mbar_init(&sm.full[i], 1); kvcd::mbar_init(&sm.empty[i], 1); }
    for (int i = 0; i < kBias; ++i) {
      kvcd::mbar_init(&sm.bias_full[i], 1);
      // released by the softmax warps that read it, else by the products
      kvcd::mbar_init(&sm.bias_empty[i], kMode == kSums ? 1 : kRowStreams ? 16 : 8);
    }
    for (int i = 0; i < 2; ++i) {
      kvcd::mbar_init(&sm.q_full[i], kMode < kCapped && a.slopes ? 2 : 1);
      kvcd::mbar_init(&sm.q_empty[i], 1);
      kvcd::mbar_init(&sm.s_full[i], 1);
      kvcd::mbar_init(&sm.p_full[i], 8);
      kvcd::mbar_init(&sm.o_done[i], 1);
    }
    kvcd::mbar_init(&sm.j_full, 4);
    kvcd::mbar_init(&sm.j_free, 8);
    kvcd::mbar_init(&sm.tail_here, 1);
    kvcd::mbar_init(&sm.cleared, 1);
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
  if (kMode < kCapped && !a.slopes) {                 // the same factors for every row
    for (int r = tid; r < 256; r += kThreads) ext_row(sm.ext_q[r >> 7], r & 127, 0.f);
    kvcd::fence_proxy_async_smem();
  }
  fence_before();
  __syncthreads();
  fence_after();
  kvcd::pdl_wait();                                    // the prepare kernel's records and appended rows
  const kvcd::AttnCost<128> cost{a};
  const kvcd::Piece piece = kvcd::locate_piece<kThreads>(cost, sm.loc);
  if (tid == 0) a.seg[blockIdx.x] = ChunkSeg{piece.item, piece.item >= 0 && piece.lo > piece.start};
  const uint32_t tmem = sm.tmem;
  volatile int* abort_flag = &sm.abort;
  const uint64_t ns = a.wait_ns;
  // outstanding copies, for the drain after a give-up: bit i of these = slot i's (or query
  // buffer i's) last copy was issued in phase 0 / 1
  uint32_t issued = 0, issued_phase = 0, q_issued = 0, q_phase = 0;

  if (warp == 0) {
    // ------------------------------------------------------------ copies
    fence_proxy_async_all();
    Ring ring;
    int li = 0;
    bool ok = true;
    for (kvcd::Walk<kvcd::AttnCost<128>> w(cost, piece); ok && w.next(); ++li) {
      const int64_t u = w.item / a.rp;
      const int t0 = (int)(w.item - u * a.rp) * a.tpb;
      const kvcd::RowMap rows = kvcd::row_map(a, u, w.r.off);
      const int total = w.r.len + w.r.n, nt = w.te - w.tb;
      const bool two = kRowStreams && t0 + a.tt < w.r.n;
      const int qb = kRowStreams ? 0 : li & 1, use = kRowStreams ? li : li >> 1;
      // the query rows: their buffer is free once the products before have read it
      if (use > 0) ok = warp_wait(&sm.q_empty[qb], (uint32_t)((use - 1) & 1), ns, abort_flag);
      if (!ok) break;
      if (lane == 0 && !a.withhold) {
        const uint32_t bytes = (uint32_t)(a.G * a.tt * 128 * kBlocks);
        kvcd::mbar_arrive_expect_tx(&sm.q_full[qb], two ? 2 * bytes : bytes);
        for (int i = 0; i < (two ? 2 : 1); ++i)
#pragma unroll
          for (int h = 0; h < kBlocks; ++h)
            tma3d(kvcd::smem_u32(sm.q[kRowStreams ? i : qb]) + h * kHalf, &qmap, h * 64, t0 + i * a.tt, (int)(u * a.G),
                  &sm.q_full[qb]);
        q_issued |= 1u << qb;
        q_phase = (q_phase & ~(1u << qb)) | ((uint32_t)(use & 1) << qb);
      }
      // K and V tiles in the order the products take them: K runs one tile (row
      // streams) or two (entry streams) ahead of V.  Rows are looked up a tile ahead.
      constexpr int kAhead = kRowStreams ? 1 : 2;
      auto first_entry = [&](int t) { return w.r.first + (w.te - 1 - t) * 128; };
      int next = tile_row(rows, first_entry(0), total, lane), row[3] = {0, 0, 0};
      for (int i = 0; ok && i < nt + kAhead; ++i) {
        row[2] = row[1];
        row[1] = row[0];
        row[0] = next;
        if (i + 1 < nt) next = tile_row(rows, first_entry(i + 1), total, lane);
#pragma unroll
        for (int v = 0; v < 2; ++v) {                  // v = 0: V of tile i - kAhead; 1: K of tile i
          const int t = v ? i : i - kAhead;
          if (t < 0 || t >= nt) continue;
          ok = warp_wait(&sm.empty[ring.slot], (uint32_t)(ring.phase ^ 1), ns, abort_flag);
          if (!ok) break;
          if (!a.withhold) {
            copy_tile<D>(rows, v ? &kmap : &vmap, kvcd::smem_u32(sm.ring[ring.slot]),
                         tile_boxes(rows, first_entry(t), total), row[v ? 0 : kAhead], &sm.full[ring.slot], lane);
            issued |= 1u << ring.slot;
            issued_phase = (issued_phase & ~(1u << ring.slot)) | ((uint32_t)ring.phase << ring.slot);
          }
          ring.step<kStages>();
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    // One thread does it all: between two products nothing but the waits for P and for the
    // next K and V tile, which are taken ahead of P.
    if (elect_one()) {
      Ring ring;
      int li = 0;
      uint32_t pphase = 0, cphase = 0;                 // bit s: parity of stream s's next P; of the cleared tails
      bool ok = true;
      // The next K or V tile.  `ahead`: it has been seen to be there (look_ahead, called while
      // the tensor cores are busy, saves the wait's latency when they are not).
      bool ahead[2] = {false, false};
      auto take = [&](int& slot, bool& seen) {
        ok = ok && (seen || wait_or_abort(&sm.full[ring.slot], (uint32_t)ring.phase, ns, abort_flag));
        seen = false;
        slot = ring.slot;
        ring.step<kStages>();
        return ok;
      };
      auto look_ahead = [&](bool two) {
        ahead[0] = mbar_test(&sm.full[ring.slot], (uint32_t)ring.phase);
        if (two) {
          Ring r2 = ring;
          r2.step<kStages>();
          ahead[1] = mbar_test(&sm.full[r2.slot], (uint32_t)r2.phase);
        }
      };
      const uint32_t q_lo = desc_lo(kvcd::smem_u32(sm.q[0]), kLboK), k_lo = desc_lo(kvcd::smem_u32(sm.ring[0]), kLboK);
      const uint32_t v_lo = desc_lo(kvcd::smem_u32(sm.ring[0]), kLboMN);
      constexpr uint32_t kTile16 = Smem::kTileBytes >> 4;        // tile stride in descriptor units
      const uint32_t eq_lo = ext_lo(kvcd::smem_u32(sm.ext_q[0])), ek_lo = ext_lo(kvcd::smem_u32(sm.ext_k[0]));
      int bcnt[2] = {0, 0};                            // bias tiles so far (row streams: [0])
      int bslot = 0;
      bool extra = false, bias_seen = false;
      auto bias_at = [&](int s, int& b, uint32_t& parity) {
        const int c = bcnt[kRowStreams ? 0 : s];
        b = kRowStreams ? c % kBias : s * (kBias / 2) + c % (kBias / 2);
        parity = (uint32_t)((kRowStreams ? c / kBias : c / (kBias / 2)) & 1);
      };
      auto take_bias = [&](int s) {                    // the tile's extra columns
        if (kMode >= kCapped) return ok;
        uint32_t parity;
        bias_at(s, bslot, parity);
        ++bcnt[kRowStreams ? 0 : s];
        ok = ok && (bias_seen || wait_or_abort(&sm.bias_full[bslot], parity, ns, abort_flag));
        bias_seen = false;
        extra = sm.extra[bslot] != 0;
        return ok;
      };
      auto look_bias = [&](int s) {
        if (kMode >= kCapped) return;
        int b;
        uint32_t parity;
        bias_at(s, b, parity);
        bias_seen = mbar_test(&sm.bias_full[b], parity);
      };
      auto qk = [&](int s, int slot, int qtile, int eq, bool last) {   // S_s = Q K^T (+ the extra step)
        const uint32_t qb = q_lo + qtile * kTile16, kb = k_lo + slot * kTile16, d = tmem + s * 128;
        fence_after();
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t at = (k >> 2) * (kHalf >> 4) + (k & 3) * 2;
          mma_ss(d, desc(qb + at), desc(kb + at), idesc(128, false), k > 0);
        }
        if (kMode < kCapped && extra)
          mma_ss(d, ext_desc(eq_lo + eq * 256), ext_desc(ek_lo + bslot * 256), idesc(128, false), 1);
        commit(&sm.s_full[s]);
        if (kMode == kSums && last) commit(&sm.bias_empty[bslot]);
      };
      auto wait_p = [&](int s) {
        ok = ok && wait_or_abort(&sm.p_full[s], (pphase >> s) & 1, ns, abort_flag);
        pphase ^= 1u << s;
        return ok;
      };
      auto pv = [&](int s, int slot, bool first, bool last) {    // O_s += P_s V
        const uint32_t vb = v_lo + slot * kTile16, d = tmem + 256 + s * D, p = tmem + s * 128;
        fence_after();
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_ts(d, p + (k >> 2) * 64 + (k & 3) * 8, desc(vb + k * 128), idesc(D, true), !(first && k == 0));
        if (last) commit(&sm.o_done[s]);
      };
      for (kvcd::Walk<kvcd::AttnCost<128>> w(cost, piece); ok && w.next(); ++li) {
        const int t0 = (int)((unsigned)w.item % (unsigned)a.rp) * a.tpb;
        const int nt = w.te - w.tb;
        const int ns2 = kRowStreams && t0 + a.tt < w.r.n ? 2 : 1;
        const int qb = kRowStreams ? 0 : li & 1, use = kRowStreams ? li : li >> 1;
        // the piece's first V tile holds rows past the last entry: warp 3 clears them
        const bool tail = w.r.len + w.r.n - w.r.first < w.te * 128;
        ok = wait_or_abort(&sm.q_full[qb], (uint32_t)(use & 1), ns, abort_flag);
        int slot = 0;
        bool none = false;
        if (!take(slot, none) || !take_bias(0)) break;
        if constexpr (kRowStreams) {
          for (int s = 0; s < ns2; ++s) qk(s, slot, s, 0, s + 1 == ns2);
          commit(&sm.empty[slot]);
          if (nt == 1) commit(&sm.q_empty[qb]);
          for (int i = 0; ok && i < nt; ++i) {
            int vs = 0, ks = 0;
            if (!take(vs, ahead[0])) break;
            if (i == 0 && tail) kvcd::mbar_arrive(&sm.tail_here);
            if (i + 1 < nt && (!take(ks, ahead[1]) || !take_bias(0))) break;
            if (i == 0 && tail) {
              ok = wait_or_abort(&sm.cleared, cphase, ns, abort_flag);
              cphase ^= 1;
            }
            for (int s = 0; s < ns2; ++s) {
              if (!wait_p(s)) break;
              pv(s, vs, i == 0, i + 1 == nt);
              if (s + 1 == ns2) commit(&sm.empty[vs]);
              if (i + 1 < nt && s == 0) look_ahead(i + 2 < nt);
              if (i + 2 < nt && s == 1) look_bias(0);
              if (i + 1 < nt) {
                qk(s, ks, s, 0, s + 1 == ns2);
                if (s + 1 == ns2) commit(&sm.empty[ks]);
              }
            }
            if (i + 2 == nt) commit(&sm.q_empty[qb]);
          }
        } else {
          qk(0, slot, qb, qb, true);
          commit(&sm.empty[slot]);
          if (nt > 1) {
            if (!take(slot, none) || !take_bias(1)) break;
            qk(1, slot, qb, qb, true);
            commit(&sm.empty[slot]);
          }
          if (nt <= 2) commit(&sm.q_empty[qb]);
          for (int j = 0; ok && j < nt; ++j) {
            const int s = j & 1;
            int ks = 0;
            if (!take(slot, none)) break;
            if (j == 0 && tail) kvcd::mbar_arrive(&sm.tail_here);
            if (j + 2 < nt && (!take(ks, none) || !take_bias(s))) break;
            if (j == 0 && tail) {
              ok = wait_or_abort(&sm.cleared, cphase, ns, abort_flag);
              cphase ^= 1;
            }
            if (!wait_p(s)) break;
            pv(s, slot, j < 2, j + 2 >= nt);
            commit(&sm.empty[slot]);
            if (j + 2 < nt) {
              qk(s, ks, qb, qb, true);
              commit(&sm.empty[ks]);
              if (j + 3 == nt) commit(&sm.q_empty[qb]);
            }
          }
        }
      }
    }
    __syncwarp();
  } else if (warp < 4) {
    // ------------------------------------------------------------ ln m and positions
    if (warp == 3 && a.len_out)
      for (int64_t u = (int64_t)blockIdx.x * 32 + lane; u < a.units; u += (int64_t)gridDim.x * 32) {
        const ChunkUnit r = kvcd::load_unit(a, u);
        const int64_t gu = kvcd::unit_global(a, u);
        a.len_out[gu] = r.n > 0 ? r.len + r.n : a.len_lh[gu];
      }
    // Row streams share a ring of kBias tiles, which the two warps fill in turn; entry streams
    // have a ring of kBias / 2 each, filled by a warp each (a stream that waited for a slot the
    // other one uses could take an old phase for the one it needs).
    int cnt = 0;                                       // tiles so far (entry streams: of this warp's stream)
    int loads = 0;                                     // K and V tiles before this piece
    uint32_t tails = 0;                                // cleared so far
    int li = 0;
    bool ok = true;
    for (kvcd::Walk<kvcd::AttnCost<128>> w(cost, piece); ok && w.next();) {
      const int64_t u = w.item / a.rp;
      const kvcd::RowMap rows = kvcd::row_map(a, u, w.r.off);
      const int total = w.r.len + w.r.n;
      const bool with_pos = a.window > 0.f || a.slopes;
      const int t0 = (int)((unsigned)w.item % (unsigned)a.rp) * a.tpb;
      const float pos0 = with_pos ? a.pos_new[u / a.per_seq] + (float)t0 : 0.f;   // the row block's first token
      if (kMode < kCapped && a.slopes && warp == 2) { // the row factors of this piece's head
        const int qb = kRowStreams ? 0 : li & 1, use = kRowStreams ? li : li >> 1;
        if (use > 0) ok = warp_wait(&sm.q_empty[qb], (uint32_t)((use - 1) & 1), ns, abort_flag);
        if (!ok) break;
        for (int r = lane; r < 128; r += 32) {
          const int g = r / a.tt;
          ext_row(sm.ext_q[qb], r, g < a.G ? a.slopes[(u % a.H) * a.G + g] / a.scale : 0.f);
        }
        kvcd::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) kvcd::mbar_arrive(&sm.q_full[qb]);
      }
      ++li;
      // Warp 3, once its part of the first tile is out of the way: rows past the last entry of
      // the piece's first V tile become zero (P is 0 there, but they may hold anything).
      const int nt = w.te - w.tb, valid = total - w.r.first - (w.te - 1) * 128;
      const int v0 = loads + (kRowStreams || nt == 1 ? 1 : 2);   // the load that brings that tile
      bool tail = warp == 3 && valid < 128;
      loads += 2 * nt;
      auto clear_tail = [&]() {
        tail = false;
        const int slot = v0 % kStages;
        ok = warp_wait(&sm.tail_here, tails & 1, ns, abort_flag);
        if (!ok) return;
        ++tails;
        for (int z = lane; z < (128 - valid) * 8 * kBlocks; z += 32) {
          const int r = valid + z / (8 * kBlocks), h = (z >> 3) & (kBlocks - 1), c = z & 7;
          *reinterpret_cast<uint4*>(sm.ring[slot] + h * kHalf + r * 128 + c * 16) = make_uint4(0, 0, 0, 0);
        }
        kvcd::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) kvcd::mbar_arrive(&sm.cleared);
      };
      for (int t = w.te - 1; ok && t >= w.tb; --t) {
        // (the products take a piece's first tile, or two, before they look for V)
        if (tail && t < w.te - (kRowStreams ? 1 : 2)) clear_tail();
        if (!ok) break;
        const int at = kRowStreams ? cnt++ : w.te - 1 - t;
        if ((at & 1) != (warp & 1)) continue;
        float lm[4], rel[4], low = INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = w.r.first + t * 128 + lane + 32 * j;
          lm[j] = rel[j] = 0.f;
          if (e < total) {
            const int64_t row = rows(e);
            lm[j] = __ldcg(a.logm + row);
            if (with_pos) {
              rel[j] = __ldcg(a.pos + row) - pos0;
              low = fminf(low, rel[j]);
            }
          }
        }
        if (kMode == kWindow) low = -kvcd::warp_max(-low);
        const int b = kRowStreams ? at % kBias : (warp & 1) * (kBias / 2) + cnt % (kBias / 2);
        const int use = kRowStreams ? at / kBias : cnt / (kBias / 2);
        if (!kRowStreams) ++cnt;
        if (use > 0) ok = warp_wait(&sm.bias_empty[b], (uint32_t)((use - 1) & 1), ns, abort_flag);
        if (!ok) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = lane + 32 * j;
          if (kMode >= kCapped) reinterpret_cast<float*>(sm.ext_k[b])[r] = lm[j] * kvcd::kLog2eC;
          else ext_key(sm.ext_k[b], r, lm[j] / a.scale, a.slopes ? rel[j] : 0.f);
          if (kMode == kWindow || kMode >= kCapPos) sm.rel[b][r] = rel[j];
        }
        const bool extra = a.slopes || __any_sync(KVC_FULL_MASK, lm[0] != 0.f || lm[1] != 0.f || lm[2] != 0.f || lm[3] != 0.f);
        if (kMode < kCapped) kvcd::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          sm.extra[b] = extra;
          if (kMode == kWindow) sm.rel_min[b] = low;
          kvcd::mbar_arrive(&sm.bias_full[b]);
        }
      }
      if (ok && tail) clear_tail();
    }
  } else {
    // ------------------------------------------------------------ softmax and output
    // Warps 4..11 and 12..19 are the two streams.  A row belongs to two threads, one for each
    // half of a tile's entries (and of the output's features); their warps meet once a tile at
    // a named barrier of 64 threads.
    const int sw = warp - 4, st = sw >> 3, half = (sw >> 2) & 1, q4 = warp & 3;   // q4: TMEM lane quarter
    const int row = q4 * 32 + lane, pair = 1 + st * 4 + q4;
    const uint32_t tl = tmem + ((uint32_t)(q4 * 32) << 16);
    const uint32_t ts = tl + st * 128 + half * 64, to = tl + 256 + st * D + half * (D / 2);
    uint32_t sphase = 0, ophase[2] = {0, 0};
    int cnt = 0;                                       // bias tiles so far (of this stream's ring)
    // entry streams: stream 1 hands m and l over (j_full) and touches its output again only
    // when stream 0 has read it (j_free); both complete once per joined piece
    uint32_t joins = 0;
    bool joined = false;
    for (kvcd::Walk<kvcd::AttnCost<128>> w(cost, piece); w.next();) {
      const int64_t u = w.item / a.rp;
      const int t0 = (int)(w.item - u * a.rp) * a.tpb + (kRowStreams ? st * a.tt : 0);
      const int tok = t0 + row % a.tt, g = row / a.tt;
      const bool live = g < a.G && tok < w.r.n;
      const bool busy = __any_sync(KVC_FULL_MASK, live);
      const int see = live ? w.r.len + tok + 1 : 0;    // entries this row sees
      RowScore rs;
      rs.scale = a.scale_log2;
      rs.cap_in = kMode == kCapLarge ? a.scale / a.softcap : kMode >= kCapped ? 2.f * a.scale_log2 / a.softcap : 0.f;
      rs.cap_out = kMode >= kCapped ? a.softcap * kvcd::kLog2eC : 0.f;
      rs.slope = a.slopes && live ? a.slopes[(u % a.H) * a.G + g] * kvcd::kLog2eC : 0.f;
      // positions count from the row block's first token, so that near entries, the ones whose
      // bias is small, lose nothing in slope rel - slope tok
      const float tokf = (float)(tok - (int)(w.item - u * a.rp) * a.tpb);
      rs.shift = rs.slope * tokf;
      rs.edge = a.window > 0.f ? tokf - a.window : -INFINITY;
      const int nt = w.te - w.tb;
      const bool mine = !kRowStreams || st == 0 || t0 < w.r.n;     // this stream has work
      float m = 0.f, l = 0.f;                          // the row's reference, and this half's sum
      bool settled = false;                            // the reference fits the entries seen so far
      for (int i = 0; i < nt; ++i) {
        if (!kRowStreams && (i & 1) != st) continue;
        const int b = kRowStreams ? cnt % kBias : st * (kBias / 2) + cnt % (kBias / 2), tile = w.te - 1 - i;
        const int bias_use = cnt / (kRowStreams ? kBias : kBias / 2);
        ++cnt;
        if (kMode != kSums) warp_join(&sm.bias_full[b], (uint32_t)(bias_use & 1), ns, abort_flag);
        if (!mine) {
          if (kMode != kSums && lane == 0) kvcd::mbar_arrive(&sm.bias_empty[b]);
          continue;
        }
        warp_join(&sm.s_full[st], sphase, ns, abort_flag);
        sphase ^= 1;
        fence_after();
        if (busy) {
          // The numerators are taken relative to m at once; if the row's largest score turns
          // out too far away (only ever for its first entries, or after a leap), both halves
          // agree on a new m, rescale O and do the tile again.
          const int lim = live ? see - w.r.first - tile * 128 - half * 64 : 64;
          const float *lm = reinterpret_cast<const float*>(sm.ext_k[b]) + half * 64, *rel = sm.rel[b] + half * 64;
          const bool cut = __any_sync(KVC_FULL_MASK, lim < 64 || (kMode == kWindow && live && !(sm.rel_min[b] > rs.edge)) ||
                                                              (kMode >= kCapPos && a.window > 0.f));
          uint32_t p[32];
          float sum;
          if (cut) sum = numerators<kMode, true>(rs, ts, lm, rel, m, lim, p);
          else sum = numerators<kMode, false>(rs, ts, lm, rel, m, lim, p);
          // the sum tells whether the reference was near enough: above 2^30 (or not a number)
          // it was too low; a row's first sum below 2^-30 may have lost entries
          settled |= l > 0.f;
          // (beyond kCoarse every tile is done again: see there)
          const bool far = live && lim > 0 && (!(sum < kFar) || (!settled && !(sum > 1.f / kFar)) || fabsf(m) > kCoarse);
          if (named_or(pair, 64, far)) {
            const float top = score_max<kMode>(rs, ts, lm, rel, lim);
            sm.xtop[st][half][row] = top;
            sm.xl[st][half][row] = l;
            named_or(pair, 64, false);
            const float t = fmaxf(top, sm.xtop[st][half ^ 1][row]);
            const bool any_seen = l > 0.f || sm.xl[st][half ^ 1][row] > 0.f;
            const bool move = live && t > (any_seen ? m + kLeap : -INFINITY);
            const float f = move ? kvcd::ex2(m - t) : 1.f;
            l = move ? (any_seen ? l * f : 0.f) : l;
            // S is ready, so the product before has ended and O is at rest
            if ((kRowStreams ? i > 0 : i > 1) && __any_sync(KVC_FULL_MASK, move && any_seen)) {
#pragma unroll 1
              for (int c = 0; c < D / 2; c += 16) {
                uint32_t o[16];
                tld16(to + c, o);
                wait_ld(o);
                const float g2 = move && any_seen ? f : 1.f;
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * g2);
                tst16(to + c, o);
              }
            }
            if (move) m = t;
            settled = any_seen || t > -INFINITY;
            // from 2^26 on, half a step of a score (4 and more) is no longer small against kFar: without
            // the rounding in between the largest could come out as 2^256, or as 0.  All further tiles take the
            // rounded scores as well, or equal ones would weigh up to half a step apart (which is left where a row's
            // reference passes 2^26 by a few: 2^4)
            sum = numerators<kMode, true, true>(rs, ts, lm, rel, m, lim, p);
            named_or(pair, 64, false);                 // xtop and xl may be written again
          }
          if (kMode != kSums && lane == 0) kvcd::mbar_arrive(&sm.bias_empty[b]);
          l += sum;
          if (!kRowStreams && st == 1 && joined) {     // stream 0 has read the results before
            warp_join(&sm.j_free, (joins - 1) & 1, ns, abort_flag);
            joined = false;
          }
          tst16(ts, reinterpret_cast<const uint32_t(&)[16]>(p[0]));
          tst16(ts + 16, reinterpret_cast<const uint32_t(&)[16]>(p[16]));
          wait_st();
        } else {
          if (kMode != kSums && lane == 0) kvcd::mbar_arrive(&sm.bias_empty[b]);
          if (!kRowStreams && st == 1 && joined) {
            warp_join(&sm.j_free, (joins - 1) & 1, ns, abort_flag);
            joined = false;
          }
        }
        fence_before();
        __syncwarp();
        if (lane == 0) kvcd::mbar_arrive(&sm.p_full[st]);
      }
      // ---- this piece's result
      const bool whole = w.whole();
      const int64_t slot = ((int64_t)blockIdx.x * 2 + (w.tb == 0 ? 1 : 0)) * (kRowStreams ? 256 : 128) +
                           (kRowStreams ? st * 128 : 0) + row;
      const int64_t orow = (u * a.G + g) * a.T + tok;
      if (kRowStreams ? !mine : (st == 1 && nt == 1)) continue;
      if (busy) {                                      // the row's sum (the halves in order)
        sm.xl[st][half][row] = l;
        named_or(pair, 64, false);
        l = sm.xl[st][0][row] + sm.xl[st][1][row];
        named_or(pair, 64, false);
      }
      if (!(l > 0.f)) m = -INFINITY;
      float f0 = 1.f, f1 = 0.f;
      if constexpr (!kRowStreams) {
        if (nt > 1) {
          if (st == 1) {                               // hand m and l over; stream 0 writes the result
            if (half == 0) {
              sm.m1[row] = m;
              sm.l1[row] = l;
              __syncwarp();
              if (lane == 0) kvcd::mbar_arrive(&sm.j_full);
            }
            ++joins;
            joined = true;
            continue;
          }
          warp_join(&sm.o_done[0], ophase[0], ns, abort_flag);
          warp_join(&sm.o_done[1], ophase[1], ns, abort_flag);
          ophase[0] ^= 1;
          ophase[1] ^= 1;
          warp_join(&sm.j_full, joins & 1, ns, abort_flag);
          const float mb = sm.m1[row], lb = sm.l1[row];
          const float mn = fmaxf(m, mb);
          f0 = m == -INFINITY ? 0.f : kvcd::ex2(m - mn);
          f1 = mb == -INFINITY ? 0.f : kvcd::ex2(mb - mn);
          l = fmaf(l, f0, lb * f1);
          m = mn;
        } else {
          warp_join(&sm.o_done[0], ophase[0], ns, abort_flag);
          ophase[0] ^= 1;
        }
      } else {
        warp_join(&sm.o_done[st], ophase[0], ns, abort_flag);
        ophase[0] ^= 1;
      }
      fence_after();
      const float inv = whole ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
      f0 *= inv;
      f1 *= inv;
      if (busy) {
#pragma unroll 1
        for (int c = 0; c < D / 2; c += 16) {
          uint32_t o[16];
          tld16(to + c, o);
          wait_ld(o);
          float v[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(o[e]) * f0;
          if (!kRowStreams && nt > 1) {
            tld16(to + D + c, o);
            wait_ld(o);
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = fmaf(__uint_as_float(o[e]), f1, v[e]);
          }
          const int at = half * (D / 2) + c;
          uint32_t x[8];
          if (live && whole) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = bf16x2(v[2 * e], v[2 * e + 1]);
            store32(static_cast<__nv_bfloat16*>(a.out) + orow * D + at, x);
          } else if (live) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int e = 0; e < 8; ++e) x[e] = __float_as_uint(v[8 * h + e]);
              store32(a.part + slot * D + at + 8 * h, x);
            }
          }
        }
        if (half == 0 && live && whole && a.lse) a.lse[orow] = l > 0.f ? m + log2f(l) : -INFINITY;
        if (half == 0 && live && !whole) *reinterpret_cast<float2*>(a.part_ml + slot * 2) = make_float2(m, l);
      }
      fence_before();
      if (!kRowStreams && nt > 1) {
        __syncwarp();
        if (lane == 0) kvcd::mbar_arrive(&sm.j_free);
        ++joins;
      }
    }
  }

  fence_before();
  __syncthreads();
  if (*abort_flag) {                                   // a bounded wait gave up
    if (warp == 0 && lane == 0) {                      // copies still in flight land first
      for (int i = 0; i < kStages; ++i)
        if ((issued >> i) & 1) kvcd::mbar_wait(&sm.full[i], (issued_phase >> i) & 1);
      for (int i = 0; i < 2; ++i)
        if ((q_issued >> i) & 1) kvcd::mbar_wait(&sm.q_full[i], (q_phase >> i) & 1);
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

// ---------------------------------------------------------------- host side
PFN_cuTensorMapEncodeTiled_v12000 g_enc = nullptr;
std::once_flag g_enc_once;
PFN_cuTensorMapEncodeTiled_v12000 enc_fn() {
  std::call_once(g_enc_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return g_enc;
}

template <int D, bool kRowStreams, int kMode>
cudaError_t launch(const CUtensorMap& km, const CUtensorMap& vm, const CUtensorMap& qm, const ChunkArgs& a, int sms,
                   cudaStream_t s) {
  const size_t smem = sizeof(AttnSmem<D>) + 1024;
  cudaError_t e = kvc::chunk_allow_smem<chunk_attn_tc_kernel<D, kRowStreams, kMode>>(smem);
  if (e != cudaSuccess) return e;
  kvc::count_launch();
  return kvc::chunk_launch(chunk_attn_tc_kernel<D, kRowStreams, kMode>, dim3(sms), dim3(kThreads), smem, s, km, vm,
                           qm, a);
}

template <int D, bool kRowStreams>
cudaError_t launch_mods(const CUtensorMap& km, const CUtensorMap& vm, const CUtensorMap& qm, const ChunkArgs& a,
                        int sms, cudaStream_t s) {
  if (a.softcap > kShortCap) return launch<D, kRowStreams, kCapLarge>(km, vm, qm, a, sms, s);
  if (a.softcap > 0.f)
    return a.slopes || a.window > 0.f ? launch<D, kRowStreams, kCapPos>(km, vm, qm, a, sms, s)
                                      : launch<D, kRowStreams, kCapped>(km, vm, qm, a, sms, s);
  if (a.window > 0.f) return launch<D, kRowStreams, kWindow>(km, vm, qm, a, sms, s);
  return launch<D, kRowStreams, kSums>(km, vm, qm, a, sms, s);
}

}  // namespace

namespace kvc {

bool chunk_tc_available() { return enc_fn() != nullptr; }

bool chunk_encode_rows(CUtensorMap* m, const void* base, int64_t rows, int d, int box_rows) {
  cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)d * 2};
  cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool chunk_encode_q(CUtensorMap* m, const void* base, int64_t heads, int T, int d, int tt, int G) {
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)T, (cuuint64_t)heads};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)T * d * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)tt, (cuuint32_t)G};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Row tiles of up to 128 rows; a unit with more than one goes by row streams.
cudaError_t chunk_attn_tc_launch(ChunkArgs& a, int d, int sms, int page_rows, cudaStream_t s) {
  a.tt = std::min(128 / a.G, a.T);
  const bool row_streams = a.T > a.tt;
  a.tpb = row_streams ? 2 * a.tt : a.tt;
  a.rp = (a.T + a.tpb - 1) / a.tpb;
  const int box = page_rows ? std::min(page_rows, 128) : 128;
  CUtensorMap km, vm, qm;
  if (!chunk_encode_rows(&km, a.Kp, a.packed_rows, d, box) || !chunk_encode_rows(&vm, a.Vp, a.packed_rows, d, box) ||
      !chunk_encode_q(&qm, a.q, a.units * a.G, a.T, d, a.tt, a.G))
    return cudaErrorInvalidValue;
  if (d == 128)
    return row_streams ? launch_mods<128, true>(km, vm, qm, a, sms, s) : launch_mods<128, false>(km, vm, qm, a, sms, s);
  return row_streams ? launch_mods<64, true>(km, vm, qm, a, sms, s) : launch_mods<64, false>(km, vm, qm, a, sms, s);
}

}  // namespace kvc

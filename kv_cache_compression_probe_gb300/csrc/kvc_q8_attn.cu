// kvc_q8_attn: attention over the 8-bit cache, over all entries or over picked pages.
//
// A warp works by itself, as a rule on every fourth 16-entry group of its CTA's part of an item: groups of codes come through a
// ring in shared memory that the warp fills itself (cp.async, three groups ahead), are turned into fp16 in registers (exact), and
// multiplied with mma.sync in the transposed form, entries or features on the 16-wide side,
// query rows on the 8-wide one:
//   S^T[16 entries x 8 rows] += K[16 x 16 features] Q^T       (d / 16 products)
//   O^T[16 features x 8 rows] += V^T[16 x 16 entries] P^T     (d / 16 products)
// A product's 16 inner positions may stand for any 16 features (or entries), as long as both
// operands agree, so each lane takes whole 16-byte pieces of a row and uses them as they are.
// P goes from the layout of S^T's results to that of P^T's operand by one 8x8 transposition
// (movmatrix) per product.
// Few rows (G heads of one token) fill the 8-wide side, where a tcgen05 product would use
// 4 of its 128 rows and the codes would have to be written to shared memory as bf16 first.
//
// Rows are 16-byte pieces at place piece ^ (row mod 8) of the ring, and row i of a product's 16
// is the group's row i ^ 4 (i & 1): then neither operand's loads have bank conflicts (d 128).
//
// fp16 operands: codes are exact; a query row is scaled by a power of two to a largest
// magnitude in [2^14, 2^15), which leaves bf16 rows exact down to 2^-29 of it (fp32 rows are
// three parts, exact to 2^-33); the softmax's numerators 2^(s - m) are rounded to 11 bits (fp32
// calls: two parts, 22 bits), where m is a loose reference: at first 7 below the largest score, moved when a
// score is more than 15 above it, so that numerators stay below 2^15 and what is lost below
// 2^-24 is under 2^-31 of the largest.  Statistics and O are fp32; O is kept in units of a page's
// scale, and numerators of pages with a scale up to 8 times smaller are scaled down (so 2^-31 becomes 2^-28); for
// others O moves to their unit.  (Neighbouring pages' scales differ by a factor of 2 at most as a rule; with O
// moved at every difference one token over 256 caches, d 64, took 48 us instead of 34.)
//
// The groups of all items (row blocks of units, or picked pages of tokens) lie on one line that is
// cut into equal pieces, one per CTA; a CTA's warps join their results in shared memory, and what a cut
// splits is joined in order by a combine kernel.  Where there is an item for every warp (kSolo) a piece is a warp's, which
// saves the joining and spreads an item's first and last steps over four times as many groups (300 tokens with
// 1024 picked entries each, 8 KV heads: 86 us, with a piece a CTA 91).  Few short items are a cluster's each
// (kTeam), which joins through distributed shared memory and needs no second kernel (one token of one layer
// over 200..512 entries 6.9 us, with pieces and combine 10.6).
// Measured: one token over 256 caches of 3200..5000 entries, d 128, G 4: 53 us, 5.1 TB/s (48.8 without the
// arithmetic, 4 of it the combine kernel); over 4096 caches of 1000..3000: 6.0 TB/s, 90% of the copy rate.  With 20
// rows (16 sequences, up to 5 tokens) 34 us: bound by instructions' latency, since the results of 24 rows leave registers for
// 8 warps an SM.
#include <algorithm>
#include <cfloat>

#include "kvc_chunk_tc.cuh"
#include "kvc_q8.cuh"

namespace {

using kvc::Q8Args;

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr float kBelow = 7.f, kRise = 15.f;            // the reference, and when it moves
constexpr float kNone = -FLT_MAX;                      // the reference of a row that has seen nothing: below every score but -inf
constexpr int kNear = 3;                               // how far below O's unit a page's scale may lie

struct Q8Attn {
  Q8Args x;
  const void* q;
  void* out;
  float* lse;
  const int32_t* sel;                  // null: all entries
  float* part;                         // [CTAs][2][rows][D]
  float2* part_ml;
  int2* tail;                          // [CTAs]: the item a piece leaves unfinished, and its last piece
  float scale_log2;
  int n_sel, tt, rp;                   // tokens per row block, row blocks per unit
  int team;                            // CTAs of an item (kTeam)
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t lo_codes(uint32_t w) { return kvcd::e4m3_f16x2((uint16_t)w); }
__device__ __forceinline__ uint32_t hi_codes(uint32_t w) { return kvcd::e4m3_f16x2((uint16_t)(w >> 16)); }

struct Unit {
  int len, n;                          // entries before the chunk, new tokens (0: nothing to do)
  int64_t gu;
};
// report: whether lengths out of range are this CTA's to report: block 0's, which looks at all units to find its
// piece; of a cluster, which looks at its own unit alone, the first CTA's.
__device__ __forceinline__ Unit load_unit(const Q8Args& x, int64_t u, bool report = blockIdx.x == 0) {
  Unit r;
  r.gu = kvcd::q8_unit_global(x, u);
  r.len = x.len_lh[r.gu];
  r.n = x.len_new[r.gu] - r.len;
  if (r.len < 0 || r.n < 0 || r.n > x.T || (int64_t)r.len + r.n > (int64_t)x.max_pages << x.shift) {
    r.n = 0;
    if (report) kvcd::record_error(x.err, KVC_EDEVICE);
  }
  return r;
}

// 16-entry groups of an item, and its steps.
template <bool kSel>
__device__ __forceinline__ int item_groups(const Q8Attn& a, const Unit& r, int t0) {
  if (t0 >= r.n) return 0;
  if (kSel) return min(a.n_sel, ((r.len + t0) >> a.x.shift) + 1) << (a.x.shift - 4);
  return (r.len + min(r.n, t0 + a.tt) + 15) >> 4;
}

struct LocateSmem {
  long long warp[kWarps];
  long long total, start;
  int item;
};
// Block-wide: this CTA's piece of the line (q groups; kSolo: this warp's), [lo, hi), and the item
// that holds the CTA's first group, with its own first group.
template <bool kSel, bool kSolo>
__device__ __forceinline__ void locate(const Q8Attn& a, LocateSmem& sm, long long& q, long long& lo, long long& hi) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = (int)a.x.units * a.rp;
  const int per = (n + kThreads - 1) / kThreads, i0 = min((long long)n, (long long)tid * per), i1 = min((long long)n, (long long)i0 + per);
  int cu = -1;                                         // the unit looked at last
  Unit cr;
  auto cost = [&](int i) {
    const int u = i / a.rp;
    if (u != cu) cr = load_unit(a.x, cu = u);
    return item_groups<kSel>(a, cr, (i - u * a.rp) * a.tt);
  };
  long long mine = 0;
  long long part[8] = {};                              // of this thread's items in eighths
  const int eighth = (per + 7) / 8;
  if (a.rp == 1) {                                     // an item a unit: eight units' lengths on their way at a time
    for (int k = 0; k < eighth; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = i0 + j * eighth + k;
        if (i < i1) part[j] += item_groups<kSel>(a, load_unit(a.x, i), 0);
      }
#pragma unroll
    for (int j = 0; j < 8; ++j) mine += part[j];
  } else {
    for (int i = i0; i < i1; ++i) mine += cost(i);
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(KVC_FULL_MASK, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sm.warp[warp] = incl;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sm.warp[w];
    total += sm.warp[w];
  }
  constexpr int kPieces = kSolo ? kWarps : 1;           // of a CTA
  const long long all = total + gridDim.x * kPieces - 1;
  q = all >> 31 ? all / (gridDim.x * kPieces) : (long long)((unsigned)all / (gridDim.x * kPieces));
  if (!kSolo) q = max(q, (long long)kWarps);
  lo = min(total, (long long)blockIdx.x * kPieces * q);
  hi = min(total, lo + kPieces * q);
  long long at = before + incl - mine;
  if (lo < hi && at <= lo && lo < at + mine) {
    int i = i0;
    if (a.rp == 1) {                                   // the eighth that holds it
#pragma unroll
      for (int j = 0; j < 7; ++j)
        if (i == i0 + j * eighth && lo >= at + part[j]) {
          at += part[j];
          i += eighth;
        }
    }
    for (; i < i1; ++i) {
      const int c = cost(i);
      if (lo < at + c) {
        sm.item = i;
        sm.start = at;
        break;
      }
      at += c;
    }
  }
  __syncthreads();
  if (kSolo) {
    lo = min(hi, lo + warp * q);
    hi = min(hi, lo + q);
  }
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {   // or zeros

  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// How the groups are shared out: kLine and kSolo as above; kTeam: a cluster an item, whose CTAs join
// their results through distributed shared memory, without a combine kernel.
enum Mode { kLine, kSolo, kTeam };

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(const void* p, int rank) {     // of the same place in another CTA
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(kvcd::smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 cluster_load4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float2 cluster_load2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}

// Shape of a kernel: CTAs per SM, and groups in a warp's ring.
template <typename T, int NT, Mode kMode>
struct Shape {
  static constexpr int kCtas = sizeof(T) != 2 || NT > 2 ? 2 : NT == 1 && kMode == kTeam ? 4 : 3;
  static constexpr int kStages = kCtas == 4 ? 3 : kCtas == 3 ? 4 : 6;
};
template <int D, int kStages>
struct WarpRing {
  static constexpr int kKeys = 16 * D, kStage = 2 * kKeys;       // bytes of a group's keys, of a group
  alignas(128) unsigned char codes[kStages][kStage];             // later this warp's O
  float lm[kStages][16];
};
template <int D, int NT>
struct SharedQ {                       // the query rows as operands, and what their products are in units of
  uint2 words[NT][D / 16][32];
  float units[NT * 8];
};
template <int D>
struct SharedQ<D, 1> {};
template <int D, int NT, int kStages>
struct AttnSmem {
  WarpRing<D, kStages> ring[kWarps];
  SharedQ<D, NT> q;
  float2 ml[kWarps][NT * 8];
  float2 joined[NT * 8];               // of the CTA's warps
  LocateSmem loc;
};

template <typename T, int D, int NT, bool kSel, Mode kMode>
__global__ void __launch_bounds__(kThreads, Shape<T, NT, kMode>::kCtas) q8_attn_kernel(const __grid_constant__ Q8Attn a) {
  constexpr bool kF32 = sizeof(T) == 4;
  constexpr int kQ = kF32 ? 3 : 1, kP = kF32 ? 2 : 1;  // fp16 parts of a query row, of the numerators
  constexpr int kH = D / 64, kS = D / 16;              // 16-byte pieces of a row per lane, products
  constexpr bool kShareQ = NT > 1;
  constexpr int kRows = NT * 8;
  constexpr int kF = D / 8;                            // features of a lane's output
  constexpr int kStages = Shape<T, NT, kMode>::kStages;
  using Smem = AttnSmem<D, NT, kStages>;
  static_assert(kRows * D * 4 <= kStages * WarpRing<D, kStages>::kStage, "O takes the ring's place");
  extern __shared__ __align__(128) unsigned char attn_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(attn_raw);
  const Q8Args& x = a.x;
  kvcd::pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  constexpr int kShare = kMode == kSolo ? 1 : kWarps;  // warps that share an item's groups
  const int me = kMode == kSolo ? 0 : warp, piece = kMode == kSolo ? blockIdx.x * kWarps + warp : blockIdx.x;
  long long q = 0, lo = 0, hi = 0, start = 0;
  int item = 0, left = -1, left_to = 0;
  if constexpr (kMode == kTeam) {                      // this CTA's share of its cluster's item
    item = blockIdx.x / a.team;
    const int rank = blockIdx.x - item * a.team, u0 = item / a.rp;
    const long long n = item_groups<kSel>(a, load_unit(x, u0, rank == 0), (item - u0 * a.rp) * a.tt);
    if (n == 0) return;
    lo = n * rank / a.team;                            // (no group of its own: it takes part in the joining all the same)
    hi = n * (rank + 1) / a.team;
  } else {
    locate<kSel, kMode == kSolo>(a, sm.loc, q, lo, hi);
    start = sm.loc.start;
    item = sm.loc.item;
  }
  bool bad = false;
  WarpRing<D, kStages>& ring = sm.ring[warp];
  const uint32_t codes0 = kvcd::smem_u32(ring.codes), lm0 = kvcd::smem_u32(ring.lm);
  // where this lane's pieces lie in a group's keys and values, and where it copies to
  const int pg = g ^ ((g & 1) << 2);                   // the group's row that stands at row g
  auto place = [](int row, int chunk) {
    return D == 128 ? row * 128 + ((chunk ^ (row & 7)) << 4) : row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
  };
  uint32_t k_at[kH], v_at[2];
#pragma unroll
  for (int h = 0; h < kH; ++h) k_at[h] = place(pg, c + 4 * h);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int row = (2 * c + j) ^ (j << 2);
    v_at[j] = D == 128 ? place(row, g) : place(row, g >> 1) + (g & 1) * 8;
  }
  constexpr int kPer = 32 / (D / 16), kCopies = 16 / kPer;       // rows of one copy instruction, copies
  const int crow = lane / (D / 16), cchunk = lane % (D / 16);
  // (the pieces' places repeat every 8 rows)
  const uint32_t c_first[2] = {(uint32_t)place(crow, cchunk), (uint32_t)place(crow + kPer, cchunk)};
  auto c_at = [&](int i) { return c_first[i * kPer / 4 % 2 * (kPer < 8)] + (i * kPer / 8) * 8 * D; };

  // Four features of a finished row.
  auto put_row = [&](int u, int t0, int row, int f4, float M, float sum, const float4& y) {
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    const int64_t orow = ((int64_t)u * x.G + row / a.tt) * x.T + t0 + row % a.tt;
    T* to = static_cast<T*>(a.out) + orow * D + 4 * f4;
    if constexpr (kF32) *reinterpret_cast<float4*>(to) = make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
    else *reinterpret_cast<uint2*>(to) = make_uint2(kvctc::bf16x2(y.x * inv, y.y * inv), kvctc::bf16x2(y.z * inv, y.w * inv));
    if (a.lse && f4 == 0) a.lse[orow] = sum > 0.f ? M + log2f(sum) : -INFINITY;
  };

  int ru = -1;
  Unit r;
  for (long long at = lo; kMode == kTeam || at < hi;) {
    // the item that holds group `at`
    int u, t0, groups;
    while (true) {
      u = item / a.rp;
      t0 = (item - u * a.rp) * a.tt;
      if (u != ru) r = load_unit(x, ru = u);
      groups = item_groups<kSel>(a, r, t0);
      if (kMode == kTeam || at < start + groups) break;
      start += groups;
      ++item;
    }
    const int tb = (int)(at - start), te = (int)min((long long)groups, hi - start);
    at = start + te;
    const int count = max(0, (te - tb - me + kShare - 1) / kShare);   // this warp's groups
    const int total = r.len + r.n, all_see = r.len + t0 + 1;   // entries; those that every row sees
    const int32_t* tab = x.table + r.gu * x.max_pages;
    const int32_t* list = kSel ? a.sel + ((int64_t)u * x.T + t0) * a.n_sel : nullptr;
    const int own = (r.len + t0) >> x.shift, inpage = (1 << x.shift) - 1;
    if (kSel && tb == 0 && me == 0)                    // places that no group stands for must hold no page
      for (int i = own + 1 + lane; i < a.n_sel; i += 32) bad |= (unsigned)list[i] <= (unsigned)own;
    // A window: lane i knows of the warp's group k0 + i its first entry, its first row (a multiple of 16)
    // and the exponents of its scales; with the latter two whether there is such a group (kThere), and whether every row
    // of the block sees all of it (kFull).
    constexpr int kThere = 1, kFull = 2;
    struct Window { int e0, row, exps; };
    auto window = [&](int k0) {
      Window w{0, 0, 0};
      const int gi = tb + me + kShare * (k0 + lane);
      if (gi < te) {
        w.e0 = gi << 4;
        bool ok = true;
        if (kSel) {
          const int per = x.shift - 4, no = list[gi >> per];
          ok = (unsigned)no <= (unsigned)own;
          w.e0 = (no << x.shift) + ((gi & ((1 << per) - 1)) << 4);
        }
        if (ok) {
          const int page = __ldg(tab + (w.e0 >> x.shift));
          if ((unsigned)page < (unsigned)x.pages) {
            const int flags = kThere | (w.e0 + 16 <= all_see ? kFull : 0);
            w.row = ((page << x.shift) + (w.e0 & inpage)) | flags;
            w.exps = (kvcd::scale_exp(x.k_scale[page]) + 64) | (kvcd::scale_exp(x.v_scale[page]) + 64) << 8 | flags << 16;
          } else {
            bad = true;
          }
        }
      }
      return w;
    };
    Window cur = window(0), nxt = window(32);
    auto entry = [&](const Window& w, int k) {
      return kSel ? __shfl_sync(KVC_FULL_MASK, w.e0, k & 31) : (tb + me + kShare * k) << 4;
    };
    auto issue = [&](int k, int base) {                // base: the first group of `cur`
      if (k < count) {
        const Window& w = k - base < 32 ? cur : nxt;
        const int got = __shfl_sync(KVC_FULL_MASK, w.row, k & 31), row = got & ~15;
        const uint32_t dst = codes0 + (k % kStages) * WarpRing<D, kStages>::kStage, to_lm = lm0 + (k % kStages) * 64 + lane * 4;
        const uint8_t* ks = x.K + (int64_t)row * D + lane * 16;
        const uint8_t* vs = x.V + (int64_t)row * D + lane * 16;
        if (got & kFull) {
#pragma unroll
          for (int i = 0; i < kCopies; ++i) {
            cp_async16(dst + c_at(i), ks + i * 512);
            cp_async16(dst + WarpRing<D, kStages>::kKeys + c_at(i), vs + i * 512);
          }
          if (x.logm && lane < 16) cp_async4(to_lm, x.logm + row + lane, true);
        } else if (got & kThere) {                     // rows past the last entry become 0
          const int e0 = entry(w, k);
#pragma unroll
          for (int i = 0; i < kCopies; ++i) {
            const bool there = e0 + crow + i * kPer < total;
            cp_async16(dst + c_at(i), ks + i * 512, there);
            cp_async16(dst + WarpRing<D, kStages>::kKeys + c_at(i), vs + i * 512, there);
          }
          if (x.logm && lane < 16) cp_async4(to_lm, x.logm + row + lane, e0 + lane < total);
        }
      }
      cp_commit();
    };
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) issue(k, 0);
    // ---- query rows: row nt*8 + g as the operand of this lane, in registers; of several row tiles in
    // shared memory, which the CTA's warps fill together
    uint32_t qr[kQ][kShareQ ? 1 : NT][kS][2];
    float fq[NT][2];
    // Entries that the row of this lane's result column sees (0: a row of no token).
    auto see = [&](int nt, int k) {
      const int row = nt * 8 + 2 * c + k, tok = t0 + row % a.tt;
      return row / a.tt < x.G && tok < r.n ? r.len + tok + 1 : 0;
    };
    auto query_tile = [&](int nt, uint32_t (&qf)[kQ][kS][2]) {   // its operand; returns what the row's products are in units of
      const int row = nt * 8 + g, head = row / a.tt, tok = t0 + row % a.tt;
      const bool live = head < x.G && tok < r.n;
      const T* src = static_cast<const T*>(a.q) + (((int64_t)u * x.G + head) * x.T + tok) * D + 16 * c;
      float v[kH][16], top = 0.f;
#pragma unroll
      for (int h = 0; h < kH; ++h)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          if (live) kvcd::load4(src + h * 64 + i, v[h] + i);
          else v[h][i] = v[h][i + 1] = v[h][i + 2] = v[h][i + 3] = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) top = fmaxf(top, fabsf(v[h][i + k]));
        }
      top = fmaxf(top, __shfl_xor_sync(KVC_FULL_MASK, top, 1));
      top = fmaxf(top, __shfl_xor_sync(KVC_FULL_MASK, top, 2));
      const int e = top > 0.f ? min(max((__float_as_int(top) >> 23) - 127, -80), 80) - 14 : 0;
      const float down = kvcd::pow2i(-e);
#pragma unroll
      for (int h = 0; h < kH; ++h)
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          float y0 = v[h][i] * down, y1 = v[h][i + 1] * down;
#pragma unroll
          for (int k = 0; k < kQ; ++k) {
            const uint32_t w = f16x2(y0, y1);
            qf[k][h * 4 + i / 4][(i >> 1) & 1] = w;
            if (k + 1 < kQ) {
              float z0, z1;
              kvcd::f16x2_f32(w, z0, z1);
              y0 -= z0;
              y1 -= z1;
            }
          }
        }
      return kvcd::pow2i(e) * a.scale_log2;
    };
    if constexpr (kShareQ) {
      for (int nt = warp; nt < NT; nt += kWarps) {
        uint32_t qf[kQ][kS][2];
        const float up = query_tile(nt, qf);
#pragma unroll
        for (int j = 0; j < kS; ++j) sm.q.words[nt][j][lane] = make_uint2(qf[0][j][0], qf[0][j][1]);
        if (c == 0) sm.q.units[nt * 8 + g] = up;
      }
      __syncthreads();
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float up = 0.f;
      if constexpr (!kShareQ) {
        uint32_t qf[kQ][kS][2];
        up = query_tile(nt, qf);
#pragma unroll
        for (int i = 0; i < kQ; ++i)
#pragma unroll
          for (int j = 0; j < kS; ++j) { qr[i][nt][j][0] = qf[i][j][0]; qr[i][nt][j][1] = qf[i][j][1]; }
      }
      // what this lane needs of its result columns, rows nt*8 + 2c and + 1
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if constexpr (kShareQ) fq[nt][k] = sm.q.units[nt * 8 + 2 * c + k];
        else fq[nt][k] = __shfl_sync(KVC_FULL_MASK, up, 8 * c + 4 * k);
      }
    }
    float o[NT][kS][4], ref[NT][2], l[NT][2];
    int xo = 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < kS; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[nt][j][k] = 0.f;
      ref[nt][0] = ref[nt][1] = kNone;
      l[nt][0] = l[nt][1] = 0.f;
    }
    for (int k = 0, base = 0; k < count; ++k) {
      if (k - base == 32) {
        base = k;
        cur = nxt;
        nxt = window(k + 32);
      }
      const int exps = __shfl_sync(KVC_FULL_MASK, cur.exps, k & 31);
      cp_wait<kStages - 2>();
      __syncwarp();
      if (exps & kThere << 16) {
        const unsigned char* st = ring.codes[k % kStages];
        float s[NT][4];
        // ---- S^T = K Q^T
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
        for (int h = 0; h < kH; ++h) {
          const uint4 ka = *reinterpret_cast<const uint4*>(st + k_at[h]), kb = *reinterpret_cast<const uint4*>(st + k_at[h] + 8 * D);
          const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t a0 = lo_codes(wa[w]), a1 = lo_codes(wb[w]), a2 = hi_codes(wa[w]), a3 = hi_codes(wb[w]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = kQ - 1; i >= 0; --i)
                if constexpr (kShareQ) {
                  const uint2 b = sm.q.words[nt][h * 4 + w][lane];
                  mma16816(s[nt], a0, a1, a2, a3, b.x, b.y);
                } else {
                  mma16816(s[nt], a0, a1, a2, a3, qr[i][nt][h * 4 + w][0], qr[i][nt][h * 4 + w][1]);
                }
          }
        }
        // ---- base-2 scores.  The reference comes off them first, exactly for scores near it: where a step of fp32
        // is 2 and more (scores beyond 2^24), reference + 15 would round to a numerator of 2^16, which fp16 does
        // not hold, and reference - `down` to the reference.
        const float ks = kvcd::pow2i((exps & 255) - 64);
        float lm[2] = {0.f, 0.f};
        if (x.logm) {
          lm[0] = ring.lm[k % kStages][pg] * kvcd::kLog2eC;
          lm[1] = ring.lm[k % kStages][pg + 8] * kvcd::kLog2eC;
        }
        bool rise = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float f = fq[nt][i] * ks;
            s[nt][i] = fmaf(s[nt][i], f, lm[0]);
            s[nt][2 + i] = fmaf(s[nt][2 + i], f, lm[1]);
          }
        if (!(exps & kFull << 16)) {
          const int e0 = entry(cur, k);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int lim = see(nt, i) - e0 - pg;
              if (lim <= 0) s[nt][i] = -INFINITY;
              if (lim <= 8) s[nt][2 + i] = -INFINITY;
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) rise |= fmaxf(s[nt][i], s[nt][2 + i]) - ref[nt][i] > kRise;
        if (__any_sync(KVC_FULL_MASK, rise)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float m = fmaxf(s[nt][i], s[nt][2 + i]);
              m = fmaxf(m, __shfl_xor_sync(KVC_FULL_MASK, m, 4));
              m = fmaxf(m, __shfl_xor_sync(KVC_FULL_MASK, m, 8));
              m = fmaxf(m, __shfl_xor_sync(KVC_FULL_MASK, m, 16));
              if (m - ref[nt][i] > kRise) {
                const float f = kvcd::ex2(ref[nt][i] - (m - kBelow));    // 0 at first
                ref[nt][i] = m - kBelow;
                l[nt][i] *= f;
#pragma unroll
                for (int j = 0; j < kS; ++j) {
                  o[nt][j][i] *= f;
                  o[nt][j][2 + i] *= f;
                }
              }
            }
        }
        // ---- numerators, in units of this page's scale over O's
        const int xv = (exps >> 8 & 255) - 64;
        if (xv > xo || xv < xo - kNear) {              // O's unit becomes this page's
          const float f = kvcd::pow2i(xo - xv);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < kS; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) o[nt][j][i] *= f;
          xo = xv;
        }
        const float down = (float)(xv - xo), back = kvcd::pow2i(xo - xv);
        uint32_t pf[kP][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float p[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) p[j] = kvcd::ex2((s[nt][j] - ref[nt][j & 1]) + down);
          l[nt][0] = fmaf(p[0] + p[2], back, l[nt][0]);
          l[nt][1] = fmaf(p[1] + p[3], back, l[nt][1]);
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < kP; ++i) {
              const uint32_t w = f16x2(p[2 * j], p[2 * j + 1]);
              pf[i][nt][j] = transpose8(w);
              if (i + 1 < kP) {
                float z0, z1;
                kvcd::f16x2_f32(w, z0, z1);
                p[2 * j] -= z0;
                p[2 * j + 1] -= z1;
              }
            }
        }
        // ---- O^T += V^T P^T
        uint32_t vw[4][kF / 4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const unsigned char* p = st + WarpRing<D, kStages>::kKeys + v_at[j & 1] + (j >> 1) * 8 * D;
          if constexpr (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(p);
            vw[j][0] = v.x; vw[j][1] = v.y; vw[j][2] = v.z; vw[j][3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            vw[j][0] = v.x; vw[j][1] = v.y;
          }
        }
#pragma unroll
        for (int w = 0; w < kF / 4; ++w)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint32_t ab = __byte_perm(vw[0][w], vw[1][w], hf ? 0x7362 : 0x5140);
            const uint32_t cd = __byte_perm(vw[2][w], vw[3][w], hf ? 0x7362 : 0x5140);
            const uint32_t a0 = lo_codes(ab), a1 = hi_codes(ab), a2 = lo_codes(cd), a3 = hi_codes(cd);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = kP - 1; i >= 0; --i) mma16816(o[nt][2 * w + hf], a0, a1, a2, a3, pf[i][nt][0], pf[i][nt][1]);
          }
      }
      issue(k + kStages - 1, base);
    }
    // ---- the warps' results joined: O in absolute units takes the ring's place
    cp_wait<0>();
    __syncwarp();
    float* mine = reinterpret_cast<float*>(ring.codes);
    const float unit = kvcd::pow2i(xo);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float sum = l[nt][i];
        sum += __shfl_xor_sync(KVC_FULL_MASK, sum, 4);
        sum += __shfl_xor_sync(KVC_FULL_MASK, sum, 8);
        sum += __shfl_xor_sync(KVC_FULL_MASK, sum, 16);
        const int row = nt * 8 + 2 * c + i;
        if (g == 0) sm.ml[warp][row] = make_float2(sum > 0.f ? ref[nt][i] : -INFINITY, sum);
        if (see(nt, i) == 0 || count == 0) continue;
        float* to = mine + row * D + kF * g;
#pragma unroll
        for (int j = 0; j < kS; j += 2)
          *reinterpret_cast<float4*>(to + 2 * j) = make_float4(o[nt][j][i] * unit, o[nt][j][2 + i] * unit,
                                                               o[nt][j + 1][i] * unit, o[nt][j + 1][2 + i] * unit);
      }
    if (kMode == kSolo) __syncwarp();
    else __syncthreads();
    const bool whole = tb == 0 && te == groups;
    if (tb == 0 && te < groups) {
      left = item;
      left_to = (int)((start + groups - 1) / q);
    }
    const int64_t slot = ((int64_t)piece * 2 + (tb == 0 ? 1 : 0)) * kRows;
    constexpr int kVec = D / 4;
    for (int i = kMode == kSolo ? lane : threadIdx.x; i < x.G * a.tt * kVec; i += 32 * kShare) {
      const int row = i / kVec, f4 = i % kVec, tok = t0 + row % a.tt;
      if (tok >= r.n) continue;
      float M = -INFINITY, sum = 0.f;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int j = 0; j < kShare; ++j) M = fmaxf(M, sm.ml[kMode == kSolo ? warp : j][row].x);
#pragma unroll
      for (int j = 0; j < kShare; ++j) {
        const int w = kMode == kSolo ? warp : j;
        const float2 ml = sm.ml[w][row];
        if (ml.x == -INFINITY) continue;               // saw nothing
        const float f = kvcd::ex2(ml.x - M);
        const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(sm.ring[w].codes) + row * D + 4 * f4);
        sum = fmaf(ml.y, f, sum);
        y.x = fmaf(v.x, f, y.x);
        y.y = fmaf(v.y, f, y.y);
        y.z = fmaf(v.z, f, y.z);
        y.w = fmaf(v.w, f, y.w);
      }
      if constexpr (kMode == kTeam) {                  // in place: only this thread uses these
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(sm.ring[0].codes) + row * D + 4 * f4) = y;
        if (f4 == 0) sm.joined[row] = make_float2(M, sum);
      } else if (whole) {
        put_row(u, t0, row, f4, M, sum, y);
      } else {
        *reinterpret_cast<float4*>(a.part + (slot + row) * D + 4 * f4) = y;
        if (f4 == 0) a.part_ml[slot + row] = make_float2(M, sum);
      }
    }
    if constexpr (kMode == kTeam) {
      cluster_sync();
      const int rank = blockIdx.x - item * a.team;
      for (int i = rank * kThreads + threadIdx.x; i < x.G * a.tt * kVec; i += a.team * kThreads) {
        const int row = i / kVec, f4 = i % kVec;
        if (t0 + row % a.tt >= r.n) continue;
        float M = -INFINITY, sum = 0.f;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < a.team; ++w) {
          const float2 ml = cluster_load2(cluster_addr(&sm.joined[row], w));
          const float4 v = cluster_load4(cluster_addr(reinterpret_cast<const float*>(sm.ring[0].codes) + row * D + 4 * f4, w));
          if (ml.x == -INFINITY) continue;             // saw nothing
          const float Mn = fmaxf(M, ml.x), f0 = kvcd::ex2(M - Mn), f1 = kvcd::ex2(ml.x - Mn);
          sum = fmaf(sum, f0, ml.y * f1);
          y.x = fmaf(y.x, f0, v.x * f1);
          y.y = fmaf(y.y, f0, v.y * f1);
          y.z = fmaf(y.z, f0, v.z * f1);
          y.w = fmaf(y.w, f0, v.w * f1);
          M = Mn;
        }
        put_row(u, t0, row, f4, M, sum, y);
      }
      cluster_sync();                                  // nobody leaves while others read from it
      break;
    }
    if (kMode == kSolo) __syncwarp();
    else __syncthreads();                              // the ring is free again
  }
  if (kMode == kSolo ? lane == 0 : kMode == kLine && threadIdx.x == 0) a.tail[piece] = make_int2(left, left_to);
  // The next kernel's CTAs may come in from here: any earlier and they take registers that
  // this kernel's or its successor's CTAs need (70 us instead of 53 for one token, all layers).
  kvcd::pdl_trigger();
  if (bad) kvcd::record_error(x.err, KVC_EDEVICE);
}

// Joins the partial results of the item that piece blockIdx.x leaves unfinished: the head in
// its slot 1, the others in slot 0 of the pieces up to the last.  blockIdx.y takes as many rows as
// the block has warps; where an item has fewer, several warps share a row's pieces.
template <typename T, int D, int kRows>
__global__ void __launch_bounds__(256) q8_combine_kernel(const __grid_constant__ Q8Attn a) {
  constexpr int C = D / 32;
  __shared__ float sm_o[8][D];
  __shared__ float2 sm_ml[8];
  kvcd::pdl_wait();
  const int2 tail = a.tail[blockIdx.x];
  if (tail.x < 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = blockDim.x >> 5, rows = min(warps, a.x.G * a.tt - (int)blockIdx.y * warps);   // of this block
  if (rows <= 0) return;
  const int share = warps / rows, row = blockIdx.y * warps + warp % rows, part = warp / rows;
  const int u = tail.x / a.rp, t0 = (tail.x - u * a.rp) * a.tt;
  const int head = row / a.tt, tok = t0 + row % a.tt;
  float M = -INFINITY, l = 0.f, o[C];
#pragma unroll
  for (int i = 0; i < C; ++i) o[i] = 0.f;
  auto add = [&](float2 ml, const float (&v)[C]) {
    if (ml.x == -INFINITY) return;
    const float Mn = fmaxf(M, ml.x), f0 = kvcd::ex2(M - Mn), f1 = kvcd::ex2(ml.x - Mn);
    l = fmaf(l, f0, ml.y * f1);
#pragma unroll
    for (int i = 0; i < C; ++i) o[i] = fmaf(o[i], f0, v[i] * f1);
    M = Mn;
  };
  const Unit r = load_unit(a.x, u);
  const bool live = part < share && tok < r.n;
  if (live)
    for (int p0 = blockIdx.x + part; p0 <= tail.y; p0 += 4 * share) {
      float2 ml[4];
      float v[4][C];
#pragma unroll
      for (int k = 0; k < 4; ++k) {                    // four pieces on their way at a time
        const int p = p0 + k * share;
        const int64_t slot = ((int64_t)min(p, tail.y) * 2 + (p == (int)blockIdx.x ? 1 : 0)) * kRows + row;
        ml[k] = a.part_ml[slot];
#pragma unroll
        for (int i = 0; i < C; ++i) v[k][i] = a.part[slot * D + lane * C + i];
        if (p > tail.y) ml[k].x = -INFINITY;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) add(ml[k], v[k]);
    }
  if (share > 1) {
#pragma unroll
    for (int i = 0; i < C; ++i) sm_o[warp][lane * C + i] = o[i];
    if (lane == 0) sm_ml[warp] = make_float2(M, l);
    __syncthreads();
    if (part > 0) return;
    for (int k = 1; k < share; ++k) {
      float v[C];
#pragma unroll
      for (int i = 0; i < C; ++i) v[i] = sm_o[warp + k * rows][lane * C + i];
      add(sm_ml[warp + k * rows], v);
    }
  }
  if (!live) return;
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const int64_t orow = ((int64_t)u * a.x.G + head) * a.x.T + tok;
  T* to = static_cast<T*>(a.out) + orow * D + lane * C;
#pragma unroll
  for (int i = 0; i < C; ++i) to[i] = kvcd::from_f<T>(o[i] * inv);
  if (a.lse && lane == 0) a.lse[orow] = l > 0.f ? M + log2f(l) : -INFINITY;
}

// ---------------------------------------------------------------- host side
struct Layout {
  size_t part, ml, tail, total;
};

// Row tiles of 8 rows: one for picked pages and fp32, else as many as the rows of a unit take, up to 4.
int row_tiles(const kvc_params* p, const kvc_chunk* c, int n_sel) {
  return p->dtype == KVC_F32 || n_sel > 0 ? 1 : std::min(4, (p->G * std::min(c->T, 32) + 7) / 8);
}
int ctas_per_sm(const kvc_params* p, int nt, bool team = false) { return p->dtype == KVC_F32 || nt > 2 ? 2 : nt == 1 && team ? 4 : 3; }

// Tokens of a row block, and items of a call.
int block_tokens(const kvc_params* p, const kvc_chunk* c, int n_sel) {
  return n_sel > 0 ? 1 : std::min(row_tiles(p, c, n_sel) * 8 / p->G, c->T);
}
int64_t item_count(const kvc_params* p, const kvc_chunk* c, int n_sel) {
  const int tt = block_tokens(p, c, n_sel);
  return (int64_t)p->B * p->H * (c->layer_end - c->layer_begin) * ((c->T + tt - 1) / tt);
}

// Whether a piece is a warp's: one row tile, and an item at least for every warp of the grid (bf16: 1824 on 152 SMs).
// A CTA's piece and a warp's, us: 1024 picked entries a token, 1840 items 75 and 67, 3200 items 117 and 107; 256 picked
// entries, 1840 items 39 and 33; one token over 2048 caches of 100..150 entries 36 and 30, of 400..600 63 and 62, of
// 1000..3000 169 and 178 (the lengths are not known here); fp32, 1200 items of 500..1000 entries 81 and 71.  Below, with
// fewer items than warps, the two come closer (480 items of 1024 picked entries 21.7 and 21.8).
bool solo(const kvc_params* p, const kvc_chunk* c, int n_sel) {
  const int nt = row_tiles(p, c, n_sel);
  return nt == 1 && item_count(p, c, n_sel) >= (int64_t)std::max(kvc::sm_count(), 1) * ctas_per_sm(p, nt) * kWarps;
}

// CTAs that take an item as a cluster, or 0: where the items are few, and short by what the pages (picked, or of
// the table) hold at most.  A warp then has kTeamGroups groups to do at most; a longer
// item wants more CTAs than a cluster has.  Pieces with a combine kernel and clusters, us, one token of one layer, by groups a
// warp: 8 (4000 entries) 16.8 and 10.4, 16 18.3 and 14.1, 23 18.6 and 18.0, 31 20.8 and 21.4, 47 21.8 and 29.3; with 2 KV
// heads 31 28.3 and 21.5, 47 30.0 and 29.1; 5 tokens, 31 31.2 and 30.7; fp32 16 18.1 and 18.0, 31 21.1 and 29.1.
constexpr int kTeamGroups = 32;
int team_size(const kvc_params* p, const kvc_chunk* c, int n_sel) {
  const int64_t items = item_count(p, c, n_sel);
  const int64_t groups = (int64_t)(n_sel > 0 ? std::min(n_sel, c->max_pages) : c->max_pages) * (c->page_rows / 16);
  const int64_t room = (int64_t)std::max(kvc::sm_count(), 1) * ctas_per_sm(p, row_tiles(p, c, n_sel), true);
  int team = 8;
  while (team > 1 && items * team > room) team /= 2;
  if (items * team > room || groups > (int64_t)team * kWarps * kTeamGroups) return 0;
  while (team > 1 && groups <= team / 2 * kWarps) team /= 2;   // no more than there are groups for
  return team;
}

// Whether the rows go to the kernel of kvc_chunk_attn (kvc_q8_chunk.cu): more than kManyRows of a unit, and more
// than kShortWork groups to do here, by what the table's pages hold at most.  Here and there (8 KV heads, G 4): 64 rows over
// 16384 entries 40 and 39 us, 128 rows 63 and 43, 8192 rows 2360 and 378; by groups: 256 rows over 2000
// entries (8.3 K groups) 22 and 30, 128 rows of 8 sequences over 500 (8.7 K) 24 and 30, 256 rows (18 K) 51 and 38,
// 68 rows of 8 sequences over 2000 (24 K) 47 and 41, 96 rows over 14000 (21 K) 43 and 40.
constexpr int kManyRows = 64;
constexpr int64_t kShortWork = 12288;
bool many_rows(const kvc_params* p, const kvc_chunk* c, int n_sel) {
  return p->dtype == KVC_BF16 && n_sel == 0 && p->G * c->T > kManyRows &&
         item_count(p, c, n_sel) * c->max_pages * (c->page_rows / 16) > kShortWork;
}

Layout layout(const kvc_params* p, const kvc_chunk* c, int n_sel) {
  const int nt = row_tiles(p, c, n_sel);
  const size_t pieces = (size_t)std::max(kvc::sm_count(), 1) * ctas_per_sm(p, nt) * (solo(p, c, n_sel) ? kWarps : 1);
  const size_t rows = pieces * 2 * nt * 8;
  Layout w;
  w.part = 0;
  w.ml = kvc::align256(rows * p->d * sizeof(float));
  w.tail = w.ml + kvc::align256(rows * sizeof(float2));
  w.total = w.tail + kvc::align256(pieces * sizeof(int2));
  return w;
}

template <typename T, int D, int NT, bool kSel, Mode kMode>
cudaError_t launch_mode(const Q8Attn& a, int sms, cudaStream_t s) {
  const size_t smem = sizeof(AttnSmem<D, NT, Shape<T, NT, kMode>::kStages>);
  cudaError_t e = kvc::chunk_allow_smem<q8_attn_kernel<T, D, NT, kSel, kMode>>(smem);
  if (e != cudaSuccess) return e;
  kvc::count_launch();
  if (kMode == kTeam) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.x.units * a.rp * a.team));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)a.team;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, q8_attn_kernel<T, D, NT, kSel, kMode>, a);
  }
  const int grid = sms * Shape<T, NT, kMode>::kCtas;
  e = kvc::chunk_launch(q8_attn_kernel<T, D, NT, kSel, kMode>, dim3(grid), dim3(kThreads), smem, s, a);
  if (e != cudaSuccess) return e;
  kvc::count_launch();
  // (kSolo: many items of few pieces, so a warp a row)
  const int warps = kMode == kSolo ? 4 : 8;
  return kvc::chunk_launch(q8_combine_kernel<T, D, NT * 8>, dim3(kMode == kSolo ? grid * kWarps : grid, NT * 8 / warps),
                           dim3(32 * warps), 0, s, a);
}

template <typename T, int D, int NT, bool kSel>
cudaError_t launch(const Q8Attn& a, bool alone, int sms, cudaStream_t s) {
  if (a.team > 0) return launch_mode<T, D, NT, kSel, kTeam>(a, sms, s);
  if constexpr (NT == 1)
    if (alone) return launch_mode<T, D, NT, kSel, kSolo>(a, sms, s);
  return launch_mode<T, D, NT, kSel, kLine>(a, sms, s);
}

template <int D>
cudaError_t launch_d(const kvc_params* p, const Q8Attn& a, int nt, bool alone, int sms, cudaStream_t s) {
  using B = __nv_bfloat16;
  if (p->dtype == KVC_F32) return a.sel ? launch<float, D, 1, true>(a, alone, sms, s) : launch<float, D, 1, false>(a, alone, sms, s);
  if (a.sel) return launch<B, D, 1, true>(a, alone, sms, s);
  return nt == 1 ? launch<B, D, 1, false>(a, alone, sms, s) : nt == 2 ? launch<B, D, 2, false>(a, alone, sms, s)
       : nt == 3 ? launch<B, D, 3, false>(a, alone, sms, s) : launch<B, D, 4, false>(a, alone, sms, s);
}

}  // namespace

extern "C" size_t kvc_q8_workspace_bytes(const kvc_params* p, const kvc_chunk* c, int32_t n_sel) {
  if (kvc::chunk_check(p, c) != KVC_OK || c->page_rows < 16 || c->page_rows > 128 || n_sel < 0) return 0;
  return many_rows(p, c, n_sel) ? kvc::q8_chunk_bytes(p, c) : layout(p, c, n_sel).total;
}

extern "C" int kvc_q8_attn(const kvc_params* p, const kvc_chunk* c, const kvc_q8* x, const void* q,
                           const int32_t* len_lh, const int32_t* len_new, const int32_t* sel, int32_t n_sel,
                           void* out, float* lse, void* workspace, size_t ws_bytes, void* stream) {
  const int st = kvc::q8_check(p, c, x);
  if (st != KVC_OK) return st;
  if (!q || !len_lh || !len_new || !out || n_sel < 0 || (sel != nullptr) != (n_sel > 0)) return KVC_EINVAL;
  if (kvc::q8_misaligned(q, 16) || kvc::q8_misaligned(out, 32)) return KVC_EINVAL;
  const bool many = many_rows(p, c, n_sel);
  const Layout w = layout(p, c, n_sel);
  if (!workspace || ws_bytes < (many ? kvc::q8_chunk_bytes(p, c) : w.total) || kvc::q8_misaligned(workspace, 256))
    return KVC_EWORKSPACE;
  Q8Attn a = {};
  kvc::q8_fill(a.x, p, c, x);
  const int sms = kvc::sm_count();
  if (!a.x.err || sms <= 0) return KVC_ECUDA;
  a.x.len_lh = len_lh;
  a.x.len_new = len_new;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (many) {
    if (a.x.units * c->max_pages >= (1LL << 31)) return KVC_EINVAL;
    if (!kvc::chunk_tc_available()) return KVC_ECUDA;
    return kvc::cuda_status(kvc::q8_chunk_launch(p, c, a.x, q, out, lse, workspace, s));
  }
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.sel = sel;
  a.n_sel = n_sel;
  char* ws = static_cast<char*>(workspace);
  a.part = reinterpret_cast<float*>(ws + w.part);
  a.part_ml = reinterpret_cast<float2*>(ws + w.ml);
  a.tail = reinterpret_cast<int2*>(ws + w.tail);
  a.scale_log2 = kvcd::kLog2eC / sqrtf((float)p->d);
  const int nt = row_tiles(p, c, n_sel);
  const bool alone = solo(p, c, n_sel);
  a.team = team_size(p, c, n_sel);
  a.tt = block_tokens(p, c, n_sel);
  a.rp = (c->T + a.tt - 1) / a.tt;
  if (a.x.units * a.rp >= (1LL << 31)) return KVC_EINVAL;
  return kvc::cuda_status(p->d == 128 ? launch_d<128>(p, a, nt, alone, sms, s) : launch_d<64>(p, a, nt, alone, sms, s));
}

// kvc_q8_attn: attention over the 8-bit cache, over all entries or over picked pages.
//
// A warp works by itself: it streams 16-entry groups of codes from global memory into
// registers, turns them into fp16 there (exact), and multiplies with mma.sync in the
// transposed form, entries or features on the 16-wide side, query rows on the 8-wide one:
//   S^T[16 entries x 8 rows] += K[16 x 16 features] Q^T       (d / 16 products)
//   O^T[16 features x 8 rows] += V^T[16 x 16 entries] P^T     (d / 16 products)
// A product's 16 inner positions may stand for any 16 features (or entries), as long as both
// operands agree, so each lane loads whole 16-byte pieces of a row and uses them as they are:
// nothing passes through shared memory.  P goes from the layout of S^T's results to that of
// P^T's operand by one 8x8 transposition (movmatrix) per product.
// Few rows (G heads of one token) fill the 8-wide side, where a tcgen05 product would use
// 4 of its 128 rows and the codes would have to be written to shared memory as bf16 first.
//
// fp16 operands: codes are exact; a query row is scaled by a power of two to a largest
// magnitude in [2^14, 2^15), which leaves bf16 rows exact down to 2^-29 of it (fp32 rows are
// three parts, exact to 2^-33); the softmax's numerators 2^(s - m) are rounded to 11 bits (fp32
// calls: two parts, 22 bits), where m is a loose reference: at first 7 below the largest score, moved when a
// score is more than 15 above it, so that numerators stay below 2^15 and what is lost below
// 2^-24 is under 2^-31 of the largest.  Statistics and O are fp32; O is kept in units of the
// scale of the values that came last, and moved by a power of two when that changes.
//
// The steps of all items (rows blocks of units, or picked pages of tokens) lie on one line that is cut into equal
// pieces, one per warp; what a cut splits is joined in order by a combine kernel.
#include <algorithm>

#include "kvc_q8.cuh"

namespace {

using kvc::Q8Args;

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr float kBelow = 7.f, kRise = 15.f;            // the reference, and when it moves

struct Q8Attn {
  Q8Args x;
  const void* q;
  void* out;
  float* lse;
  const int32_t* sel;                  // null: all entries
  float* part;                         // [pieces][2][rows][D]
  float2* part_ml;
  int2* tail;                          // [pieces]: the item a piece leaves unfinished, and its last piece
  float scale_log2;
  int n_sel, tt, rp;                   // tokens per row block, row blocks per unit
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
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
__device__ __forceinline__ Unit load_unit(const Q8Args& x, int64_t u) {
  Unit r;
  r.gu = kvcd::q8_unit_global(x, u);
  r.len = __ldg(x.len_lh + r.gu);
  r.n = __ldg(x.len_new + r.gu) - r.len;
  if (r.len < 0 || r.n < 0 || r.n > x.T || (int64_t)r.len + r.n > (int64_t)x.max_pages << x.shift) {
    r.n = 0;
    if (blockIdx.x == 0) kvcd::record_error(x.err, KVC_EDEVICE);
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
// Block-wide: the total of steps, and the item that holds step lo (or -1), with its first step.
template <int kGroups, bool kSel>
__device__ __forceinline__ void locate(const Q8Attn& a, long long pieces, LocateSmem& sm, long long& q) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = (int)a.x.units * a.rp;
  const int per = (n + kThreads - 1) / kThreads, i0 = min((long long)n, (long long)tid * per), i1 = min((long long)n, (long long)i0 + per);
  auto cost = [&](int i) {
    const int u = i / a.rp;
    const Unit r = load_unit(a.x, u);
    return (item_groups<kSel>(a, r, (i - u * a.rp) * a.tt) + kGroups - 1) / kGroups;
  };
  long long mine = 0;
#pragma unroll 4
  for (int i = i0; i < i1; ++i) mine += cost(i);
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(KVC_FULL_MASK, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sm.warp[warp] = incl;
  if (tid == 0) sm.item = -1;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sm.warp[w];
    total += sm.warp[w];
  }
  q = (total + pieces - 1) / pieces;
  const long long lo = (long long)blockIdx.x * kWarps * q;
  long long at = before + incl - mine;
  if (at <= lo && lo < at + mine) {
    for (int i = i0; i < i1; ++i) {
      const int c = cost(i);
      if (lo < at + c) {
        sm.item = i;
        sm.start = at;
        break;
      }
      at += c;
    }
  }
  if (tid == 0) sm.total = total;
  __syncthreads();
}

// A lane's share of a group's codes: of K, 16-byte pieces h of rows g and g + 8; of V, the
// features 16 g' (8 g' for d 64) of rows 2c, 2c+1, 2c+8, 2c+9 (lane = 4 g + c, g' = g).
template <int D>
struct KFrag { uint4 w[2][D / 64]; };
template <int D> struct VFrag;
template <> struct VFrag<128> { uint4 w[4]; };
template <> struct VFrag<64> { uint2 w[4]; };

template <typename T, int D, int NT, int kGroups, bool kSel>
__global__ void __launch_bounds__(kThreads, NT == 1 && sizeof(T) == 2 ? 3 : 2)
    q8_attn_kernel(const __grid_constant__ Q8Attn a) {
  constexpr bool kF32 = sizeof(T) == 4;
  constexpr int kQ = kF32 ? 3 : 1, kP = kF32 ? 2 : 1;  // fp16 parts of a query row, of the numerators
  constexpr int kH = D / 64, kS = D / 16;              // 16-byte pieces of a row per lane, products
  constexpr int kRows = NT * 8;
  constexpr int kF = D / 8;                            // features of a lane's output
  __shared__ LocateSmem sm;
  const Q8Args& x = a.x;
  kvcd::pdl_trigger();
  kvcd::pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const long long pieces = (long long)gridDim.x * kWarps;
  const int piece = blockIdx.x * kWarps + warp;
  long long q;
  locate<kGroups, kSel>(a, pieces, sm, q);
  const long long lo = min(sm.total, (long long)piece * q), hi = min(sm.total, lo + q);
  long long start = sm.start;
  int item = sm.item, left = -1, left_to = 0;
  bool bad = false;
  for (long long at = lo; at < hi;) {
    // the item that holds step `at`
    Unit r;
    int u, t0, groups, tiles;
    while (true) {
      u = item / a.rp;
      t0 = (item - u * a.rp) * a.tt;
      r = load_unit(x, u);
      groups = item_groups<kSel>(a, r, t0);
      tiles = (groups + kGroups - 1) / kGroups;
      if (at < start + tiles) break;
      start += tiles;
      ++item;
    }
    const int tb = (int)(at - start), te = (int)min((long long)tiles, hi - start);
    at = start + te;
    // ---- query rows: row nt*8 + g as the operand of this lane
    uint32_t qf[kQ][NT][kS][2];
    float fq[NT][2];
    int see[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = nt * 8 + g, head = row / a.tt, tok = t0 + row % a.tt;
      const bool live = head < x.G && tok < r.n;
      const T* src = static_cast<const T*>(a.q) + (((int64_t)u * x.G + head) * x.T + tok) * D + 16 * c;
      float v[kH][16], top = 0.f;
#pragma unroll
      for (int h = 0; h < kH; ++h)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          if (live) kvcd::VecLoad<T, 4>::ld(src + h * 64 + i, v[h] + i);
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
            qf[k][nt][h * 4 + i / 4][(i >> 1) & 1] = w;
            if (k + 1 < kQ) {
              float z0, z1;
              kvcd::f16x2_f32(w, z0, z1);
              y0 -= z0;
              y1 -= z1;
            }
          }
        }
      // what this lane needs of its result columns, rows nt*8 + 2c and + 1
      const float up = kvcd::pow2i(e) * a.scale_log2;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        fq[nt][k] = __shfl_sync(KVC_FULL_MASK, up, 8 * c + 4 * k);
        const int row2 = nt * 8 + 2 * c + k, tok2 = t0 + row2 % a.tt;
        see[nt][k] = row2 / a.tt < x.G && tok2 < r.n ? r.len + tok2 + 1 : 0;
      }
    }
    const int total = r.len + r.n, all_see = r.len + t0 + 1;   // entries; those that every row sees
    const int32_t* tab = x.table + r.gu * x.max_pages;
    const int32_t* list = kSel ? a.sel + ((int64_t)u * x.T + t0) * a.n_sel : nullptr;
    const int own = (r.len + t0) >> x.shift;
    // first entry of a group, or -1 for none
    auto entry_of = [&](int gi) {
      if (gi >= groups) return -1;
      if (!kSel) return gi << 4;
      const int per = x.shift - 4, no = __ldg(list + (gi >> per));
      return (unsigned)no <= (unsigned)own ? (no << x.shift) + ((gi & ((1 << per) - 1)) << 4) : -1;
    };
    auto page_of = [&](int e) {
      const int page = e >= 0 ? __ldg(tab + (e >> x.shift)) : 0;
      if ((unsigned)page < (unsigned)x.pages) return page;
      bad = true;
      return 0;
    };
    KFrag<D> kf[kGroups];
    VFrag<D> vf[kGroups];
    float ks[kGroups], vs[kGroups], lm[kGroups][2];
    int e0[kGroups] = {}, page[kGroups] = {}, e0n[kGroups], pagen[kGroups];
    const int inpage = (1 << x.shift) - 1;
    auto load_k = [&](int i) {
      const int64_t row = ((int64_t)page[i] << x.shift) + (e0[i] & inpage);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint8_t* p = x.K + (row + g + 8 * j) * D + 16 * c;
#pragma unroll
        for (int h = 0; h < kH; ++h)
          kf[i].w[j][h] = e0[i] >= 0 ? __ldg(reinterpret_cast<const uint4*>(p + 64 * h)) : make_uint4(0, 0, 0, 0);
        lm[i][j] = x.logm && e0[i] >= 0 ? __ldg(x.logm + row + g + 8 * j) : 0.f;
      }
      ks[i] = __ldg(x.k_scale + page[i]);
    };
    auto load_v = [&](int i) {
      const int64_t row = ((int64_t)page[i] << x.shift) + (e0[i] & inpage);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint8_t* p = x.V + (row + 2 * c + (j & 1) + 8 * (j >> 1)) * D + kF * g;
        if constexpr (D == 128) vf[i].w[j] = e0[i] >= 0 ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
        else vf[i].w[j] = e0[i] >= 0 ? __ldg(reinterpret_cast<const uint2*>(p)) : make_uint2(0, 0);
      }
      vs[i] = __ldg(x.v_scale + page[i]);
    };
    float o[NT][kS][4], ref[NT][2], l[NT][2];
    int xo = 0;
    bool any_v = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < kS; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[nt][j][k] = 0.f;
      ref[nt][0] = ref[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      e0[i] = entry_of(tb * kGroups + i);
      page[i] = page_of(e0[i]);
      load_k(i);
      load_v(i);
      e0n[i] = tb + 1 < te ? entry_of((tb + 1) * kGroups + i) : -1;
      pagen[i] = page_of(e0n[i]);
    }
    for (int tile = tb; tile < te; ++tile) {
      float s[kGroups][NT][4];
      // ---- S^T = K Q^T
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[i][nt][0] = s[i][nt][1] = s[i][nt][2] = s[i][nt][3] = 0.f;
#pragma unroll
        for (int h = 0; h < kH; ++h) {
          const uint32_t wa[4] = {kf[i].w[0][h].x, kf[i].w[0][h].y, kf[i].w[0][h].z, kf[i].w[0][h].w};
          const uint32_t wb[4] = {kf[i].w[1][h].x, kf[i].w[1][h].y, kf[i].w[1][h].z, kf[i].w[1][h].w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t a0 = lo_codes(wa[w]), a1 = lo_codes(wb[w]), a2 = hi_codes(wa[w]), a3 = hi_codes(wb[w]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int k = kQ - 1; k >= 0; --k)
                mma16816(s[i][nt], a0, a1, a2, a3, qf[k][nt][h * 4 + w][0], qf[k][nt][h * 4 + w][1]);
          }
        }
      }
      // ---- base-2 scores
      int ecur[kGroups];
      float vcur[kGroups];
      bool rise = false;
      float mx[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mx[nt][0] = mx[nt][1] = -INFINITY;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        ecur[i] = e0[i];
        const bool cut = e0[i] < 0 || e0[i] + 16 > all_see;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float f = fq[nt][k] * ks[i];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float y = fmaf(s[i][nt][2 * j + k], f, lm[i][j] * kvcd::kLog2eC);
              if (cut) y = e0[i] >= 0 && e0[i] + g + 8 * j < see[nt][k] ? y : -INFINITY;
              s[i][nt][2 * j + k] = y;
              mx[nt][k] = fmaxf(mx[nt][k], y);
            }
          }
      }
      // the next step's keys are on their way from here
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        vcur[i] = vs[i];
        e0[i] = e0n[i];
        page[i] = pagen[i];
        load_k(i);
        e0n[i] = tile + 2 < te ? entry_of((tile + 2) * kGroups + i) : -1;
        pagen[i] = page_of(e0n[i]);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) rise |= mx[nt][0] > ref[nt][0] + kRise || mx[nt][1] > ref[nt][1] + kRise;
      if (__any_sync(KVC_FULL_MASK, rise)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float m = mx[nt][k];
            m = fmaxf(m, __shfl_xor_sync(KVC_FULL_MASK, m, 4));
            m = fmaxf(m, __shfl_xor_sync(KVC_FULL_MASK, m, 8));
            m = fmaxf(m, __shfl_xor_sync(KVC_FULL_MASK, m, 16));
            if (m > ref[nt][k] + kRise) {
              const float f = kvcd::ex2(ref[nt][k] - (m - kBelow));      // 0 at first
              ref[nt][k] = m - kBelow;
              l[nt][k] *= f;
#pragma unroll
              for (int j = 0; j < kS; ++j) {
                o[nt][j][k] *= f;
                o[nt][j][2 + k] *= f;
              }
            }
          }
      }
      // ---- numerators, and O^T += V^T P^T
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        uint32_t pf[kP][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float b0 = ref[nt][0] == -INFINITY ? 0.f : ref[nt][0], b1 = ref[nt][1] == -INFINITY ? 0.f : ref[nt][1];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float p0 = kvcd::ex2(s[i][nt][2 * j] - b0), p1 = kvcd::ex2(s[i][nt][2 * j + 1] - b1);
            l[nt][0] += p0;
            l[nt][1] += p1;
#pragma unroll
            for (int k = 0; k < kP; ++k) {
              const uint32_t w = f16x2(p0, p1);
              pf[k][nt][j] = transpose8(w);
              if (k + 1 < kP) {
                float z0, z1;
                kvcd::f16x2_f32(w, z0, z1);
                p0 -= z0;
                p1 -= z1;
              }
            }
          }
        }
        if (ecur[i] >= 0) {
          const int xv = kvcd::scale_exp(vcur[i]);
          if (any_v && xv != xo) {                     // O's unit becomes this page's
            const float f = kvcd::pow2i(xo - xv);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < kS; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[nt][j][k] *= f;
          }
          xo = xv;
          any_v = true;
          if (ecur[i] + 16 > total) {                  // rows past the last entry may hold anything
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (ecur[i] + 2 * c + (j & 1) + 8 * (j >> 1) >= total) {
                vf[i].w[j].x = vf[i].w[j].y = 0;
                if constexpr (D == 128) vf[i].w[j].z = vf[i].w[j].w = 0;
              }
          }
        }
#pragma unroll
        for (int w = 0; w < kF / 4; ++w) {
          auto word = [&](int j) {
            if constexpr (D == 128) return w == 0 ? vf[i].w[j].x : w == 1 ? vf[i].w[j].y : w == 2 ? vf[i].w[j].z : vf[i].w[j].w;
            else return w == 0 ? vf[i].w[j].x : vf[i].w[j].y;
          };
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint32_t ab = __byte_perm(word(0), word(1), hf ? 0x7362 : 0x5140);
            const uint32_t cd = __byte_perm(word(2), word(3), hf ? 0x7362 : 0x5140);
            const uint32_t a0 = lo_codes(ab), a1 = hi_codes(ab), a2 = lo_codes(cd), a3 = hi_codes(cd);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int k = kP - 1; k >= 0; --k) mma16816(o[nt][2 * w + hf], a0, a1, a2, a3, pf[k][nt][0], pf[k][nt][1]);
          }
        }
        load_v(i);
      }
    }
    // ---- this piece's result
    const bool whole = tb == 0 && te == tiles;
    if (tb == 0 && te < tiles) {
      left = item;
      left_to = (int)((start + tiles - 1) / q);
    }
    const int64_t slot = ((int64_t)piece * 2 + (tb == 0 ? 1 : 0)) * kRows;
    const float unit = kvcd::pow2i(xo);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float sum = l[nt][k];
        sum += __shfl_xor_sync(KVC_FULL_MASK, sum, 4);
        sum += __shfl_xor_sync(KVC_FULL_MASK, sum, 8);
        sum += __shfl_xor_sync(KVC_FULL_MASK, sum, 16);
        const int row = nt * 8 + 2 * c + k;
        if (see[nt][k] == 0) continue;
        const float f = whole ? (sum > 0.f ? unit / sum : 0.f) : unit;
        const float m = sum > 0.f ? ref[nt][k] : -INFINITY;
        float y[kF];
#pragma unroll
        for (int j = 0; j < kS; ++j) {
          y[2 * j] = o[nt][j][k] * f;
          y[2 * j + 1] = o[nt][j][2 + k] * f;
        }
        if (whole) {
          const int64_t orow = ((int64_t)u * x.G + row / a.tt) * x.T + t0 + row % a.tt;
          T* to = static_cast<T*>(a.out) + orow * D + kF * g;
#pragma unroll
          for (int i = 0; i < kF; i += 8) {
            if constexpr (kF32) {
              *reinterpret_cast<float4*>(to + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
              *reinterpret_cast<float4*>(to + i + 4) = make_float4(y[i + 4], y[i + 5], y[i + 6], y[i + 7]);
            } else {
              uint4 w;
              w.x = __bfloat16_as_ushort(__float2bfloat16_rn(y[i])) | (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(y[i + 1])) << 16;
              w.y = __bfloat16_as_ushort(__float2bfloat16_rn(y[i + 2])) | (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(y[i + 3])) << 16;
              w.z = __bfloat16_as_ushort(__float2bfloat16_rn(y[i + 4])) | (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(y[i + 5])) << 16;
              w.w = __bfloat16_as_ushort(__float2bfloat16_rn(y[i + 6])) | (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(y[i + 7])) << 16;
              *reinterpret_cast<uint4*>(to + i) = w;
            }
          }
          if (a.lse && g == 0) a.lse[orow] = sum > 0.f ? m + log2f(sum) : -INFINITY;
        } else {
          float* to = a.part + (slot + row) * D + kF * g;
#pragma unroll
          for (int i = 0; i < kF; i += 4) *reinterpret_cast<float4*>(to + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
          if (g == 0) a.part_ml[slot + row] = make_float2(m, sum);
        }
      }
  }
  if (lane == 0) a.tail[piece] = make_int2(left, left_to);
  if (bad && lane == 0) kvcd::record_error(x.err, KVC_EDEVICE);
}

// Joins the partial results of the item that piece blockIdx.x leaves unfinished: the head in
// its slot 1, the others in slot 0 of the pieces up to the last.  A warp a row.
template <typename T, int D, int kRows>
__global__ void __launch_bounds__(256) q8_combine_kernel(const __grid_constant__ Q8Attn a) {
  constexpr int C = D / 32;
  kvcd::pdl_trigger();
  kvcd::pdl_wait();
  const int2 tail = a.tail[blockIdx.x];
  if (tail.x < 0) return;
  const int lane = threadIdx.x & 31, row = blockIdx.y * 8 + (threadIdx.x >> 5);
  const int u = tail.x / a.rp, t0 = (tail.x - u * a.rp) * a.tt;
  const int head = row / a.tt, tok = t0 + row % a.tt;
  const Unit r = load_unit(a.x, u);
  if (head >= a.x.G || tok >= r.n) return;
  float M = -INFINITY, l = 0.f, o[C];
#pragma unroll
  for (int i = 0; i < C; ++i) o[i] = 0.f;
#pragma unroll 4
  for (int p = blockIdx.x; p <= tail.y; ++p) {
    const int64_t slot = ((int64_t)p * 2 + (p == (int)blockIdx.x ? 1 : 0)) * kRows + row;
    const float2 ml = a.part_ml[slot];
    float v[C];
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = a.part[slot * D + lane * C + i];
    if (ml.x == -INFINITY) continue;
    const float Mn = fmaxf(M, ml.x), f0 = kvcd::ex2(M - Mn), f1 = kvcd::ex2(ml.x - Mn);
    l = fmaf(l, f0, ml.y * f1);
#pragma unroll
    for (int i = 0; i < C; ++i) o[i] = fmaf(o[i], f0, v[i] * f1);
    M = Mn;
  }
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

// Row tiles of 8 rows and the CTAs per SM: one tile for picked pages, fp32, and up to 8 rows.
int row_tiles(const kvc_params* p, const kvc_chunk* c, int n_sel) {
  return p->dtype == KVC_F32 || n_sel > 0 || p->G * c->T <= 8 ? 1 : 2;
}
int ctas_per_sm(const kvc_params* p, int nt) { return nt == 1 && p->dtype == KVC_BF16 ? 3 : 2; }

Layout layout(const kvc_params* p, const kvc_chunk* c, int n_sel) {
  const int nt = row_tiles(p, c, n_sel);
  const size_t pieces = (size_t)std::max(kvc::sm_count(), 1) * ctas_per_sm(p, nt) * kWarps, rows = pieces * 2 * nt * 8;
  Layout w;
  w.part = 0;
  w.ml = kvc::align256(rows * p->d * sizeof(float));
  w.tail = w.ml + kvc::align256(rows * sizeof(float2));
  w.total = w.tail + kvc::align256(pieces * sizeof(int2));
  return w;
}

template <typename T, int D, int NT, int kGroups, bool kSel>
cudaError_t launch(const Q8Attn& a, int grid, cudaStream_t s) {
  kvc::count_launch();
  cudaError_t e = kvc::chunk_launch(q8_attn_kernel<T, D, NT, kGroups, kSel>, dim3(grid), dim3(kThreads), 0, s, a);
  if (e != cudaSuccess) return e;
  kvc::count_launch();
  return kvc::chunk_launch(q8_combine_kernel<T, D, NT * 8>, dim3(grid * kWarps, NT), dim3(256), 0, s, a);
}

template <int D>
cudaError_t launch_d(const kvc_params* p, const Q8Attn& a, int nt, int grid, cudaStream_t s) {
  if (p->dtype == KVC_F32)
    return a.sel ? launch<float, D, 1, 1, true>(a, grid, s) : launch<float, D, 1, 1, false>(a, grid, s);
  if (a.sel) return launch<__nv_bfloat16, D, 1, 2, true>(a, grid, s);
  if (nt == 1) return launch<__nv_bfloat16, D, 1, 2, false>(a, grid, s);
  return launch<__nv_bfloat16, D, 2, 1, false>(a, grid, s);
}

}  // namespace

extern "C" size_t kvc_q8_workspace_bytes(const kvc_params* p, const kvc_chunk* c, int32_t n_sel) {
  if (kvc::chunk_check(p, c) != KVC_OK || c->page_rows < 16 || c->page_rows > 128 || n_sel < 0) return 0;
  return layout(p, c, n_sel).total;
}

extern "C" int kvc_q8_attn(const kvc_params* p, const kvc_chunk* c, const kvc_q8* x, const void* q,
                           const int32_t* len_lh, const int32_t* len_new, const int32_t* sel, int32_t n_sel,
                           void* out, float* lse, void* workspace, size_t ws_bytes, void* stream) {
  const int st = kvc::q8_check(p, c, x);
  if (st != KVC_OK) return st;
  if (!q || !len_lh || !len_new || !out || n_sel < 0 || (sel != nullptr) != (n_sel > 0)) return KVC_EINVAL;
  if (kvc::q8_misaligned(q, 16) || kvc::q8_misaligned(out, 32)) return KVC_EINVAL;
  const Layout w = layout(p, c, n_sel);
  if (!workspace || ws_bytes < w.total || kvc::q8_misaligned(workspace, 256)) return KVC_EWORKSPACE;
  Q8Attn a = {};
  kvc::q8_fill(a.x, p, c, x);
  const int sms = kvc::sm_count();
  if (!a.x.err || sms <= 0) return KVC_ECUDA;
  a.x.len_lh = len_lh;
  a.x.len_new = len_new;
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
  a.tt = n_sel > 0 ? 1 : std::min(nt * 8 / p->G, c->T);
  a.rp = (c->T + a.tt - 1) / a.tt;
  if (a.x.units * a.rp >= (1LL << 31)) return KVC_EINVAL;
  const int grid = sms * ctas_per_sm(p, nt);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return kvc::cuda_status(p->d == 128 ? launch_d<128>(p, a, nt, grid, s) : launch_d<64>(p, a, nt, grid, s));
}

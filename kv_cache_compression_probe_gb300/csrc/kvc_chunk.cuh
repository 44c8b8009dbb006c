// What the chunk kernels share (kvc_chunk_attn, kvc_chunk_mass, kvc_mass_evict):
// the argument block, row addressing of contiguous and paged caches, and the
// split of the work over the CTAs.
//
// A unit is one (b,l,h) of the layer range; its record (entries before the
// chunk, new tokens, first row) is written by the prepare kernel, with n = 0 for
// a unit that is skipped.  An item is one unit's row block (attention) or key
// tile (mass); it costs as many steps as it has key tiles (row tiles).  The
// steps of all items lie on one line, which is cut into equal pieces, one per
// CTA: every CTA has the same work to within one step whatever the lengths are,
// and an item that crosses a cut leaves one partial result per CTA, which a
// combine kernel joins in CTA order (so results do not depend on timing).
#pragma once
#include <atomic>
#include <utility>

#include "kvc_common.cuh"

namespace kvc {

struct ChunkUnit {                     // as stored: 16 bytes (len, n, off)
  int32_t len, n;                      // entries before the chunk, new tokens (0: skipped)
  int64_t off;                         // first row (contiguous cache)
  int32_t first;                       // entries below this 128-multiple are outside every token's window
};

// Where a CTA's piece of the step line starts: the item, and whether inside it.
struct ChunkSeg {
  int64_t item, mid;
};

struct ChunkArgs {
  const void* q;
  const void* k_new;                   // null: nothing to append (mass)
  const void* v_new;
  const float* pos_new;
  void* Kp;
  void* Vp;
  float* logm;
  float* pos;
  const int32_t* len_lh;
  const int32_t* cap_lh;               // null: no capacity is checked (mass only)
  const int64_t* off_lh;
  void* out;
  float* lse;                          // attention: written when not null; mass: read
  int32_t* len_out;
  float* mass;
  const int32_t* page_table;           // null: contiguous
  const int32_t* n_new;                // null: T
  const float* slopes;
  // workspace
  int4* rec;                           // [units] records (store_unit / load_unit)
  int32_t* first;                      // [units], written and read when there is a window
  ChunkSeg* seg;                       // [grid]
  float* part;                         // per CTA two slots (kvc_chunk.cu)
  float* part_ml;
  int32_t* err;
  int64_t packed_rows, units;
  int64_t lh_span, lh_gap, lh_base;    // layer range, as lh_global
  int T, H, G, per_seq;                // per_seq: units of one sequence
  int max_pages, page_shift;
  int tt, tpb, rp;                     // tokens per row tile, tokens per row block, row blocks per unit
  float scale, scale_log2, softcap, window, decay;
  uint64_t wait_ns;
  int withhold;
};

}  // namespace kvc

namespace kvcd {

constexpr float kLog2eC = 1.4426950408889634f;

__device__ __forceinline__ int64_t unit_global(const kvc::ChunkArgs& a, int64_t u) {
  return u + (u / a.lh_span) * a.lh_gap + a.lh_base;
}

// Row of entry e of a unit.
struct RowMap {
  const int32_t* table;
  int64_t off;
  int shift;
  __device__ __forceinline__ int64_t operator()(int e) const {
    if (!table) return off + e;
    return ((int64_t)__ldg(table + (e >> shift)) << shift) + (e & ((1 << shift) - 1));
  }
};
__device__ __forceinline__ RowMap row_map(const kvc::ChunkArgs& a, int64_t u, int64_t off) {
  RowMap m;
  m.table = a.page_table ? a.page_table + unit_global(a, u) * a.max_pages : nullptr;
  m.off = off;
  m.shift = a.page_shift;
  return m;
}

__device__ __forceinline__ void store_unit(const kvc::ChunkArgs& a, int64_t u, int len, int n, int64_t off) {
  a.rec[u] = make_int4(len, n, (int)(uint32_t)off, (int)(off >> 32));
}
__device__ __forceinline__ kvc::ChunkUnit load_unit(const kvc::ChunkArgs& a, int64_t u) {
  const int4 v = __ldcg(a.rec + u);
  kvc::ChunkUnit r;
  r.len = v.x;
  r.n = v.y;
  r.off = ((int64_t)(uint32_t)v.z) | ((int64_t)v.w << 32);
  r.first = a.window > 0.f ? __ldcg(a.first + u) : 0;
  return r;
}

// Steps of attention item i: key tiles of kTile entries from the unit's first
// visible one to the row block's last token; 0 past the unit's tokens.
template <int kTile>
struct AttnCost {
  const kvc::ChunkArgs& a;
  __device__ __forceinline__ int items() const { return (int)a.units * a.rp; }   // below 2^31 (chunk_check)
  __device__ __forceinline__ int operator()(int i, kvc::ChunkUnit& r) const {
    r = load_unit(a, (int)((unsigned)i / (unsigned)a.rp));
    return of(i, r);
  }
  __device__ __forceinline__ int of(int i, const kvc::ChunkUnit& r) const {   // r: the item's record
    const int t0 = (int)((unsigned)i % (unsigned)a.rp) * a.tpb;
    if (t0 >= r.n) return 0;
    return (r.len + min(r.n, t0 + a.tpb) + kTile - 1) / kTile - r.first / kTile;
  }
};

// Block-wide: this CTA's piece [lo, hi) of the step line and the item that holds
// step lo, with that item's first step and its unit's record.  item = -1 for an
// empty piece.
struct Piece {
  long long lo, hi, start;
  kvc::ChunkUnit r;
  int item;
};
struct LocateSmem {
  long long warp[32];
  Piece piece;
};
template <int kThreads, class Cost>
__device__ Piece locate_piece(const Cost& cost, LocateSmem& sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = cost.items();
  const int per = (int)((unsigned)(n + kThreads - 1) / kThreads);
  const int i0 = min((long long)n, (long long)tid * per), i1 = min((long long)n, (long long)i0 + per);
  kvc::ChunkUnit r;
  r.len = r.n = r.first = 0;
  r.off = 0;
  long long mine = 0;
#pragma unroll 4
  for (int i = i0; i < i1; ++i) mine += cost(i, r);
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
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += sm.warp[w];
    total += sm.warp[w];
  }
  const long long all = total + gridDim.x - 1;
  const long long q = all >> 31 ? all / gridDim.x : (long long)((unsigned)all / gridDim.x);
  const long long lo = min(total, (long long)blockIdx.x * q), hi = min(total, lo + q);
  long long at = before + incl - mine;
  if (lo >= hi) {
    if (tid == 0) sm.piece = Piece{lo, hi, 0, r, -1};
  } else if (at <= lo && lo < at + mine) {
    if (per == 1) {                                    // r is that item's record already
      sm.piece = Piece{lo, hi, at, r, i0};
    } else {
      for (int i = i0; i < i1; ++i) {
        const int64_t c = cost(i, r);
        if (lo < at + c) {
          sm.piece = Piece{lo, hi, at, r, i};
          break;
        }
        at += c;
      }
    }
  }
  __syncthreads();
  return sm.piece;
}

// Walks the items of a piece: for (Walk w(cost, piece); w.next(); ) visits the
// steps [w.tb, w.te) of item w.item, of its w.tiles.
template <class Cost>
struct Walk {
  const Cost& cost;
  Piece p;
  kvc::ChunkUnit r;
  int item, tb, te, tiles;
  bool begun;
  __device__ __forceinline__ Walk(const Cost& c, const Piece& pc) : cost(c), p(pc), r(pc.r), item(pc.item), begun(false) {}
  __device__ __forceinline__ bool next() {
    if (begun) {
      p.start += tiles;
      ++item;
    }
    if (p.item < 0 || p.start >= p.hi) return false;
    if (begun) {
      while ((tiles = cost(item, r)) == 0) ++item;    // a step follows: p.start < p.hi <= all steps
    } else {
      tiles = cost.of(item, r);
    }
    tb = begun ? 0 : (int)(p.lo - p.start);
    te = (int)min((long long)tiles, p.hi - p.start);
    begun = true;
    return true;
  }
  __device__ __forceinline__ bool whole() const { return tb == 0 && te == tiles; }
};

// Mass: the items of a unit are its key tiles, their steps the unit's row tiles.
// The line is located by unit; inside a unit the division gives tile and row tile.
template <int kTile>
struct MassCost {
  const kvc::ChunkArgs& a;
  __device__ __forceinline__ int items() const { return (int)a.units; }
  __device__ __forceinline__ int row_tiles(const kvc::ChunkUnit& r) const { return max(1, (r.n + a.tt - 1) / a.tt); }
  __device__ __forceinline__ int key_tiles(const kvc::ChunkUnit& r) const { return (r.len + r.n + kTile - 1) / kTile - r.first / kTile; }
  __device__ __forceinline__ int64_t operator()(int64_t u, kvc::ChunkUnit& r) const {
    r = load_unit(a, u);
    return (int64_t)key_tiles(r) * row_tiles(r);
  }
};

// for (MassWalk w(cost, piece); w.next(); ): row tiles [w.tb, w.te) of the w.rs of
// key tile w.tile (counted from the unit's first visible one) of unit w.u.
template <int kTile>
struct MassWalk {
  const MassCost<kTile>& cost;
  long long left;                      // steps of the piece still to come
  int64_t u;
  kvc::ChunkUnit r;
  int rs, tile, tiles, tb, te;
  long long at;
  __device__ __forceinline__ MassWalk(const MassCost<kTile>& c, const Piece& p)
      : cost(c), left(p.item >= 0 ? p.hi - p.lo : 0), u(p.item), r(p.r), rs(0), at(p.lo - p.start) {}
  __device__ __forceinline__ bool next() {
    if (rs > 0) left -= te - tb;
    if (left <= 0) return false;
    if (rs == 0) {                                     // the piece's first item
      rs = cost.row_tiles(r);
      tiles = cost.key_tiles(r);
      tile = (int)(at / rs);
      tb = (int)(at - (long long)tile * rs);
    } else {
      tb = 0;
      ++tile;
      while (tile >= tiles) {                          // a step follows, so a unit with tiles does
        cost(++u, r);
        rs = cost.row_tiles(r);
        tiles = cost.key_tiles(r);
        tile = 0;
      }
    }
    te = (int)min((long long)rs, tb + left);
    return true;
  }
  __device__ __forceinline__ bool whole() const { return tb == 0 && te == rs; }
};

// The item and offset at which a piece starts.
template <int kTile>
__device__ __forceinline__ kvc::ChunkSeg mass_seg(const MassCost<kTile>& cost, const Piece& p) {
  if (p.item < 0) return kvc::ChunkSeg{-1, 0};
  const int rs = cost.row_tiles(p.r);
  const long long at = p.lo - p.start;
  return kvc::ChunkSeg{((int64_t)p.item << 32) | (at / rs), at % rs > 0};
}

__device__ __forceinline__ void mass_store(const kvc::ChunkArgs& a, const kvc::ChunkUnit& r, const RowMap& rows, int e,
                                           float sum) {
  const int64_t row = rows(e);
  a.mass[row] = e < r.len ? fmaf(a.decay, a.mass[row], sum) : sum;
}

}  // namespace kvcd

namespace kvc {

// Launch with programmatic stream serialization: the kernel calls pdl_wait
// before it reads what its predecessor writes.
template <typename... Params, typename... Args>
cudaError_t chunk_launch(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem,
                         cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Allows a kernel its dynamic shared memory, once per device.
template <auto kKernel>
cudaError_t chunk_allow_smem(size_t bytes) {
  static std::atomic<uint32_t> done[8];                // a bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 256) return e != cudaSuccess ? e : cudaErrorInvalidDevice;
  const uint32_t bit = 1u << (dev & 31);
  if (done[dev >> 5].load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) done[dev >> 5].fetch_or(bit, std::memory_order_release);
  return e;
}

// Argument checks shared by the calls (p, c and the page table), and the fields
// of the argument block that come from them.
int chunk_check(const kvc_params* p, const kvc_chunk* c);
void chunk_fill(ChunkArgs& a, const kvc_params* p, const kvc_chunk* c);

// kvc_chunk_attn in bf16 without its first kernel, for callers that have written the units' records and
// contiguous rows of entries themselves: the workspace for `units` of them, its
// members in the argument block, and the launches.
size_t chunk_rows_bytes(const kvc_params* p, int64_t units);
void chunk_rows_workspace(ChunkArgs& a, const kvc_params* p, int64_t units, void* workspace);
cudaError_t chunk_attn_rows(ChunkArgs& a, int d, int sms, cudaStream_t s);

}  // namespace kvc

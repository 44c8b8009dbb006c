// kvc_q8_attn for many query rows in bf16: the codes become bf16 rows in the workspace
// (exact: 4 significant bits times a power of two), and the tcgen05 kernel of kvc_chunk_attn
// attends over these.  Converting in the attention kernel would be done again for every 256
// query rows (32 times in a 2048-token chunk with four heads a group), on the same issue slots
// that bound its softmax; here it is done once: 12 us of the 382 of 2048 tokens over 16384 entries (8 KV heads, G 4).
#include <algorithm>

#include "kvc_chunk_tc.cuh"
#include "kvc_q8.cuh"

namespace {

using kvc::Q8Args;

constexpr int kThreads = 256;

struct Q8Expand {
  Q8Args x;
  __nv_bfloat16* K;                    // [units][rows][D]
  __nv_bfloat16* V;
  float* logm;                         // [units][rows]
  int4* rec;
  int64_t u0;                          // first unit of the group
  int rows;                            // max_pages * page_rows
};

// One CTA per (unit, page): 16 codes a thread at a time.
template <int D>
__global__ void __launch_bounds__(kThreads) q8_expand_kernel(const __grid_constant__ Q8Expand a) {
  constexpr int kC = D / 16;
  const Q8Args& x = a.x;
  kvcd::pdl_wait();
  const int64_t u = blockIdx.x / x.max_pages;
  const int j = (int)(blockIdx.x - u * x.max_pages), R = 1 << x.shift;
  const int64_t gu = kvcd::q8_unit_global(x, a.u0 + u);
  const int len = x.len_lh[gu];
  int n = x.len_new[gu] - len;
  const bool bad = len < 0 || n < 0 || n > x.T || (int64_t)len + n > a.rows;
  if (bad) n = 0;
  if (j == 0 && threadIdx.x == 0) {
    if (bad) kvcd::record_error(x.err, KVC_EDEVICE);
    const int64_t off = u * a.rows;
    a.rec[u] = make_int4(n ? len : 0, n, (int)(uint32_t)off, (int)(off >> 32));
  }
  const int count = min(R, len + n - (j << x.shift));
  if (n > 0 && count > 0) {
    const int page = __ldg(x.table + gu * x.max_pages + j);
    const bool there = (unsigned)page < (unsigned)x.pages;
    if (!there && threadIdx.x == 0) kvcd::record_error(x.err, KVC_EDEVICE);
    const int64_t from = (int64_t)(there ? page : 0) << x.shift, to = u * a.rows + (j << x.shift);
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const float s = (v ? x.v_scale : x.k_scale)[there ? page : 0];
      const uint4* src = reinterpret_cast<const uint4*>((v ? x.V : x.K) + from * D);
      __nv_bfloat16* dst = (v ? a.V : a.K) + to * D;
#pragma unroll 2
      for (int i = threadIdx.x; i < count * kC; i += kThreads) {
        const uint4 w = src[i];
        const uint32_t c[4] = {w.x, w.y, w.z, w.w};
        uint32_t o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float lo, hi;
          kvcd::e4m3_f32((uint16_t)(c[k >> 1] >> ((k & 1) * 16)), lo, hi);
          o[k] = kvctc::bf16x2(lo * s, hi * s);
        }
        kvctc::store32(dst + (int64_t)i * 16, o);
      }
    }
    for (int i = threadIdx.x; i < count; i += kThreads) a.logm[to + i] = x.logm ? x.logm[from + i] : 0.f;
  }
  kvcd::pdl_trigger();
}

struct ChunkLayoutQ8 {
  int64_t units;                       // of a group
  int64_t rows;                        // of a unit
  size_t K, V, logm, chunk, total;
};

constexpr size_t kGroupBytes = 1u << 30;     // of expanded rows: units beyond go in further groups (256 units of 4000 entries, 128 rows
                                             // each: 232 us; in groups of 256 MB 256, of 64 MB, which stay in L2, 355)

ChunkLayoutQ8 chunk_layout_q8(const kvc_params* p, const kvc_chunk* c) {
  ChunkLayoutQ8 w;
  const int64_t units = (int64_t)p->B * p->H * (c->layer_end - c->layer_begin);
  w.rows = (int64_t)c->max_pages * c->page_rows;
  const size_t unit = (size_t)w.rows * (4 * p->d + 4);
  w.units = std::min<int64_t>(units, std::max<int64_t>(1, (int64_t)(kGroupBytes / unit)));
  w.units = std::min<int64_t>(w.units, std::max<int64_t>(1, ((1LL << 31) - 1) / w.rows));
  const size_t rows = (size_t)(w.units * w.rows);
  w.K = 0;
  w.V = kvc::align256(rows * p->d * 2);
  w.logm = w.V + kvc::align256(rows * p->d * 2);
  w.chunk = w.logm + kvc::align256(rows * 4);
  w.total = w.chunk + kvc::chunk_rows_bytes(p, w.units);
  return w;
}

}  // namespace

namespace kvc {

size_t q8_chunk_bytes(const kvc_params* p, const kvc_chunk* c) { return chunk_layout_q8(p, c).total; }

cudaError_t q8_chunk_launch(const kvc_params* p, const kvc_chunk* c, const Q8Args& x, const void* q, void* out,
                            float* lse, void* workspace, cudaStream_t s) {
  const ChunkLayoutQ8 w = chunk_layout_q8(p, c);
  char* ws = static_cast<char*>(workspace);
  for (int64_t u0 = 0; u0 < x.units; u0 += w.units) {
    const int64_t units = std::min(w.units, x.units - u0);
    const size_t heads = (size_t)u0 * x.G * x.T;
    ChunkArgs a = {};
    chunk_fill(a, p, c);
    chunk_rows_workspace(a, p, w.units, ws + w.chunk);
    a.q = static_cast<const char*>(q) + heads * p->d * 2;
    a.out = static_cast<char*>(out) + heads * p->d * 2;
    a.lse = lse ? lse + heads : nullptr;
    a.Kp = ws + w.K;
    a.Vp = ws + w.V;
    a.logm = reinterpret_cast<float*>(ws + w.logm);
    a.page_table = nullptr;
    a.packed_rows = w.units * w.rows;
    a.units = units;
    a.per_seq = (int)units;
    a.err = x.err;
    Q8Expand e = {};
    e.x = x;
    e.K = static_cast<__nv_bfloat16*>(a.Kp);
    e.V = static_cast<__nv_bfloat16*>(a.Vp);
    e.logm = a.logm;
    e.rec = a.rec;
    e.u0 = u0;
    e.rows = (int)w.rows;
    const dim3 grid((unsigned)(units * c->max_pages));
    count_launch();
    cudaError_t st = p->d == 128 ? chunk_launch(q8_expand_kernel<128>, grid, dim3(kThreads), 0, s, e)
                                 : chunk_launch(q8_expand_kernel<64>, grid, dim3(kThreads), 0, s, e);
    if (st == cudaSuccess) st = chunk_attn_rows(a, p->d, sm_count(), s);
    if (st != cudaSuccess) return st;
  }
  return cudaSuccess;
}

}  // namespace kvc

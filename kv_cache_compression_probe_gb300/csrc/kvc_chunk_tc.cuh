// Tensor-core building blocks of the bf16 chunk kernels: tcgen05 descriptors and
// instructions, TMEM moves, tensor-map copies, packed fp32 arithmetic and the
// score function.
#pragma once
#include <cuda.h>

#include "kvc_chunk.cuh"

namespace kvctc {

constexpr uint32_t kHalf = 128 * 128;  // bytes of 128 rows x 64 features (one swizzled block)

// 128-byte-swizzled operand descriptors.  The high word is the same for all; the
// low word is the address in 16-byte units and, for an MN-major operand, the
// distance between 64-feature blocks.  Steps inside a tile add to the low word, so
// the issuing warp keeps them in uniform registers.
constexpr uint32_t kDescHi = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return ((saddr & 0x3FFFFu) >> 4) | (lbo << 16); }
constexpr uint32_t kLboK = 1, kLboMN = kHalf >> 4;
__device__ __forceinline__ uint64_t desc(uint32_t lo) { return ((uint64_t)kDescHi << 32) | lo; }
// K-major without swizzle: 8-row x 16-byte blocks, 128 bytes to the next along K, 256
// to the next 8 rows (a 16-wide operand of 32 bytes a row).
constexpr uint32_t kExtHi = (256 >> 4) | (1u << 14);
__device__ __forceinline__ uint32_t ext_lo(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | ((128u >> 4) << 16); }
__device__ __forceinline__ uint64_t ext_desc(uint32_t lo) { return ((uint64_t)kExtHi << 32) | lo; }
// bf16 x bf16 -> fp32, M = 128; b_mn: the B operand is MN-major.
__host__ __device__ constexpr uint32_t idesc(int n, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (8u << 24) | (b_mn ? 1u << 16 : 0u);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc));
}
// A operand from TMEM.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(acc));
}
// One lane of a converged warp; the compiler knows that what it uses is uniform.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n selp.u32 %0, 1, 0, e;\n}\n" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   kvcd::smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Earlier generic writes to global memory (another kernel's) before async-proxy reads.
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

#define KVC_R4(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3])
#define KVC_R16(a, i) KVC_R4(a, i), KVC_R4(a, i + 4), KVC_R4(a, i + 8), KVC_R4(a, i + 12)
#define KVC_I4(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3])
#define KVC_I16(a, i) KVC_I4(a, i), KVC_I4(a, i + 4), KVC_I4(a, i + 8), KVC_I4(a, i + 12)

// Waits for the TMEM loads so far; the loaded registers pass through, so nothing that
// uses them moves up.
#define KVC_P4(a, i) "+r"(a[i]), "+r"(a[i + 1]), "+r"(a[i + 2]), "+r"(a[i + 3])
#define KVC_P16(a, i) KVC_P4(a, i), KVC_P4(a, i + 4), KVC_P4(a, i + 8), KVC_P4(a, i + 12)
__device__ __forceinline__ void wait_ld(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : KVC_P16(r, 0));
}
// 16 consecutive TMEM columns of this thread's lane (no wait).
__device__ __forceinline__ void tld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : KVC_R16(r, 0)
      : "r"(addr));
}
__device__ __forceinline__ void tst16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          addr),
      KVC_I16(r, 0)
      : "memory");
}

__device__ __forceinline__ void tma2d(uint32_t dst, const CUtensorMap* m, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(kvcd::smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma3d(uint32_t dst, const CUtensorMap* m, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(kvcd::smem_u32(bar))
      : "memory");
}

// 32 bytes, one whole sector, in one store (32-byte aligned).
__device__ __forceinline__ void store32(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), KVC_I4(v, 0), KVC_I4(v, 4) : "memory");
}

// Packed pairs of fp32.
__device__ __forceinline__ uint64_t pk(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void upk(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// (bf16(lo), bf16(hi)) in one register, each rounded to nearest.
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// tanh(y) in fp32: y times a degree-5 polynomial in y^2 below y^2 = 1/2 (least
// squares of the relative error over that range; off by at most 9e-8 of the
// value), 1 - 2 / (1 + e^2y) above, where nothing cancels.
__device__ __forceinline__ float tanh_f(float y) {
  const float z = y * y;
  float p = fmaf(z, -0.005034883506596088f, 0.019964737817645073f);
  p = fmaf(z, p, -0.053502924740314484f);
  p = fmaf(z, p, 0.13328056037425995f);
  p = fmaf(z, p, -0.3333311080932617f);
  p = fmaf(y * z, p, y);
  return z < 0.5f ? p : fmaf(-2.f, rcp(1.f + kvcd::ex2(y * 2.885390081777927f)), 1.f);
}

// Announces bytes of copies without arriving.
__device__ __forceinline__ void mbar_expect(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(kvcd::smem_u32(bar)), "r"(bytes) : "memory");
}

// Whether a phase has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(kvcd::smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// An extra 16-wide step of a product carries per-row and per-entry terms of the scores:
// the fp32 value x as the sum of three bf16 parts (8 bits each), times 1.  ext_store
// writes a row's 16 columns (8-row blocks of 16-byte pieces, as ext_desc says).
__device__ __forceinline__ void split3(float x, uint32_t (&p)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const __nv_bfloat16 h = __float2bfloat16_rn(x);
    p[i] = __bfloat16_as_ushort(h);
    x = isinf(x) ? 0.f : x - __bfloat162float(h);
  }
}
__device__ __forceinline__ void ext_store(unsigned char* tile, int row, const uint4& c0, const uint4& c1) {
  unsigned char* p = tile + (row >> 3) * 256 + (row & 7) * 16;
  *reinterpret_cast<uint4*>(p) = c0;
  *reinterpret_cast<uint4*>(p + 128) = c1;
}
// A suspended wait of the hardware's own length (with a hint of 1 ms, as elsewhere here, the
// 2048-token chunk took 378 us instead of 375 and the 1024-token masses 93.4 instead of 92.2).
__device__ __forceinline__ bool mbar_try(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(kvcd::smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits for a phase; gives up when another role has, or after `ns` nanoseconds.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, uint64_t ns, volatile int* abort) {
  if (mbar_try(bar, parity)) return true;
  if (*abort) return false;
  const uint64_t t0 = kvcd::global_timer_ns();
  while (!mbar_try(bar, parity)) {
    if (*abort) return false;
    if (kvcd::global_timer_ns() - t0 > ns) {
      *abort = 1;
      return false;
    }
  }
  return true;
}

// The same for a whole warp, which leaves converged.
__device__ __forceinline__ void warp_join(uint64_t* bar, uint32_t parity, uint64_t ns, volatile int* abort) {
  wait_or_abort(bar, parity, ns, abort);
  __syncwarp();
}
// And every lane gets the same answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint64_t ns, volatile int* abort) {
  return __all_sync(KVC_FULL_MASK, wait_or_abort(bar, parity, ns, abort));
}

// Or of a predicate over the `n` threads of named barrier `id` (whole warps, converged),
// which also orders their shared-memory accesses.
__device__ __forceinline__ bool named_or(int id, int n, bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %3, 0;\n bar.red.or.pred q, %1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(id), "r"(n), "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

// Copies of one 128-entry tile of K or V, entries from e0 on, of `total` in all, by
// a whole warp.  Contiguous: one box per 64-feature block, rows past the last entry
// included.  Paged: one box per page (or part of one) and block; boxes with no entry
// are not copied.  tile_row is what a lane has to look up first (the row of its box),
// so that a caller can do it ahead.
__device__ __forceinline__ int tile_boxes(const kvcd::RowMap& rows, int e0, int total) {
  const int shift = min(rows.shift, 7);
  return rows.table ? (min(128, total - e0) + (1 << shift) - 1) >> shift : 1;
}
__device__ __forceinline__ int tile_row(const kvcd::RowMap& rows, int e0, int total, int lane) {
  return lane < tile_boxes(rows, e0, total) ? (int)rows(e0 + (lane << min(rows.shift, 7))) : 0;
}
template <int D>
__device__ __forceinline__ void copy_tile(const kvcd::RowMap& rows, const CUtensorMap* map, uint32_t dst, int boxes,
                                          int row, uint64_t* bar, int lane) {
  constexpr int kBlocks = D / 64;
  const uint32_t bytes = rows.table ? 128u << min(rows.shift, 7) : kHalf;   // of one box
  if (lane == 0) kvcd::mbar_arrive_expect_tx(bar, boxes * bytes * kBlocks);
  __syncwarp();
  if (lane < boxes)
#pragma unroll
    for (int h = 0; h < kBlocks; ++h) tma2d(dst + h * kHalf + lane * bytes, map, h * 64, row, bar);
}

}  // namespace kvctc

namespace kvc {
// bf16 [rows, d] in 128-byte-swizzled boxes of 64 features x box_rows rows; and
// the query array [units * G, T, d] in boxes of 64 x tt x G.
bool chunk_encode_rows(CUtensorMap* m, const void* base, int64_t rows, int d, int box_rows);
bool chunk_encode_q(CUtensorMap* m, const void* base, int64_t heads, int T, int d, int tt, int G);
bool chunk_tc_available();
cudaError_t chunk_mass_tc_launch(ChunkArgs& a, int d, int sms, int page_rows, cudaStream_t s);
cudaError_t chunk_attn_tc_launch(ChunkArgs& a, int d, int sms, int page_rows, cudaStream_t s);
}  // namespace kvc

// Internal declarations of the E4M3 (block-of-128 scales) operators: argument
// blocks, launchers, and the sm_100a primitives their kernels use.
#pragma once

#include <cuda.h>

#include "moe_internal.cuh"

namespace moe {

constexpr int kFp8Block = 128;          // values that share a scale, in both directions
constexpr float kFp8Max = 448.f;        // largest E4M3 magnitude
constexpr float kFp8MinScale = 1.17549435e-38f;  // 2^-126: a block of zeros gets codes 0 and this scale

__host__ __device__ inline int fp8_blocks(int n) { return (n + kFp8Block - 1) / kFp8Block; }

// Scale of a block from its largest magnitude (float32, correctly rounded).
__device__ __forceinline__ float fp8_scale(float amax) {
  return fmaxf(amax / kFp8Max, kFp8MinScale);
}

// Two floats -> two E4M3 codes (lo in the low byte), round to nearest even,
// saturating at +-448, NaN kept.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
  return r;
}
// Two float32 operations in one instruction, each rounded as by itself.
__device__ __forceinline__ unsigned long long pack2(float2 a) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ float2 unpack2(unsigned long long a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pack2(a)), "l"(pack2(b)));
  return unpack2(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pack2(a)), "l"(pack2(b)), "l"(pack2(c)));
  return unpack2(r);
}

// Quotients of a block's values by its scale s, as its codes need them.  v * (1 /
// s) is up to 1.5 units off, which next to a rounding border is the neighbouring
// code.  With h = 1 / s rounded and e = 1 - h s, which is exact, 1 / s = h / (1 - e),
// so v / s is v h + v h (e + e^2) to within 3 * 2^-24 units before the sum's one
// rounding.  The quotients of float32 values that lie so near to where the float32
// next to a code's border begins are few enough to be enumerated
// (tests/test_fp8_host.py), and all of them round as v / s does.  Nothing leaves
// float32's range: h is normal, and the products are of the codes' size.  In pairs
// it costs the norm 1 to 9 % (T = 4096, H = 4096: 27.1 -> 27.6 us; T = 777, H =
// 7088, codes only: f16 7.1 -> 7.5, f32 8.4 -> 9.1) and gate / up nothing to speak
// of; the division cost 10 to 35 % and 10 % (29.9, 9.5 us; T = 2048: 860 -> 945 us).
struct Fp8Quotient {
  float h, e;
  __device__ __forceinline__ explicit Fp8Quotient(float s) : h(1.f / s) {
    const float d = fmaf(-h, s, 1.f);
    e = h == 0.f ? 0.f : fmaf(d, d, d);  // s infinite: finite values give 0, infinite ones NaN
  }
  __device__ __forceinline__ float2 operator()(float2 v) const {
    const float2 hh = make_float2(h, h);
    const float2 q = fma2(v, hh, mul2(mul2(v, hh), make_float2(e, e)));
    // (a negative zero's terms have opposite signs where e is negative)
    return make_float2(copysignf(q.x, v.x), copysignf(q.y, v.y));
  }
};
// Codes of N pairs of values over their scale, two pairs to a word
template <int N>
__device__ __forceinline__ void fp8_codes(const float2 (&v)[N], float scale, uint32_t (&q)[(N + 1) / 2]) {
  const Fp8Quotient of(scale);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float2 d = of(v[i]);
    const uint32_t two = f32x2_to_e4m3x2(d.x, d.y);
    q[i / 2] = i % 2 ? q[i / 2] | (two << 16) : two;
  }
}

// ---------------------------------------------------------------- launchers ---
struct NormFp8Args {
  const void* x;
  const void* residual;   // or nullptr
  const float* weight;
  void* residual_out;     // or nullptr (same storage as residual or x allowed)
  void* y;                // or nullptr
  uint8_t* q;
  float* s;
  int rows, H, dtype;
  float eps;
};
cudaError_t launch_norm_fp8(const NormFp8Args& a, cudaStream_t st);

// One grouped (or, without offsets, single-group) product; swiglu: gate / up
// pair with an E4M3 result.
struct Fp8GemmArgs {
  const uint8_t* a_q;
  const float* a_s;       // [a_rows, blocks(K)]
  const uint8_t* w_q[2];  // [E, N, K]: the weights; or gate and up
  const float* w_s[2];    // [E, blocks(N), blocks(K)]
  const int32_t* offsets; // [E + 1], or nullptr: one group of all P rows
  const int32_t* entries; // [P], or nullptr when neither gathered nor scattered
  void* out;              // [P, N] out_type
  uint8_t* q_out;         // swiglu: [P, N], in bucket order
  float* s_out;           // swiglu: [P, blocks(N)]
  int* err;
  int a_rows, P, E, N, K;
  int a_div;              // > 0: row p of the buckets is A row entries[p] / a_div; 0: row p
  int scatter;            // output row entries[p] instead of p
  int out_type;
};
cudaError_t launch_gemm_fp8(const Fp8GemmArgs& a, bool swiglu, cudaStream_t st);

// 2-D map of a [rows, row_bytes] uint8 matrix, boxes of box_rows x box_bytes
// (64 or 128) with the swizzle of the same width.
bool make_tma_map_u8_box(CUtensorMap* m, const void* base, uint64_t row_bytes, uint64_t rows,
                         uint32_t box_bytes, uint32_t box_rows);

// The same matrix seen as [K / 128, rows, 128]: boxes of depth x box_rows x 128.
bool make_tma_map_u8_deep(CUtensorMap* m, const void* base, uint64_t row_bytes, uint64_t rows,
                          uint32_t box_rows, uint32_t depth);

// --------------------------------------------------------------- primitives ---
__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ unsigned long long global_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// The same, seeing what the cluster's other CTAs wrote before they arrived.
__device__ __forceinline__ bool bar_try_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// What a role needs to give up a wait: the CTA's abort flag and the error words,
// which hold the limit.
struct WaitCtl {
  volatile int* abort_flag;
  int* err;
};
constexpr unsigned long long kFp8GraceNs = 20000;  // the limit is not read before a wait lasts that long
// Bounded wait of a whole warp; false if it gave up (or another role already
// did).  Every lane asks, so the code around it stays warp-uniform.
template <bool CLUSTER = false>
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, const WaitCtl& c, int where) {
  auto try_once = [&] {
    return __all_sync(kFull, CLUSTER ? bar_try_cluster(bar, parity) : bar_try(bar, parity)) != 0;
  };
  if (try_once()) return true;
  const unsigned long long t0 = global_ns();
  while (!try_once()) {
    if (__any_sync(kFull, *c.abort_flag != 0)) return false;
    const unsigned long long waited = global_ns() - t0;
    bool over = false;
    if (waited > kFp8GraceNs) {
      const unsigned us = *(reinterpret_cast<const volatile unsigned*>(c.err) + 2);
      over = waited > (us ? us : kDefaultWaitUs) * 1000ull;
    }
    if (__any_sync(kFull, over)) {
      *c.abort_flag = 1;
      if ((threadIdx.x & 31) == 0) latch_error(c.err, MOE_ERR_TIMEOUT, where);
      return false;
    }
  }
  return true;
}
// One lane of a converged warp.  Loops that issue copies or MMAs run on the
// whole warp and only the instruction itself stands under this predicate: the
// compiler then keeps descriptors and coordinates in uniform registers (under
// `lane == 0` four MMAs took about 490 clocks to issue).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar,
                                       uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "l"(policy)
      : "memory");
}
// Blocks z.. of rows y.. (a map of make_tma_map_u8_deep).
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int z, int y, uint32_t bar,
                                       uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(z), "r"(bar), "l"(policy)
      : "memory");
}
// Four rows of the matrix (a map with one-row boxes) into four consecutive
// rows of the tile.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, int x, int r0, int r1,
                                            int r2, int r3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(r0), "r"(r1), "r"(r2), "r"(r3), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tcgen_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tcgen_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tcgen_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
               : "memory");
}
// D (TMEM, float32) = A x B^T (+ D): E4M3 operands in shared memory, K = 32.
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b),
      "r"(idesc), "r"(accumulate)
      : "memory");
}
// K-major operand, 128-byte swizzle, rows of 128 bytes, 8-row groups 1024
// bytes apart.
__device__ __forceinline__ uint64_t desc_k_sw128(uint32_t addr) {
  return uint64_t((addr & 0x3FFFFu) >> 4) | (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32) |
         (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// Instruction descriptor: E4M3 x E4M3 -> float32, both K-major, M x N.
__host__ __device__ constexpr uint32_t idesc_e4m3(int m, int n) {
  return (1u << 4) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}
// NC columns of this warp's TMEM quarter -> registers; complete after
// tmem_wait(), whose operands keep the uses behind it.
template <int NC>
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[NC]) {
  if constexpr (NC == 32) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
  } else {
    static_assert(NC == 16);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
  }
}
template <int NC>
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[NC]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < NC; ++i) asm volatile("" : "+r"(r[i]));
}
// (acc.lo, acc.hi) += (d.lo, d.hi) * s, one rounding each
__device__ __forceinline__ void fma_pair(float2& acc, uint32_t d0, uint32_t d1, float2 s) {
  unsigned long long a, d, m;
  asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(acc.x), "f"(acc.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(d0), "r"(d1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(m) : "f"(s.x), "f"(s.y));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(a) : "l"(d), "l"(m));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(acc.x), "=f"(acc.y) : "l"(a));
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
// Every thread of every CTA of the cluster, with release / acquire ordering.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// Shared-memory address `addr` of CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_st(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

}  // namespace moe

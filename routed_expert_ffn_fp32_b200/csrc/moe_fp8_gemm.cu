// E4M3 x E4M3 -> float32 products with a float32 scale per 128 x 128 block of
// the weights and per row and 128 values of the activations, dense or grouped
// by expert with ragged bucket sizes:
//
//   y[p, n] = sum_b sa[p, b] sw[n / 128, b] sum_{k in block b} a[p, k] w[n, k]
//
// and the gate / up pair h = silu(g) u with its own E4M3 quantisation fused in.
//
// The scales are general float32 values, so they cannot ride in the tensor
// core's power-of-two scale factors.  Instead each K block of 128 is one
// accumulation of four tcgen05.mma (K = 32 each) into a TMEM buffer, and the
// epilogue warps add it, times sa * sw, to float32 registers while the next
// block's MMAs fill the other buffer.  With the activations on the MMA's M
// side a thread's TMEM lane is one row and its columns lie in one weight block,
// so a block costs one scale product per thread and one (packed) FMA a value.
//
// Tile: 128 rows x BN weight rows, one CTA per SM, persistent over the tiles of
// all buckets.  Warps 0-7 promote and store (4 TMEM quarters x 2 column halves),
// warp 8 is the TMA producer, warp 9 issues the MMAs.  Rows of a bucket are
// fetched by TMA row gather (token rows picked by the entries) or, when they
// are consecutive, by boxes of 32 rows; only the rows that exist are fetched,
// so a decode bucket costs its own bytes (the MMA's other rows hold leftovers
// that nothing reads: rows of a product do not mix).
//
// Few tiles (decode): a cluster of up to 8 CTAs splits K; every CTA leaves its
// float32 sums in shared memory and the rows are added over the cluster in rank
// order through distributed shared memory: no workspace, no atomics, the same
// result every time.
#include "moe_fp8.cuh"

namespace moe {
namespace {

constexpr int kBM = 128;             // bucket rows per tile (MMA M)
constexpr int kEpiWarps = 8;
constexpr int kThreads = (kEpiWarps + 2) * 32;
constexpr unsigned long long kLimitNs = 2000000000ull;  // default bound of a wait: 2 s

template <bool SWIGLU, int BN>
struct Cfg {
  static constexpr int COLS = SWIGLU ? BN / 2 : BN;  // output columns per tile
  static constexpr int A_BYTES = kBM * 128;
  static constexpr int B_BYTES = BN * 128;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int NS = 192 * 1024 / STAGE;
  static constexpr int CP = BN / 2;                  // accumulator columns per thread
  static constexpr int RED_PITCH = BN + 4;           // floats per row of the split sums
  static constexpr int CTL = NS * STAGE;             // barriers, exchange, tables follow
  static constexpr int XCH = CTL + 256;              // float [2][2][128] block maxima
  static constexpr int TAB = XCH + 2048;             // int [3][E + 1]
  static_assert(kBM * RED_PITCH * 4 <= NS * STAGE, "split sums fit the stages");
  static size_t smem(int E) { return size_t(TAB) + 12 * size_t(E + 1) + 1024 /*alignment*/; }
};

struct Maps {
  CUtensorMap a;     // A rows: 1-row boxes (gather) or 32-row boxes
  CUtensorMap w[2];  // weights, 128-row boxes (gate and up, or twice the same)
};

struct Tile {
  int e, nt;
  int row0;    // first bucket position of the tile
  int nvalid;  // rows
};

__device__ __forceinline__ Tile tile_of(const int* t_off, const int* t_beg, const int* t_cnt, int E,
                                        int it) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t_off[mid] <= it) lo = mid;
    else hi = mid - 1;
  }
  const int li = it - t_off[lo];
  const int mtiles = (t_cnt[lo] + kBM - 1) / kBM;
  Tile t;
  t.e = lo;
  t.nt = li / mtiles;  // row tiles fastest: neighbours share the weight tile in L2
  const int mt = li - t.nt * mtiles;
  t.row0 = t_beg[lo] + mt * kBM;
  t.nvalid = min(kBM, t_cnt[lo] - mt * kBM);
  return t;
}

// True if `ok` holds in all 256 epilogue threads.  They meet here once per tile
// of the fused pair, also when a wait was given up, so none is left behind.
__device__ __forceinline__ bool epi_vote(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "barrier.cta.red.and.pred p, 1, 256, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(uint32_t(ok))
      : "memory");
  return r != 0;
}

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.f + expf(-g)) * u; }

__device__ __forceinline__ void store_one(void* out, int type, size_t i, float v) {
  if (type == MOE_DTYPE_F32) static_cast<float*>(out)[i] = v;
  else if (type == MOE_DTYPE_BF16) static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(out)[i] = __float2half_rn(v);
}

__device__ __forceinline__ uint32_t pack16(int type, float a, float b) {
  if (type == MOE_DTYPE_F16) return f32x2_to_f16x2(a, b);
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// NC consecutive values of one row from element i on, `left` of them inside
// the row; vec: i and the row pitch keep 16-byte alignment.
template <int NC>
__device__ __forceinline__ void store_row(void* out, int type, size_t i, const float2 (&v)[NC / 2],
                                          int left, bool vec) {
  if (vec && left >= NC) {
    if (type == MOE_DTYPE_F32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + i);
#pragma unroll
      for (int j = 0; j < NC / 4; ++j)
        o[j] = make_float4(v[2 * j].x, v[2 * j].y, v[2 * j + 1].x, v[2 * j + 1].y);
    } else {
      uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + i);
#pragma unroll
      for (int j = 0; j < NC / 8; ++j)
        o[j] = make_uint4(pack16(type, v[4 * j].x, v[4 * j].y), pack16(type, v[4 * j + 1].x, v[4 * j + 1].y),
                          pack16(type, v[4 * j + 2].x, v[4 * j + 2].y),
                          pack16(type, v[4 * j + 3].x, v[4 * j + 3].y));
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < NC; ++j)
    if (j < left) store_one(out, type, i + j, j & 1 ? v[j / 2].y : v[j / 2].x);
}

template <bool SWIGLU, int BN>
__global__ void __launch_bounds__(kThreads, 1)
    k_gemm_fp8(const __grid_constant__ Fp8GemmArgs a, const __grid_constant__ Maps maps) {
  using C = Cfg<SWIGLU, BN>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::CTL);
  uint64_t* empty = full + C::NS;
  uint64_t* acc_full = empty + C::NS;  // [2]
  uint64_t* acc_empty = acc_full + 2;  // [2]
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* xch = reinterpret_cast<float*>(smem + C::XCH);
  int* t_off = reinterpret_cast<int*>(smem + C::TAB);
  int* t_beg = t_off + (a.E + 1);
  int* t_cnt = t_beg + (a.E + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = int(cluster_rank()), S = int(cluster_size());
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NS; ++s) {
      bar_init(smem_addr(&full[s]), 1);
      bar_init(smem_addr(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      bar_init(smem_addr(&acc_full[b]), 1);
      bar_init(smem_addr(&acc_empty[b]), kEpiWarps);
    }
    bar_init(smem_addr(drain), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.a) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.w[0]) : "memory");
    if (SWIGLU) asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.w[1]) : "memory");
  }
  if (warp == kEpiWarps + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tmem_slot)),
                 "r"(2 * BN)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  pdl_trigger();
  const unsigned wait_us = *(reinterpret_cast<const volatile unsigned*>(a.err) + 2);
  const unsigned debug = *(reinterpret_cast<const volatile unsigned*>(a.err) + 3);
  const WaitCtl ctl{abort_flag, a.err, wait_us ? wait_us * 1000ull : kLimitNs};

  // bucket starts and sizes; offsets that are not ascending inside [0, P] stop
  // the whole call (latched, nothing written)
  const int NT = (a.N + C::COLS - 1) / C::COLS;
  int bad = 0;
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    const int b = a.offsets ? a.offsets[e] : 0, n = a.offsets ? a.offsets[e + 1] : a.P;
    bad |= b < 0 || n < b || n > a.P;
    t_beg[e] = b;
    t_cnt[e] = n - b;
  }
  tcgen_fence_before();
  bad = __syncthreads_or(bad);
  tcgen_fence_after();
  if (bad && threadIdx.x == 0) latch_error(a.err, MOE_ERR_DEVICE_DATA, 500);
  if (warp == 0) {
    int run = 0;
    for (int base = 0; base < a.E; base += 32) {
      const int e = base + lane;
      const int n = e < a.E && !bad ? (t_cnt[e] + kBM - 1) / kBM * NT : 0;
      int inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, inc, o);
        if (lane >= o) inc += y;
      }
      if (e < a.E) t_off[e] = run + inc - n;
      run += __shfl_sync(kFull, inc, 31);
    }
    if (lane == 0) t_off[a.E] = run;
  }
  __syncthreads();
  const uint32_t tmem = *tmem_slot;
  const int n_tiles = t_off[a.E];
  const int KB = fp8_blocks(a.K);
  // this CTA's tiles and K blocks; a split launch has a cluster for every tile
  const int first = blockIdx.x / S, step = gridDim.x / S;
  const int kb0 = KB * rank / S, kb1 = KB * (rank + 1) / S;
  const bool gather = a.a_div > 0;

  if (warp == kEpiWarps) {
    // -------------------------------------------------------------- producer
    int stage = 0;
    uint32_t phase = 0, fills = 0, used = 0;
    uint64_t keep, once;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(keep));
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
    bool ok = true;
    for (int it = first; it < n_tiles && ok; it += step) {
      const Tile t = tile_of(t_off, t_beg, t_cnt, a.E, it);
      // weights that one row tile alone reads are not worth keeping in L2
      const uint64_t pol = t_cnt[t.e] <= kBM ? once : keep;
      int r[4];
      uint32_t bytes = C::B_BYTES;
      if (gather) {
        // rows 4 lane .. 4 lane + 3 of the tile; positions past the bucket
        // repeat its last row, an index out of range reads row 0
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int p = t.row0 + min(4 * lane + j, t.nvalid - 1);
          const int src = a.entries[p] / a.a_div;
          r[j] = src >= 0 && src < a.a_rows ? src : 0;
        }
        bytes += (t.nvalid + 3) / 4 * 512;
      } else {
        bytes += (t.nvalid + 31) / 32 * 4096;
      }
      const int wrow = t.e * a.N + t.nt * C::COLS;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!bar_wait_warp(smem_addr(&empty[stage]), phase ^ 1u, ctl, 510)) {
          ok = false;
          break;
        }
        const uint32_t st = smem_addr(smem + stage * C::STAGE), fb = smem_addr(&full[stage]);
        const int x = kb * 128;
        if ((debug & MOE_DEBUG_STARVE_FIRST_WAIT) && blockIdx.x == 0 && it == first && kb == kb0) {
          // debug switch: the first stage gets no copies, so the MMA thread's
          // bounded wait on it runs out
          if (++stage == C::NS) {
            stage = 0;
            phase ^= 1u;
          }
          continue;
        }
        if (lane == 0) {
          bar_expect(fb, bytes);
          if constexpr (SWIGLU) {
            tma_2d(st + C::A_BYTES, &maps.w[0], x, wrow, fb, pol);
            tma_2d(st + C::A_BYTES + 128 * 128, &maps.w[1], x, wrow, fb, pol);
          } else {
#pragma unroll
            for (int j = 0; j < BN / 128; ++j)
              tma_2d(st + C::A_BYTES + j * 128 * 128, &maps.w[0], x, wrow + 128 * j, fb, pol);
          }
        }
        __syncwarp();
        if (gather) {
          if (4 * lane < t.nvalid) tma_gather4(st + lane * 512, &maps.a, x, r[0], r[1], r[2], r[3], fb);
        } else if (32 * lane < t.nvalid) {
          tma_2d(st + lane * 4096, &maps.a, x, t.row0 + 32 * lane, fb, keep);
        }
        fills ^= 1u << stage;
        used |= 1u << stage;
        if (++stage == C::NS) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (S > 1) break;
    }
    // after a give-up, let every copy this warp requested land (bounded)
    if (*abort_flag && lane == 0) {
      for (int s = 0; s < C::NS; ++s) {
        if (!((used >> s) & 1u)) continue;
        const unsigned long long t0 = global_ns();
        while (!bar_try(smem_addr(&full[s]), ((fills >> s) & 1u) ^ 1u) && global_ns() - t0 < 100000000ull) {
        }
      }
    }
  } else if (warp == kEpiWarps + 1) {
    // ------------------------------------------------------------------- MMA
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, g = 0;  // g: K blocks so far
      bool ok = true;
      constexpr uint32_t idesc = idesc_e4m3(kBM, BN);
      for (int it = first; it < n_tiles && ok; it += step) {
        for (int kb = kb0; kb < kb1; ++kb, ++g) {
          const uint32_t buf = g & 1u;
          ok = bar_wait(smem_addr(&acc_empty[buf]), ((g >> 1) & 1u) ^ 1u, ctl, 520) &&
               bar_wait(smem_addr(&full[stage]), phase, ctl, 521);
          if (!ok) break;
          tcgen_fence_after();
          const uint32_t st = smem_addr(smem + stage * C::STAGE);
          const int steps = min(4, (a.K - kb * 128 + 31) / 32);  // the tail reads zero fill
          for (int k = 0; k < steps; ++k)
            mma_e4m3(tmem + buf * BN, desc_k_sw128(st + 32 * k), desc_k_sw128(st + C::A_BYTES + 32 * k),
                     idesc, k != 0);
          tcgen_commit(smem_addr(&empty[stage]));
          tcgen_commit(smem_addr(&acc_full[buf]));
          if (++stage == C::NS) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (S > 1) break;
      }
      if (!ok || *abort_flag) {
        // let issued MMAs finish before TMEM is released (bounded)
        tcgen_commit(smem_addr(drain));
        const unsigned long long t0 = global_ns();
        while (!bar_try(smem_addr(drain), 0) && global_ns() - t0 < 200000000ull) {
        }
      }
    }
  } else {
    // --------------------------------------------------- promotion, epilogue
    const int q = warp & 3, half = warp >> 2;
    const int row = 32 * q + lane;
    uint32_t g = 0;
    bool ok = true;
    int local = 0;  // tiles of this CTA so far
    for (int it = first; it < n_tiles && ok; it += step, ++local) {
      const Tile t = tile_of(t_off, t_beg, t_cnt, a.E, it);
      const bool in = row < t.nvalid;
      const int p = t.row0 + min(row, t.nvalid - 1);
      int src = p, dst = p;
      bool good = in;
      if (gather || a.scatter) {
        const int ent = a.entries[p];
        if (gather) src = ent / a.a_div;
        if (a.scatter) dst = ent;
        if (ent < 0 || src >= a.a_rows || dst >= a.P) {
          if (in) latch_error(a.err, MOE_ERR_DEVICE_DATA, 501);
          good = false;
          src = dst = 0;
        }
      }
      const float* sa = a.a_s + size_t(src) * KB;
      // the weight block(s) of this thread's columns
      const int NB = fp8_blocks(a.N);
      const int nb = SWIGLU ? t.nt : min(t.nt * (BN / 128) + (BN == 256 ? half : 0), NB - 1);
      const float* sw0 = a.w_s[0] + (size_t(t.e) * NB + nb) * KB;
      const float* sw1 = SWIGLU ? a.w_s[1] + (size_t(t.e) * NB + nb) * KB : sw0;
      const bool work = 32 * q < t.nvalid;  // this warp's rows exist
      float2 acc[C::CP / 2];
#pragma unroll
      for (int j = 0; j < C::CP / 2; ++j) acc[j] = make_float2(0.f, 0.f);
      float na = kb0 < kb1 ? sa[kb0] : 0.f, n0 = kb0 < kb1 ? sw0[kb0] : 0.f, n1 = SWIGLU && kb0 < kb1 ? sw1[kb0] : 0.f;
      for (int kb = kb0; kb < kb1; ++kb, ++g) {
        const uint32_t buf = g & 1u;
        const float s0 = na * n0, s1 = SWIGLU ? na * n1 : 0.f;
        if (kb + 1 < kb1) {
          na = sa[kb + 1];
          n0 = sw0[kb + 1];
          if (SWIGLU) n1 = sw1[kb + 1];
        }
        if (!bar_wait_warp(smem_addr(&acc_full[buf]), (g >> 1) & 1u, ctl, 530)) {
          ok = false;
          break;
        }
        if (work) {
          tcgen_fence_after();
          const uint32_t col = tmem + buf * BN + (uint32_t(32 * q) << 16);
#pragma unroll
          for (int c = 0; c < C::CP / 32; ++c) {
            // swiglu: this half's 64 gate columns, then its 64 up columns
            const int c0 = SWIGLU ? (c < C::CP / 64 ? 0 : C::CP / 2) + half * (C::CP / 2) + 32 * c
                                  : half * C::CP + 32 * c;
            uint32_t d[32];
            tmem_load32(col + c0, d);
            const float s = SWIGLU && c >= C::CP / 64 ? s1 : s0;
#pragma unroll
            for (int j = 0; j < 16; ++j) fma_pair(acc[16 * c + j], d[2 * j], d[2 * j + 1], make_float2(s, s));
          }
          tcgen_fence_before();
        }
        __syncwarp();
        if (lane == 0) bar_arrive(smem_addr(&acc_empty[buf]));
      }
      if (!ok) {
        // the other epilogue warps meet this one in the tile's vote
        if (SWIGLU && S == 1) epi_vote(false);
        break;
      }
      if (S > 1) {
        // the split sums of the rows that exist, for the cluster
        float* red = reinterpret_cast<float*>(smem) + size_t(row) * C::RED_PITCH;
        if (in) {
#pragma unroll
          for (int j = 0; j < C::CP / 4; ++j) {
            const int c0 = SWIGLU ? (j < C::CP / 8 ? 0 : C::CP / 2) + half * (C::CP / 2) + 4 * j
                                  : half * C::CP + 4 * j;
            *reinterpret_cast<float4*>(red + c0) =
                make_float4(acc[2 * j].x, acc[2 * j].y, acc[2 * j + 1].x, acc[2 * j + 1].y);
          }
        }
        break;
      }
      if constexpr (SWIGLU) {
        // h in place of the gate values; its block maximum over both halves
        const int n0c = t.nt * C::COLS + half * (C::COLS / 2);
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < C::CP / 4; ++j) {
          acc[j].x = silu_mul(acc[j].x, acc[C::CP / 4 + j].x);
          acc[j].y = silu_mul(acc[j].y, acc[C::CP / 4 + j].y);
          if (n0c + 2 * j < a.N) amax = fmaxf(amax, fmaxf(fabsf(acc[j].x), fabsf(acc[j].y)));
        }
        // (two exchange buffers: a thread is past its read of one before any
        // other thread writes it again two tiles later)
        float* x = xch + (local & 1) * 256;
        x[half * 128 + row] = amax;
        if (!epi_vote(ok)) break;
        amax = fmaxf(amax, x[(half ^ 1) * 128 + row]);
        const float s = fp8_scale(amax), inv = 1.f / s;
        if (good) {
          uint8_t* o = a.q_out + size_t(p) * a.N + n0c;
#pragma unroll
          for (int j = 0; j < C::CP / 32; ++j) {
            if (n0c + 16 * j >= a.N) break;  // N is a multiple of 16
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = f32x4_to_e4m3x4(acc[8 * j + 2 * i].x * inv, acc[8 * j + 2 * i].y * inv,
                                     acc[8 * j + 2 * i + 1].x * inv, acc[8 * j + 2 * i + 1].y * inv);
            *reinterpret_cast<uint4*>(o + 16 * j) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          if (half == 0) a.s_out[size_t(p) * NB + t.nt] = s;
        }
      } else {
        const int n0c = t.nt * BN + half * C::CP;
        if (good && n0c < a.N) {
          const bool vec = a.N % (a.out_type == MOE_DTYPE_F32 ? 4 : 8) == 0;
          store_row<C::CP>(a.out, a.out_type, size_t(dst) * a.N + n0c, acc, a.N - n0c, vec);
        }
      }
    }
  }

  if (S > 1) {
    // every CTA of the cluster takes this path, whatever happened above
    __syncwarp();
    cluster_barrier();
    if (warp < kEpiWarps && first < n_tiles && !*abort_flag) {
      const Tile t = tile_of(t_off, t_beg, t_cnt, a.E, first);
      const int NB = fp8_blocks(a.N);
      constexpr int RW = SWIGLU ? 2 : 256 / BN;  // rows in flight: 256 threads, one column each
      const int tid = threadIdx.x;
      const int sub = SWIGLU ? tid / (BN / 2) : tid / BN;
      const int c = SWIGLU ? tid % (BN / 2) : tid % BN;
      for (int r0 = rank * RW; r0 < t.nvalid; r0 += S * RW) {
        const int r = r0 + sub;
        const bool in = r < t.nvalid;
        const uint32_t at = smem_addr(smem) + uint32_t(r * C::RED_PITCH + c) * 4;
        const int p = t.row0 + min(r, t.nvalid - 1);
        float v = 0.f, u = 0.f;
        if (in) {
          for (int k = 0; k < S; ++k) v += cluster_ld(cluster_map(at, k));
          if (SWIGLU)
            for (int k = 0; k < S; ++k) u += cluster_ld(cluster_map(at + (BN / 2) * 4, k));
        }
        if constexpr (SWIGLU) {
          const int n = t.nt * C::COLS + c;
          const float h = in && n < a.N ? silu_mul(v, u) : 0.f;
          float amax = fabsf(h);
          if (!(amax >= 0.f)) amax = 0.f;  // NaN: not part of the maximum
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
          if (lane == 0) xch[warp] = amax;
          asm volatile("bar.sync 1, 256;" ::: "memory");
          const int w0 = warp & ~3;
          amax = fmaxf(fmaxf(xch[w0], xch[w0 + 1]), fmaxf(xch[w0 + 2], xch[w0 + 3]));
          asm volatile("bar.sync 1, 256;" ::: "memory");
          const float s = fp8_scale(amax);
          const int ent = gather && in ? a.entries[p] : 0;
          const bool good = in && ent >= 0 && (!gather || ent / a.a_div < a.a_rows);
          if (good && n < a.N) a.q_out[size_t(p) * a.N + n] = uint8_t(f32x2_to_e4m3x2(h * (1.f / s), 0.f));
          if (good && c == 0) a.s_out[size_t(p) * NB + t.nt] = s;
        } else {
          const int n = t.nt * BN + c;
          int src = p, dst = p;
          bool good = in && n < a.N;
          if (in && (gather || a.scatter)) {
            const int ent = a.entries[p];
            if (gather) src = ent / a.a_div;
            if (a.scatter) dst = ent;
            good = good && ent >= 0 && src < a.a_rows && dst < a.P;
          }
          if (good) store_one(a.out, a.out_type, size_t(dst) * a.N + n, v);
        }
      }
    }
    __syncwarp();
    cluster_barrier();  // no CTA leaves while another reads its sums
  }

  __syncwarp();
  tcgen_fence_before();
  __syncthreads();
  if (warp == kEpiWarps + 1) {
    tcgen_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * BN)
                 : "memory");
  }
}

// --------------------------------------------------------------- host side ---
template <bool SWIGLU, int BN>
cudaError_t launch(const Fp8GemmArgs& a, long long max_tiles, int split, cudaStream_t st) {
  using C = Cfg<SWIGLU, BN>;
  Maps m;
  const uint64_t wrows = uint64_t(a.E) * a.N;
  if (!make_tma_map_u8_box(&m.a, a.a_q, a.K, a.a_rows, 128, a.a_div > 0 ? 1 : 32) ||
      !make_tma_map_u8_box(&m.w[0], a.w_q[0], a.K, wrows, 128, 128) ||
      !make_tma_map_u8_box(&m.w[1], a.w_q[SWIGLU ? 1 : 0], a.K, wrows, 128, 128))
    return cudaErrorInvalidValue;
  auto kern = k_gemm_fp8<SWIGLU, BN>;
  const size_t smem = C::smem(a.E);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const long long sms = device_info().sm_count;
  cfg.gridDim = dim3(unsigned(split > 1 ? max_tiles * split : max_tiles < sms ? max_tiles : sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(split);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a, m);
}

}  // namespace

cudaError_t launch_gemm_fp8(const Fp8GemmArgs& a, bool swiglu, cudaStream_t st) {
  if (a.P == 0) return cudaSuccess;
  const long long sms = device_info().sm_count;
  // row tiles at most: one per non-empty bucket, plus one per full 128 rows
  const long long groups = a.offsets ? (a.E < a.P ? a.E : a.P) : 1;
  const long long row_tiles = a.offsets ? groups + a.P / kBM : (a.P + kBM - 1) / kBM;
  const bool wide = swiglu || row_tiles * ((a.N + 255) / 256) >= sms;
  const int cols = swiglu ? 128 : wide ? 256 : 128;
  const long long tiles = row_tiles * ((a.N + cols - 1) / cols);
  int split = 1;
  while (split < 8 && tiles * split * 2 <= sms && fp8_blocks(a.K) >= split * 4) split *= 2;
  if (swiglu) return launch<true, 256>(a, tiles, split, st);
  return wide ? launch<false, 256>(a, tiles, split, st) : launch<false, 128>(a, tiles, split, st);
}

}  // namespace moe

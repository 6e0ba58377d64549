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
// blocks' MMAs fill the other buffers.  With the activations on the MMA's M
// side a thread's TMEM lane is one row and its columns lie in one weight block,
// so a block costs one scale product per thread and one (packed) FMA a value.
//
// Tile: MR rows x BN weight rows over all of K, one persistent CTA per SM.
//   warps 0-7  promote and store (4 TMEM quarters x 2 column halves)
//   warp 8     TMA of the weight tiles
//   warp 9     TMEM allocation, MMA issue
//   warp 10    TMA of the activation rows: gathered four at a time by the
//              bucket's entries, or boxes of consecutive rows
//   warp 11    the scales of each K block, through shared memory
// Only rows that exist are fetched.  Small buckets take MR = 16: the stage
// keeps 2 KB of activations and the other 48 rows of an M = 64 MMA read whatever
// lies behind (rows of a product do not mix, and nobody reads theirs); two warps
// promote and the other six store the tile before.
//
// What bounds it (B200, K loop of the full tile, per K block of 128): the MMAs
// and the copies of a 128 x 256 tile move 48 KB into and 48 KB out of shared
// memory, about 750 clocks without any promotion (106 us for 4096 x 8192 x
// 4096); with it 137 us, 2.0 PFLOP/s, as the promoting warps' chain of wait,
// TMEM load and FMA is the longer one (TMEM loads alone cost nothing, half the
// FMAs saves 10 us, the scales 10 us).  Grouped products of many experts are
// bound by HBM: down, T = 5, k = 8, 256 experts, H = 4096, I = 2048: 53 us for
// 316 MB (6.0 TB/s); T = 2048: 380 us (6.1 TB/s); gate / up T = 1: 26.3 us for
// 134 MB (5.1 TB/s), T = 2048: 755 to 890 us (up to 5.7 TB/s, TMA row gather and
// the tile's end beside the weights).  Under a sustained load the card's power limit
// lowers the clock, and the full tiles follow it (161, 460 and 915 us).
//
// Few rows mean few tiles, so the tile gets narrower (down to 64 weight rows)
// to spread the weights over more SMs; K is never split, so nothing has to be
// joined.  The fused pair needs the largest |h| of each 128 columns: its narrow
// tiles form a cluster of 2 or 4 CTAs that share such a block and exchange each
// row's maximum through distributed shared memory.
#include <atomic>
#include <type_traits>

#include "moe_fp8.cuh"

namespace moe {
namespace {

// SECTORS: the output's rows are whole 32-byte sectors (always with swiglu, or
// MR = 16).
template <bool SWIGLU, int BN, int MR, bool SECTORS>
struct Cfg {
  static constexpr int S = SWIGLU ? 256 / BN : 1;    // CTAs that share a block of 128 columns
  static constexpr int COLS = SWIGLU ? 128 : BN;     // output columns per tile (of the cluster)
  static constexpr int WBOX = SWIGLU ? BN / 2 : BN;  // weight rows per copy
  static constexpr int ABOX = MR < 32 ? MR : 32;     // activation rows per copy
  // K blocks per stage: narrow tiles take several, their barriers cost more
  // than their MMAs
  static constexpr int KU = BN == 256 || (BN == 128 && MR == 128) ? 1 : BN == 128 || MR == 128 ? 2 : 4;
  static constexpr int A_BLK = MR * 128, B_BLK = BN * 128;
  static constexpr int A_BYTES = KU * A_BLK, B_BYTES = KU * B_BLK;  // per stage
  static constexpr int EW = 8;                       // promoting warps: 4 TMEM quarters x PARTS column parts
  static constexpr int PARTS = EW / 4;
  static constexpr int THREADS = (EW + 4) * 32;
  static constexpr int CP = BN / PARTS;              // accumulator columns per thread
  // columns per TMEM load: what fits in registers beside the accumulators
  static constexpr int CH = CP == 128 || (SWIGLU && CP == 32) ? 16 : 32;
  static constexpr int UB = KU * CH > 64 ? 64 / CH : KU;  // K blocks per round of TMEM loads
  // TMEM accumulator sets, one accumulator per K block of a stage
  static constexpr int BUFS = BN * KU >= 256 ? 2 : 4;
  static constexpr int TMEM = BN * KU * BUFS;
  static constexpr int PROMOTERS = MR == 16 ? 2 : EW;
  // Row maxima of a block's parts: [PARTS S][MR] (MR = 16: [S][MR], none alone).
  // A cluster has one tile; a CTA by itself has many, and two buffers for them.
  static constexpr int XCH = MR == 16 ? (S > 1 ? S * MR : 0) : PARTS * S * MR;  // floats
  static constexpr int XCH_BYTES = SWIGLU ? (S > 1 ? 1 : 2) * XCH * 4 : 0;
  // MR = 16: a tile's sums.  Otherwise per lane the values of a store round
  // (without SECTORS), then its output row and the tile's column block.
  static constexpr int PC = BN == 256 ? 8 : 16;
  static constexpr int STG_PITCH = SECTORS ? 2 : PC + 4;
  static constexpr int STG_BYTES = MR == 16 ? 16 * (BN + 4) * 4 : EW * 32 * STG_PITCH * 4;
  static constexpr int LIMIT = 227 * 1024 - 8 * (kMaxExperts + 1) - 1024;  // less tables, alignment
  static constexpr int FIT = (LIMIT - STG_BYTES - XCH_BYTES - 20 * 1024) / (A_BYTES + B_BYTES);
  static constexpr int NS = BN == 256 && MR == 128 ? 4 : FIT > 24 ? 24 : FIT;
  // Scale slots: sa * sw of every row of a K block, for the two column halves
  // (or gate and up).  The scale warp fills block g's slot once the MMAs of
  // block g - NS are done, so the epilogue is past block g - NS - BUFS.
  static constexpr int SLOTS = NS + BUFS;
  static constexpr int SLOT = 2 * MR;                // floats, per K block
  // the activation stages come first: an MR = 16 operand overruns into the
  // weight stages, never out of them
  static constexpr int W0 = NS * A_BYTES;
  static constexpr int STG = NS * (A_BYTES + B_BYTES);
  static constexpr int XCH0 = STG + STG_BYTES;
  static constexpr int SCL = XCH0 + XCH_BYTES;
  static constexpr int CTL = SCL + SLOTS * KU * SLOT * 4; // barriers and flags
  static constexpr int CTL_BYTES = ((2 * NS + 2 * BUFS + SLOTS + 4) * 8 + 4 * (2 + THREADS / 32) + 15) / 16 * 16;
  static constexpr int TAB = CTL + CTL_BYTES;        // int [2][E + 1]: tiles and rows before e
  // registers of a promoting thread (0: no split; the others get what is left of
  // 3 x 168)
  static constexpr int KREG = BN == 256 ? 216 : 0;
  static_assert(NS >= 3 && NS * B_BYTES >= 128 * 128 && TAB <= LIMIT && TMEM <= 512, "shared memory, TMEM");
  static size_t smem(int E) { return size_t(TAB) + 8 * size_t(E + 1) + 1024 /*alignment*/; }
};

// One box holds one K block of 128 bytes; with `deep` (K a multiple of 128) the
// KU blocks of a stage, as a third dimension: one copy instead of KU, and a copy
// costs its warp about 100 clocks.
struct Maps {
  CUtensorMap a;     // A rows: 1-row boxes (gather) or ABOX-row boxes
  CUtensorMap w[2];  // weights, WBOX-row boxes (gate and up, or twice the same)
  int deep;
};

// Rows fetched four at a time: picked by the entries, or too few to fill a box
// (a box that runs past the matrix is slow: T = 1, N = 2048, K = 4096 took
// 12.5 us with 16-row boxes, 8.7 us so).
__host__ __device__ inline bool rows_by_four(const Fp8GemmArgs& a) { return a.a_div > 0 || a.P < 16; }

struct Tile {
  int e, nt;
  int row0;    // first bucket position of the tile
  int nvalid;  // rows
};

// An MMA of M = 64 keeps row r in lane r % 16 of TMEM quarter r / 16 (M = 128:
// lane r % 32 of quarter r / 32).
// The tensor cores then leave the rows alone that do not exist: at T = 2048 on
// 256 experts, where the card runs at its power limit, 4 % less time.
template <bool HALF>
__device__ __forceinline__ bool half_tile(const Tile& t) { return HALF && t.nvalid <= 64; }
// Row of a TMEM lane; past every tile for the lanes that hold none.
template <bool HALF>
__device__ __forceinline__ int row_at(const Tile& t, int place) {
  if (!half_tile<HALF>(t)) return place;
  return (place & 16) ? 1 << 20 : place / 32 * 16 + (place & 15);
}

template <int MR>
__device__ __forceinline__ Tile tile_of(const int* t_off, const int* t_beg, int E,
                                        int it) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t_off[mid] <= it) lo = mid;
    else hi = mid - 1;
  }
  const int li = it - t_off[lo], rows = t_beg[lo + 1] - t_beg[lo];
  const int mtiles = (rows + MR - 1) / MR;
  Tile t;
  t.e = lo;
  t.nt = li / mtiles;  // row tiles fastest: neighbours share the weight tile in L2
  const int mt = li - t.nt * mtiles;
  t.row0 = t_beg[lo] + mt * MR;
  t.nvalid = min(MR, rows - mt * MR);
  return t;
}

// silu(g) u = g u / (1 + e^-g).  The reciprocal is the hardware's (1 unit of 2^-23;
// a division costs gate / up 9 % at T = 2048); beyond g = -88.7, where e^-g leaves
// float32, it is 0 (silu is below 4e-37 there).
__device__ __forceinline__ float silu_mul(float g, float u) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.f + expf(-g)));
  return g * r * u;
}

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

__device__ __forceinline__ void st_sector(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// CP values of one row from column n0 on, 32 bytes a store; n0 and N are
// multiples of the values in 32 bytes.
template <int CP, typename T>
__device__ __forceinline__ void store_sectors(T* out, int N, int n0, const float2 (&v)[CP / 2], int dst) {
  constexpr int E = 32 / sizeof(T);
  T* o = out + size_t(dst) * N + n0;
#pragma unroll
  for (int c = 0; c < CP / E; ++c) {
    if (n0 + c * E >= N) break;
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if constexpr (sizeof(T) == 4) w[k] = __float_as_uint(k & 1 ? v[c * 4 + k / 2].y : v[c * 4 + k / 2].x);
      else w[k] = pack16(std::is_same_v<T, __half> ? MOE_DTYPE_F16 : MOE_DTYPE_BF16, v[c * 8 + k].x, v[c * 8 + k].y);
    }
    st_sector(o + c * E, w);
  }
}

// W consecutive values of one row
template <int W>
__device__ __forceinline__ void store_word(void* out, int type, size_t o, const float* f) {
  if constexpr (W == 1) {
    store_one(out, type, o, f[0]);
  } else if (type == MOE_DTYPE_F32) {
    float* d = static_cast<float*>(out) + o;
    if constexpr (W == 4) *reinterpret_cast<float4*>(d) = *reinterpret_cast<const float4*>(f);
    else *reinterpret_cast<float2*>(d) = *reinterpret_cast<const float2*>(f);
  } else {
    uint16_t* d = static_cast<uint16_t*>(out) + o;
    if constexpr (W == 4) *reinterpret_cast<uint2*>(d) = make_uint2(pack16(type, f[0], f[1]), pack16(type, f[2], f[3]));
    else *reinterpret_cast<uint32_t*>(d) = pack16(type, f[0], f[1]);
  }
}

// A warp's 32 rows x CP columns (lane l: row l in v, its output row dst or -1)
// to rows of any width N, a multiple of W.  They pass through shared memory PC
// columns at a time, so that a store covers runs of a few rows instead of one
// word in each of 32.
template <int W, int CP, int PC>
__device__ __forceinline__ void store_tile(void* out, int type, int N, int n0, const float2 (&v)[CP / 2], float* stg,
                                           int dst) {
  constexpr int PITCH = PC + 4, LPR = PC / W, RPI = 32 / LPR;  // lanes per row, rows per store
  const int lane = threadIdx.x & 31, j = W * (lane % LPR), r0 = lane / LPR;
  int drow[LPR];
#pragma unroll
  for (int i = 0; i < LPR; ++i) drow[i] = __shfl_sync(kFull, dst, i * RPI + r0);
#pragma unroll
  for (int c = 0; c < CP / PC; ++c) {
    if (n0 + c * PC >= N) break;
#pragma unroll
    for (int k = 0; k < PC / 4; ++k)
      *reinterpret_cast<float4*>(stg + lane * PITCH + 4 * k) =
          make_float4(v[c * PC / 2 + 2 * k].x, v[c * PC / 2 + 2 * k].y, v[c * PC / 2 + 2 * k + 1].x,
                      v[c * PC / 2 + 2 * k + 1].y);
    __syncwarp();
    const int n = n0 + c * PC + j;
#pragma unroll
    for (int i = 0; i < LPR; ++i)
      if (drow[i] >= 0 && n < N)
        store_word<W>(out, type, size_t(drow[i]) * N + n, stg + (i * RPI + r0) * PITCH + j);
    __syncwarp();
  }
}

// A stage ring's position.
template <int NS>
struct Ring {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++stage == NS) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

// HALF: tiles of at most 64 rows run as MMAs of M = 64 (buckets; a dense product
// has no use for it, and the code costs it 137 -> 148 us on 4096 x 8192 x 4096).
template <bool SWIGLU, int BN, int MR, bool SECTORS, bool HALF>
__global__ void __launch_bounds__(Cfg<SWIGLU, BN, MR, SECTORS>::THREADS, 1)
    k_gemm_fp8(const __grid_constant__ Fp8GemmArgs a, const __grid_constant__ Maps maps) {
  using C = Cfg<SWIGLU, BN, MR, SECTORS>;
  constexpr int S = C::S, kEpiWarps = C::EW, kThreads = C::THREADS;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::CTL);
  uint64_t* empty = full + C::NS;
  uint64_t* acc_full = empty + C::NS;          // [BUFS]
  uint64_t* acc_empty = acc_full + C::BUFS;    // [BUFS]
  uint64_t* scl_full = acc_empty + C::BUFS;    // [SLOTS]
  uint64_t* drain = scl_full + C::SLOTS;
  uint64_t* xbar = drain + 1;                  // row maxima of the cluster are in place
  uint64_t* stg_full = xbar + 1;               // MR = 16: a tile's sums are in shared memory
  uint64_t* stg_empty = stg_full + 1;          // and have been stored
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(stg_empty + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* xch = reinterpret_cast<float*>(smem + C::XCH0);
  float* scl = reinterpret_cast<float*>(smem + C::SCL);
  int* s_part = const_cast<int*>(abort_flag) + 1;  // [warps]
  int* t_off = reinterpret_cast<int*>(smem + C::TAB);
  int* t_beg = t_off + (a.E + 1);

  const int warp = __shfl_sync(kFull, int(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
  const int rank = S > 1 ? int(cluster_rank()) : 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NS; ++s) {
      bar_init(smem_addr(&full[s]), 3);  // the weights', the rows' and the scales' producer
      bar_init(smem_addr(&empty[s]), 1);
    }
    for (int b = 0; b < C::BUFS; ++b) {
      bar_init(smem_addr(&acc_full[b]), 1);
      bar_init(smem_addr(&acc_empty[b]), C::PROMOTERS);
    }
    for (int s = 0; s < C::SLOTS; ++s) bar_init(smem_addr(&scl_full[s]), 1);
    bar_init(smem_addr(drain), 1);
    bar_init(smem_addr(xbar), (MR == 16 ? kEpiWarps - 2 : kEpiWarps) * S);
    bar_init(smem_addr(stg_full), 2);
    bar_init(smem_addr(stg_empty), kEpiWarps - 2);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.a) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.w[0]) : "memory");
    if (SWIGLU) asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.w[1]) : "memory");
  }
  if (warp == kEpiWarps + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tmem_slot)),
                 "r"(C::TMEM)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  const int NT = (a.N + C::COLS - 1) / C::COLS;
  if (a.offsets == nullptr && threadIdx.x == 0) {  // one group of all rows
    t_off[0] = t_beg[0] = 0;
    t_off[1] = (a.P + MR - 1) / MR * NT;
    t_beg[1] = a.P;
  }
  tcgen_fence_before();
  if (S > 1) cluster_barrier();  // the other CTAs' barriers exist before anyone arrives on them
  else __syncthreads();
  tcgen_fence_after();
  const uint32_t tmem = *tmem_slot;
  // everything above runs while the kernel before drains; from here on memory
  // is read (a dense product goes straight to its copies)
  pdl_wait();
  pdl_trigger();

  // rows and tiles before every bucket: a thread takes PER neighbouring
  // buckets, warps scan their sums, and everyone adds the warps before its own.
  // Offsets that are not ascending inside [0, P] stop the whole call (latched,
  // nothing written).
  if (a.offsets != nullptr) {
    constexpr int PER = (kMaxExperts + kThreads - 1) / kThreads;
    const int per = (a.E + kThreads - 1) / kThreads;
    int beg[PER + 1], sum = 0, bad = 0;
#pragma unroll
    for (int j = 0; j <= PER; ++j) {
      const int e = int(threadIdx.x) * per + j;
      beg[j] = j <= per && e <= a.E ? a.offsets[e] : 0;
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int e = int(threadIdx.x) * per + j;
      if (j < per && e < a.E) {
        bad |= beg[j] < 0 || beg[j + 1] < beg[j] || beg[j + 1] > a.P;
        sum += (beg[j + 1] - beg[j] + MR - 1) / MR * NT;
      }
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) s_part[warp] = inc;
    bad = __syncthreads_or(bad);
    if (bad && threadIdx.x == 0) latch_error(a.err, MOE_ERR_DEVICE_DATA, 500);
    int run = inc - sum;
    for (int w = 0; w < warp; ++w) run += s_part[w];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int e = int(threadIdx.x) * per + j;
      if (j < per && e < a.E) {
        t_off[e] = run;
        t_beg[e] = beg[j];
        run += (beg[j + 1] - beg[j] + MR - 1) / MR * NT;
        if (e == a.E - 1) {
          t_off[a.E] = bad ? 0 : run;
          t_beg[a.E] = beg[j + 1];
        }
      }
    }
    __syncthreads();
  }
  const int n_tiles = t_off[a.E];
  const int KB = fp8_blocks(a.K), KG = (KB + C::KU - 1) / C::KU;  // K blocks, stages of them
  const int first = blockIdx.x / S, step = gridDim.x / S;
  const bool gather = a.a_div > 0, scatter = a.scatter;
  const bool by_row = MR == 16 ? rows_by_four(a) : gather;
  const WaitCtl ctl{abort_flag, a.err};

  // the end of every role.  (Each side of the register split calls it by itself
  // and returns: where the two meet again, ptxas holds both to the launch's
  // registers and the accumulators spill.)
  auto finish = [&] {
    __syncwarp();
    tcgen_fence_before();
    if (S > 1) cluster_barrier();  // no CTA leaves while another may write its maxima
    else __syncthreads();
    if (*abort_flag) {
      // Given up, and nobody issues copies any more.  A stage's barrier may lack
      // a producer for good, so those in flight get a millisecond, far beyond
      // any copy's time, before the CTA leaves its shared memory.
      const unsigned long long t0 = global_ns();
      while (global_ns() - t0 < 1000000ull) {
      }
    }
    if (warp == kEpiWarps + 1) {
      tcgen_fence_after();
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM)
                   : "memory");
    }
  };

  // Gathered rows: four at a time, one copy per lane.  A warp's lanes issue
  // their copies one after the other, about 40 clocks each, so a full tile's 32
  // copies are shared by the two producers (even groups of four, odd groups).
  constexpr int GW = MR == 128 ? 2 : 1;
  auto group_of = [&](int g) { return GW * lane + g; };
  auto gather_rows = [&](const Tile& t, int g, int (&r)[4]) {
    // positions past the bucket repeat its last row, an index out of range
    // reads row 0
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      int src = t.row0 + min(4 * group_of(g) + j, t.nvalid - 1);
      if (gather) src = a.entries[src] / a.a_div;
      r[j] = src >= 0 && src < a.a_rows ? src : 0;
    }
  };
  // bytes a producer's groups bring per K block
  auto gather_bytes = [&](const Tile& t, int g) { return uint32_t(((t.nvalid + 3) / 4 - g + GW - 1) / GW * 512); };
  auto gather_block = [&](const Tile& t, int g, const int (&r)[4], uint32_t to, int x, uint32_t fb) {
    const int i = group_of(g);
    if (i < MR / 4 && 4 * i < t.nvalid) tma_gather4(to + i * 512, &maps.a, x, r[0], r[1], r[2], r[3], fb);
  };

  if (warp >= kEpiWarps) {
    if constexpr (C::KREG != 0) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(504 - 2 * C::KREG));
    if (warp == kEpiWarps) {
      // ------------------------------------------------------ weight producer
      // (a pair's gate and up rows alternate by K block, so it takes them singly)
      constexpr bool DEEP_W = C::KU > 1 && !SWIGLU;
      Ring<C::NS> ring;
      uint64_t keep, once;
      asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(keep));
      asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
      bool ok = true;
      for (int it = first; it < n_tiles && ok; it += step) {
        const Tile t = tile_of<MR>(t_off, t_beg, a.E, it);
        // weights that one row tile alone reads are not worth keeping in L2
        const uint64_t pol = t_beg[t.e + 1] - t_beg[t.e] <= MR ? once : keep;
        const int wrow = t.e * a.N + t.nt * C::COLS + rank * C::WBOX;
        const bool rows = GW == 2 && by_row;
        int r[4] = {0, 0, 0, 0};
        if (rows) gather_rows(t, 1, r);
        const uint32_t bytes = C::B_BLK + (rows ? gather_bytes(t, 1) : 0);
        for (int kg = 0; kg < KG; ++kg, ring.next()) {
          ok = bar_wait(smem_addr(&empty[ring.stage]), ring.phase ^ 1u, ctl, 510);
          if (!ok) break;
          const uint32_t w = smem_addr(smem + C::W0 + ring.stage * C::B_BYTES);
          const uint32_t fb = smem_addr(&full[ring.stage]);
          if (elect_one()) {
            const int kn = min(C::KU, KB - kg * C::KU);
            if (DEEP_W && maps.deep) {  // blocks past K arrive as zeros
              bar_expect(fb, C::B_BYTES + kn * (bytes - C::B_BLK));
              tma_3d(w, &maps.w[0], kg * C::KU, wrow, fb, pol);
            } else {
              bar_expect(fb, kn * bytes);
#pragma unroll
              for (int u = 0; u < C::KU; ++u) {
                if (u >= kn) break;
                const int x = (kg * C::KU + u) * 128;
                tma_2d(w + u * C::B_BLK, &maps.w[0], x, wrow, fb, pol);
                if (SWIGLU) tma_2d(w + u * C::B_BLK + C::WBOX * 128, &maps.w[1], x, wrow, fb, pol);
              }
            }
          }
          __syncwarp();
          if (rows) {
            const uint32_t st = smem_addr(smem + ring.stage * C::A_BYTES);
#pragma unroll
            for (int u = 0; u < C::KU; ++u)
              if (kg * C::KU + u < KB) gather_block(t, 1, r, st + u * C::A_BLK, (kg * C::KU + u) * 128, fb);
            __syncwarp();
          }
        }
      }
    } else if (warp == kEpiWarps + 2) {
      // --------------------------------------------------------- row producer
      constexpr bool DEEP_A = C::KU > 1 && MR == C::ABOX;  // a block's rows are one box
      Ring<C::NS> ring;
      uint64_t keep;
      asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(keep));
      bool ok = true;
      for (int it = first; it < n_tiles && ok; it += step) {
        const Tile t = tile_of<MR>(t_off, t_beg, a.E, it);
        int r[4] = {0, 0, 0, 0};
        if (by_row) gather_rows(t, 0, r);
        const uint32_t bytes = by_row ? gather_bytes(t, 0) : (t.nvalid + C::ABOX - 1) / C::ABOX * C::ABOX * 128;
        for (int kg = 0; kg < KG; ++kg, ring.next()) {
          ok = bar_wait(smem_addr(&empty[ring.stage]), ring.phase ^ 1u, ctl, 511);
          if (!ok) break;
          const uint32_t st = smem_addr(smem + ring.stage * C::A_BYTES), fb = smem_addr(&full[ring.stage]);
          const int kn = min(C::KU, KB - kg * C::KU);
          const bool deep = DEEP_A && maps.deep && !by_row;
          if (elect_one()) bar_expect(fb, (deep ? C::KU : kn) * bytes);
          __syncwarp();
          if (deep) {
            if (elect_one()) tma_3d(st, &maps.a, kg * C::KU, t.row0, fb, keep);
            __syncwarp();
            continue;
          }
#pragma unroll
          for (int u = 0; u < C::KU; ++u) {
            if (u >= kn) break;
            const int x = (kg * C::KU + u) * 128;
            const uint32_t to = st + u * C::A_BLK;
            if (by_row) {
              gather_block(t, 0, r, to, x, fb);
            } else if (elect_one()) {
#pragma unroll
              for (int j = 0; j < MR / C::ABOX; ++j)
                if (C::ABOX * j < t.nvalid)
                  tma_2d(to + j * C::ABOX * 128, &maps.a, x, t.row0 + C::ABOX * j, fb, keep);
            }
          }
          __syncwarp();
        }
      }
    } else if (warp == kEpiWarps + 3) {
      // ------------------------------------------------------- scale producer
      // lane l holds the rows of TMEM lanes l, l + 32, .. and both weight scales
      // (the column halves' blocks, or gate and up).  UK K blocks a round, and
      // the next round's loads in flight: their latency is several stages'.
      constexpr int RJ = (MR + 31) / 32, UK = MR == 16 ? 8 : 2, UG = UK / C::KU;
      Ring<C::NS> ring;
      Ring<C::SLOTS> slot;
      const int NB = fp8_blocks(a.N);
      // debug switch: the first stage's scales never arrive, so the bounded waits
      // for it run out
      const unsigned debug = *(reinterpret_cast<const volatile unsigned*>(a.err) + 3);
      bool starve = (debug & MOE_DEBUG_STARVE_FIRST_WAIT) && blockIdx.x == 0;
      bool ok = true;
      for (int it = first; it < n_tiles && ok; it += step) {
        const Tile t = tile_of<MR>(t_off, t_beg, a.E, it);
        const float* sa[RJ];
#pragma unroll
        for (int j = 0; j < RJ; ++j) {
          int src = t.row0 + min(row_at<HALF>(t, lane + 32 * j), t.nvalid - 1);
          if (gather) src = a.entries[src] / a.a_div;
          sa[j] = a.a_s + size_t(src >= 0 && src < a.a_rows ? src : 0) * KB;
        }
        const float* sw[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int nb = SWIGLU ? t.nt : min((t.nt * BN + h * (BN / 2)) / kFp8Block, NB - 1);
          sw[h] = a.w_s[SWIGLU ? h : 0] + (size_t(t.e) * NB + nb) * KB;
        }
        float next_a[UK][RJ], next_w[UK][2];
        auto load = [&](int kg) {
#pragma unroll
          for (int u = 0; u < UK; ++u) {
            const int k = min(kg * C::KU + u, KB - 1);
#pragma unroll
            for (int j = 0; j < RJ; ++j) next_a[u][j] = sa[j][k];
            next_w[u][0] = sw[0][k];
            next_w[u][1] = sw[1][k];
          }
        };
        load(0);
        for (int kg = 0; kg < KG && ok; kg += UG) {
          float va[UK][RJ], vw[UK][2];
#pragma unroll
          for (int u = 0; u < UK; ++u) {
#pragma unroll
            for (int j = 0; j < RJ; ++j) va[u][j] = next_a[u][j];
            vw[u][0] = next_w[u][0];
            vw[u][1] = next_w[u][1];
          }
          if (kg + UG < KG) load(kg + UG);
#pragma unroll
          for (int g = 0; g < UG; ++g) {
            if (kg + g >= KG) break;
            ok = bar_wait(smem_addr(&empty[ring.stage]), ring.phase ^ 1u, ctl, 512);
            if (!ok) break;
#pragma unroll
            for (int u = 0; u < C::KU; ++u) {
              float* to = scl + (slot.stage * C::KU + u) * C::SLOT;
              const int i = g * C::KU + u;
#pragma unroll
              for (int j = 0; j < RJ; ++j)
                if (MR >= 32 || lane < MR) {
                  to[lane + 32 * j] = va[i][j] * vw[i][0];
                  to[MR + lane + 32 * j] = va[i][j] * vw[i][1];
                }
            }
            __syncwarp();
            if (lane == 0 && !starve) {
              bar_arrive(smem_addr(&scl_full[slot.stage]));
              // the MMAs wait for this warp too: it must not fall a round of
              // the ring behind, where the empty barrier's parity repeats
              bar_arrive(smem_addr(&full[ring.stage]));
            }
            starve = false;
            ring.next();
            slot.next();
          }
        }
      }
    } else if (warp == kEpiWarps + 1) {
      // ----------------------------------------------------------------- MMA
      Ring<C::NS> ring;
      Ring<C::BUFS> acc;
      bool ok = true;
      const uint64_t da0 = desc_k_sw128(smem_addr(smem)), dw0 = desc_k_sw128(smem_addr(smem + C::W0));
      // one tile's MMAs
      auto issue = [&](auto m) {
        constexpr uint32_t idesc = idesc_e4m3(decltype(m)::value, BN);
        for (int kg = 0; kg < KG; ++kg, ring.next(), acc.next()) {
          ok = bar_wait(smem_addr(&acc_empty[acc.stage]), acc.phase ^ 1u, ctl, 520) &&
               bar_wait(smem_addr(&full[ring.stage]), ring.phase, ctl, 521);
          if (!ok) return;
          tcgen_fence_after();
          const int left = a.K - kg * C::KU * 128;  // a tail of K reads zero fill to its next 32
          if (elect_one()) {
#pragma unroll
            for (int u = 0; u < C::KU; ++u) {
              // descriptors count addresses in units of 16 bytes
              const uint64_t da = da0 + uint32_t((ring.stage * C::A_BYTES + u * C::A_BLK) / 16);
              const uint64_t dw = dw0 + uint32_t((ring.stage * C::B_BYTES + u * C::B_BLK) / 16);
              const uint32_t d = tmem + (acc.stage * C::KU + u) * BN;
              if (left > u * 128) mma_e4m3(d, da, dw, idesc, 0);
              if (left > u * 128 + 32) mma_e4m3(d, da + 2, dw + 2, idesc, 1);
              if (left > u * 128 + 64) mma_e4m3(d, da + 4, dw + 4, idesc, 1);
              if (left > u * 128 + 96) mma_e4m3(d, da + 6, dw + 6, idesc, 1);
            }
            tcgen_commit(smem_addr(&empty[ring.stage]));
            tcgen_commit(smem_addr(&acc_full[acc.stage]));
          }
          __syncwarp();
        }
      };
      for (int it = first; it < n_tiles && ok; it += step) {
        if (MR == 16 || half_tile<HALF>(tile_of<MR>(t_off, t_beg, a.E, it))) issue(std::integral_constant<int, 64>{});
        else issue(std::integral_constant<int, 128>{});
      }
      if (!ok || *abort_flag) {
        // let issued MMAs finish before TMEM is released (bounded)
        if (elect_one()) tcgen_commit(smem_addr(drain));
        const unsigned long long t0 = global_ns();
        while (!bar_try(smem_addr(drain), 0) && global_ns() - t0 < 200000000ull) {
        }
      }
    }
    finish();
  } else {
    // --------------------------------------------------- promotion, epilogue
    if constexpr (C::KREG != 0) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::KREG));
    const int q = warp & 3, part = warp >> 2;
    const int place = 32 * q + lane;  // TMEM lane: scale slots and maxima go by it
    const int NB = fp8_blocks(a.N);
    Ring<C::BUFS> acc;
    Ring<C::SLOTS> slot;
    uint32_t local = 0;  // tiles so far
    // column of this part's value o (swiglu: its gate, then its up columns)
    constexpr int HP = C::CP / 2;
    auto at = [&](int o) { return SWIGLU ? (o < HP ? o : BN / 2 + o - HP) + part * HP : part * C::CP + o; };
    // the sums of one tile over K; work: this warp's rows exist
    auto promote = [&](float2 (&v)[C::CP / 2], bool work) {
#pragma unroll
      for (int j = 0; j < C::CP / 2; ++j) v[j] = make_float2(0.f, 0.f);
      float s0[C::KU], s1[C::KU];
      auto scales = [&] {
        if (!bar_wait(smem_addr(&scl_full[slot.stage]), slot.phase, ctl, 531)) return false;
        const float* sc = scl + slot.stage * C::KU * C::SLOT + (MR >= 128 ? place : place & (MR - 1));
#pragma unroll
        for (int u = 0; u < C::KU; ++u) {
          s0[u] = sc[u * C::SLOT + (SWIGLU ? 0 : part * MR)];
          s1[u] = SWIGLU ? sc[u * C::SLOT + MR] : 0.f;
        }
        slot.next();
        return true;
      };
      for (int kg = 0; kg < KG; ++kg, acc.next()) {
        const int kn = min(C::KU, KB - kg * C::KU);
        if (!scales()) return false;
        if (!bar_wait(smem_addr(&acc_full[acc.stage]), acc.phase, ctl, 530)) return false;
        auto release = [&] {  // the MMAs may have the buffer
          tcgen_fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(smem_addr(&acc_empty[acc.stage]));
        };
        if (work) {
          tcgen_fence_after();
          const uint32_t col = tmem + acc.stage * C::KU * BN + (uint32_t(32 * q) << 16);
          constexpr int CH = C::CH, UB = C::UB, NCH = C::CP / CH;
#pragma unroll
          for (int c = 0; c < NCH; ++c) {
#pragma unroll
            for (int u0 = 0; u0 < C::KU; u0 += UB) {
              // a short last stage reads an old accumulator and leaves it out
              uint32_t d[UB][CH];
#pragma unroll
              for (int u = 0; u < UB; ++u) tmem_load<CH>(col + (u0 + u) * BN + at(c * CH), d[u]);
#pragma unroll
              for (int u = 0; u < UB; ++u) tmem_wait<CH>(d[u]);
              if (c + 1 == NCH && u0 + UB >= C::KU) release();
#pragma unroll
              for (int u = 0; u < UB; ++u) {
                if (u0 + u >= kn) break;
                const float s = SWIGLU && c * CH >= HP ? s1[u0 + u] : s0[u0 + u];
#pragma unroll
                for (int j = 0; j < CH / 2; ++j)
                  fma_pair(v[c * CH / 2 + j], d[u][2 * j], d[u][2 * j + 1], make_float2(s, s));
              }
            }
          }
        } else {
          release();
        }
      }
      return true;
    };
    // output row of bucket position p, or -1 (latched) for an entry that names
    // no row
    auto out_row = [&](int p) {
      if (!gather && !scatter) return p;
      const int ent = a.entries[p];
      if (ent < 0 || (gather && ent / a.a_div >= a.a_rows) || (scatter && ent >= a.P)) {
        latch_error(a.err, MOE_ERR_DEVICE_DATA, 501);
        return -1;
      }
      return scatter ? ent : p;
    };
    if constexpr (MR == 16) {
      // Only TMEM quarter 0 holds rows: its two warps promote, leave the tile in
      // shared memory and go on; the other six store it meanwhile.
      constexpr int PITCH = BN + 4;
      float* buf = reinterpret_cast<float*>(smem + C::STG);
      if (q == 0) {
        for (int it = first; it < n_tiles; it += step, ++local) {
          float2 v[C::CP / 2];
          if (!promote(v, true) || !bar_wait(smem_addr(stg_empty), (local & 1u) ^ 1u, ctl, 541)) break;
          if (lane < 16) {
#pragma unroll
            for (int j = 0; j < C::CP / 4; ++j)
              *reinterpret_cast<float4*>(buf + lane * PITCH + at(4 * j)) =
                  make_float4(v[2 * j].x, v[2 * j].y, v[2 * j + 1].x, v[2 * j + 1].y);
          }
          __syncwarp();
          if (lane == 0) bar_arrive(smem_addr(stg_full));
        }
      } else {
        const int hw = warp - (part ? 2 : 1);  // 0 .. 5
        for (int it = first; it < n_tiles; it += step, ++local) {
          const Tile t = tile_of<MR>(t_off, t_beg, a.E, it);
          const int dst = lane < t.nvalid ? out_row(t.row0 + lane) : -1;  // of row `lane`
          if (!bar_wait(smem_addr(stg_full), local & 1u, ctl, 542)) break;
          if constexpr (SWIGLU) {
            // a warp per row, up to three of them; CPL columns per lane
            constexpr int HC = BN / 2, CPL = HC / 32, HR = 3;
            const int c = lane * CPL, n = t.nt * 128 + rank * HC + c;
            float h[HR][CPL], amax[HR];
#pragma unroll
            for (int i = 0; i < HR; ++i) {
              const int r = hw + 6 * i;
              amax[i] = 0.f;
#pragma unroll
              for (int j = 0; j < CPL; ++j) {
                h[i][j] = 0.f;
                if (r < t.nvalid && n + j < a.N)
                  h[i][j] = silu_mul(buf[r * PITCH + c + j], buf[r * PITCH + HC + c + j]);
                amax[i] = fmaxf(amax[i], fabsf(h[i][j]));
              }
#pragma unroll
              for (int o = 16; o > 0; o >>= 1) amax[i] = fmaxf(amax[i], __shfl_xor_sync(kFull, amax[i], o));
            }
            if constexpr (S > 1) {
              // the block's other columns are in the cluster's other CTAs (and
              // this is its one tile)
              if (lane < S) {
#pragma unroll
                for (int i = 0; i < HR; ++i)
                  if (hw + 6 * i < t.nvalid)
                    cluster_st(cluster_map(smem_addr(xch + rank * MR + hw + 6 * i), lane), amax[i]);
                cluster_arrive(cluster_map(smem_addr(xbar), lane));
              }
              __syncwarp();
              if (!bar_wait<true>(smem_addr(xbar), 0, ctl, 540)) break;
#pragma unroll
              for (int i = 0; i < HR; ++i)
                if (hw + 6 * i < t.nvalid)
#pragma unroll
                  for (int k = 0; k < S; ++k) amax[i] = fmaxf(amax[i], xch[k * MR + hw + 6 * i]);
            }
#pragma unroll
            for (int i = 0; i < HR; ++i) {
              const int r = hw + 6 * i;
              if (r >= t.nvalid) break;
              const int drow = __shfl_sync(kFull, dst, r);
              if (drow < 0) continue;
              const float s = fp8_scale(amax[i]);
              if (lane == 0 && rank == 0) a.s_out[size_t(drow) * NB + t.nt] = s;
              if (n < a.N) {  // N is a multiple of 16
                uint8_t* o = a.q_out + size_t(drow) * a.N + n;
                float2 hp[(CPL + 1) / 2];
#pragma unroll
                for (int j = 0; j < (CPL + 1) / 2; ++j)
                  hp[j] = make_float2(h[i][2 * j], 2 * j + 1 < CPL ? h[i][(2 * j + 1) % CPL] : 0.f);
                uint32_t code[1];
                fp8_codes(hp, s, code);
                if constexpr (CPL == 4) *reinterpret_cast<uint32_t*>(o) = code[0];
                else if constexpr (CPL == 2) *reinterpret_cast<uint16_t*>(o) = uint16_t(code[0]);
                else *o = uint8_t(code[0]);
              }
            }
          } else {
            // four columns of a row per lane, all rows' quads in turn
            constexpr int QUADS = BN / 4;
            const bool vec = a.N % 4 == 0;
            for (int b = hw * 32; b < t.nvalid * QUADS; b += 6 * 32) {
              const int r = (b + lane) / QUADS, j = 4 * ((b + lane) % QUADS);
              const int drow = __shfl_sync(kFull, dst, r & 15), left = a.N - t.nt * BN - j;
              if (r >= t.nvalid || drow < 0 || left <= 0) continue;
              const float4 f = *reinterpret_cast<const float4*>(buf + r * PITCH + j);
              const size_t o = size_t(drow) * a.N + t.nt * BN + j;
              if (!vec) {
                store_one(a.out, a.out_type, o, f.x);
                if (left > 1) store_one(a.out, a.out_type, o + 1, f.y);
                if (left > 2) store_one(a.out, a.out_type, o + 2, f.z);
                if (left > 3) store_one(a.out, a.out_type, o + 3, f.w);
              } else if (a.out_type == MOE_DTYPE_F32) {
                *reinterpret_cast<float4*>(static_cast<float*>(a.out) + o) = f;
              } else {
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + o) =
                    make_uint2(pack16(a.out_type, f.x, f.y), pack16(a.out_type, f.z, f.w));
              }
            }
          }
          __syncwarp();
          if (lane == 0) bar_arrive(smem_addr(stg_empty));
        }
      }
      finish();
      return;
    }
    float* stg = reinterpret_cast<float*>(smem + C::STG) + warp * 32 * C::STG_PITCH;
    // what the tile's end needs waits in shared memory: the registers are the
    // accumulators'
    volatile int* park = reinterpret_cast<volatile int*>(stg + lane * C::STG_PITCH) + (SECTORS ? 0 : C::PC);
    for (int it = first; it < n_tiles; it += step, ++local) {
      bool work;
      {
        const Tile t = tile_of<MR>(t_off, t_beg, a.E, it);
        const int r = row_at<HALF>(t, place);
        work = row_at<HALF>(t, 32 * q) < t.nvalid;
        park[0] = r < t.nvalid ? out_row(t.row0 + r) : -1;
        park[1] = t.nt;
      }
      float2 v[C::CP / 2];
      if (!promote(v, work)) break;
      const int dst = park[0], nt = park[1];  // output row, negative: none
      if constexpr (SWIGLU) {
        // h in place of the gate values, and its largest magnitude over the
        // block's 128 columns (PARTS here, in each of S CTAs).  A CTA by itself
        // has two exchange buffers: who writes one again has seen everyone arrive
        // for the other, and they arrive after their reads.
        const int n0 = nt * 128 + rank * C::WBOX + part * HP;
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < HP / 2; ++j) {
          v[j].x = silu_mul(v[j].x, v[HP / 2 + j].x);
          v[j].y = silu_mul(v[j].y, v[HP / 2 + j].y);
          if (n0 + 2 * j < a.N) amax = fmaxf(amax, fmaxf(fabsf(v[j].x), fabsf(v[j].y)));
        }
        const uint32_t turn = S > 1 ? 0 : local & 1u;
        float* x = xch + turn * C::XCH;
        float* mine = x + (C::PARTS * rank + part) * MR + place;
        if constexpr (S > 1) {
#pragma unroll
          for (int k = 0; k < S; ++k) cluster_st(cluster_map(smem_addr(mine), k), amax);
        } else {
          *mine = amax;
        }
        __syncwarp();
        if (lane < S) {
          if (S > 1) cluster_arrive(cluster_map(smem_addr(xbar), lane));
          else bar_arrive(smem_addr(xbar));
        }
        if (!bar_wait<(S > 1)>(smem_addr(xbar), turn, ctl, 540)) break;
#pragma unroll
        for (int k = 0; k < C::PARTS * S; ++k) amax = fmaxf(amax, x[k * MR + place]);
        if (dst >= 0 && n0 < a.N) {
          const float s = fp8_scale(amax);
          if (part == 0 && rank == 0) a.s_out[size_t(dst) * NB + nt] = s;
          uint8_t* o = a.q_out + size_t(dst) * a.N + n0;
#pragma unroll
          for (int j = 0; j < HP / 16; ++j)
            if (n0 + 16 * j < a.N) {  // N is a multiple of 16
              float2 h[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) h[i] = v[8 * j + i];
              uint32_t code[4];
              fp8_codes(h, s, code);
              *reinterpret_cast<uint4*>(o + 16 * j) = make_uint4(code[0], code[1], code[2], code[3]);
            }
        }
      } else if (work) {
        const int n0 = nt * BN + part * C::CP;
        if constexpr (SECTORS) {
          // every lane stores its own row, 32 bytes a time
          if (dst >= 0) {
            if (a.out_type == MOE_DTYPE_F32) store_sectors<C::CP>(static_cast<float*>(a.out), a.N, n0, v, dst);
            else if (a.out_type == MOE_DTYPE_BF16) store_sectors<C::CP>(static_cast<__nv_bfloat16*>(a.out), a.N, n0, v, dst);
            else store_sectors<C::CP>(static_cast<__half*>(a.out), a.N, n0, v, dst);
          }
        } else {
          // words that stay aligned in every row.  (In a kernel of its own: its
          // code costs the K loop registers, 142 -> 157 us on 4096 x 8192 x 4096.)
          if (a.N % 4 == 0) store_tile<4, C::CP, C::PC>(a.out, a.out_type, a.N, n0, v, stg, dst);
          else if (a.N % 2 == 0) store_tile<2, C::CP, C::PC>(a.out, a.out_type, a.N, n0, v, stg, dst);
          else store_tile<1, C::CP, C::PC>(a.out, a.out_type, a.N, n0, v, stg, dst);
        }
      }
    }
    finish();
  }
}

// --------------------------------------------------------------- host side ---
// Map of a [rows, K] code matrix: boxes of box_rows x 128 bytes (128-byte
// swizzle); depth > 0 (K a multiple of 128): boxes of `depth` neighbouring K
// blocks, one block's rows after the other's.
bool make_map(CUtensorMap* m, const uint8_t* base, uint64_t K, uint64_t rows, uint32_t box_rows, uint32_t depth) {
  if (depth == 0) return make_tma_map_u8_box(m, base, K, rows, 128, box_rows);
  return make_tma_map_u8_deep(m, base, K, rows, box_rows, depth);
}

template <bool SWIGLU, int BN, int MR, bool SECTORS, bool HALF>
cudaError_t launch_kernel(const Fp8GemmArgs& a, long long max_tiles, cudaStream_t st) {
  using C = Cfg<SWIGLU, BN, MR, SECTORS>;
  Maps m;
  const uint64_t wrows = uint64_t(a.E) * a.N;
  m.deep = C::KU > 1 && a.K % 128 == 0;
  const bool four = rows_by_four(a), deep_a = m.deep && C::ABOX == MR && !four, deep_w = m.deep && !SWIGLU;
  if (!make_map(&m.a, a.a_q, a.K, a.a_rows, four ? 1 : C::ABOX, deep_a ? C::KU : 0) ||
      !make_map(&m.w[0], a.w_q[0], a.K, wrows, C::WBOX, deep_w ? C::KU : 0))
    return cudaErrorInvalidValue;
  m.w[1] = m.w[0];
  if (SWIGLU && !make_map(&m.w[1], a.w_q[1], a.K, wrows, C::WBOX, 0)) return cudaErrorInvalidValue;
  auto kern = k_gemm_fp8<SWIGLU, BN, MR, SECTORS, HALF>;
  const size_t smem = C::smem(a.E);
  // the kernel's shared-memory limit, set once per device
  static std::atomic<unsigned long long> set{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (dev >= 64 || !(set.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(C::smem(kMaxExperts)));
    if (e != cudaSuccess) return e;
    set.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  const long long most = device_info().sm_count / C::S;
  if (C::S > 1 && max_tiles > most) return cudaErrorInvalidValue;  // a cluster exchanges its maxima once
  cfg.gridDim = dim3(unsigned((max_tiles < most ? max_tiles : most) * C::S));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(C::S);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C::S > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, a, m);
}

template <bool SWIGLU, int BN, int MR>
cudaError_t launch(const Fp8GemmArgs& a, long long max_tiles, cudaStream_t st) {
  if constexpr (!SWIGLU && MR == 128) {
    const int per = a.out_type == MOE_DTYPE_F32 ? 8 : 16;  // values in a sector
    const bool sectors = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0 && a.N % per == 0;
    if (a.offsets == nullptr)
      return sectors ? launch_kernel<false, BN, MR, true, false>(a, max_tiles, st)
                     : launch_kernel<false, BN, MR, false, false>(a, max_tiles, st);
    if (!sectors) return launch_kernel<false, BN, MR, false, true>(a, max_tiles, st);
  }
  return launch_kernel<SWIGLU, BN, MR, true, true>(a, max_tiles, st);
}

template <int MR>
cudaError_t pick(const Fp8GemmArgs& a, bool swiglu, cudaStream_t st) {
  const long long sms = device_info().sm_count;
  // row tiles at most: one per non-empty bucket, plus one per MR rows
  const long long groups = a.offsets ? (a.E < a.P ? a.E : a.P) : 1;
  const long long rt = a.offsets ? groups + a.P / MR : (a.P + MR - 1) / MR;
  if (swiglu) {
    const long long t = rt * ((a.N + 127) / 128);
    // a cluster shares a block of 128 columns while all clusters fit at once, one
    // tile each (T = 1, one expert of I = 2048, H = 4096: 10.0 us with 4 CTAs, 12.3
    // with 2, 17.0 with 1, 18.6 with 8; T = 1, k = 4: 17.6 with 2, 18.8 with 1)
    if (t * 4 <= sms) return launch<true, 64, MR>(a, t, st);
    if (t * 2 <= sms) return launch<true, 128, MR>(a, t, st);
    return launch<true, 256, MR>(a, t, st);
  }
  // An MMA costs about the same for 16 to 128 weight rows, and every column
  // tile reads the rows again, so tiles below 64 columns lose what their number
  // gains (T = 1, N = 4096, K = 2048: 9.2 us at 16 columns, 7.3 at 32, 6.6 at
  // 64, 7.3 at 128).  Small buckets stream weights: 128 columns once the tiles
  // outnumber the SMs (T = 5, k = 8, 256 experts of N = 4096, K = 2048: 55.2 us
  // at 64, 51.6 at 128, 54.7 at 256).  Full tiles take the narrowest whose tiles
  // all fit the SMs at once, and 256 columns where none do (T = 300, N = 2048, K =
  // 4096: 12.8 us at 64, 15.2 at 128; T = 512, N = 4096: 21.7 at 64, 17.0 at 128,
  // 20.1 at 256).
  auto tiles = [&](int bn) { return rt * ((a.N + bn - 1) / bn); };
  if constexpr (MR == 16) {
    return tiles(128) > sms ? launch<false, 128, MR>(a, tiles(128), st) : launch<false, 64, MR>(a, tiles(64), st);
  } else {
    if (tiles(64) <= sms) return launch<false, 64, MR>(a, tiles(64), st);
    if (tiles(128) <= sms) return launch<false, 128, MR>(a, tiles(128), st);
    return launch<false, 256, MR>(a, tiles(256), st);
  }
}

}  // namespace

cudaError_t launch_gemm_fp8(const Fp8GemmArgs& a, bool swiglu, cudaStream_t st) {
  if (a.P == 0) return cudaSuccess;
  const bool small = a.P <= 16 || (a.offsets && a.P <= 8LL * a.E);
  return small ? pick<16>(a, swiglu, st) : pick<128>(a, swiglu, st);
}

}  // namespace moe

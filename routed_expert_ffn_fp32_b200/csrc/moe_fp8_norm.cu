// Residual addition, root-mean-square norm and E4M3 quantisation of token rows
// in one pass: what stands in front of the layer's 8-bit projections.
//
//   v = x + r,  n = v * rsqrt(mean(v^2) + eps) * w          (float32)
//   per 128 values: s = max(max|n| / 448, 2^-126), q = e4m3(n / s)
//
// One CTA per row.  The row is read once into registers, so the traffic is the
// algorithmic one: bf16 rows of 4096 with residual and all outputs move 9 bytes
// a value, 151 MB at T = 4096, in 27.6 us (5.5 TB/s, 83 % of a plain copy).
// Bound by HBM when rows are many, by two dependent memory latencies (row,
// weight) and the launch when they are few (2.3 us at T = 1).
// A thread owns 8 consecutive values per chunk (16-byte loads of 16-bit types),
// 16 neighbouring lanes own a block of 128, and the row's sum of squares is
// reduced with shuffles and one exchange between the row's warps.
#include "moe_fp8.cuh"

namespace moe {
namespace {

template <typename T>
struct Io;
template <>
struct Io<__nv_bfloat16> {
  static __device__ __forceinline__ void load(const void* p, size_t i, float (&f)[8]) {
    const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __uint_as_float(w[j] << 16);
      f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(void* p, size_t i, const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Io<__half> {
  static __device__ __forceinline__ void load(const void* p, size_t i, float (&f)[8]) {
    const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 d = f16x2_to_f32x2(w[j]);
      f[2 * j] = d.x;
      f[2 * j + 1] = d.y;
    }
  }
  static __device__ __forceinline__ void store(void* p, size_t i, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
        make_uint4(f32x2_to_f16x2(f[0], f[1]), f32x2_to_f16x2(f[2], f[3]),
                   f32x2_to_f16x2(f[4], f[5]), f32x2_to_f16x2(f[6], f[7]));
  }
};
template <>
struct Io<float> {
  static __device__ __forceinline__ void load(const void* p, size_t i, float (&f)[8]) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = q[0], b = q[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  static __device__ __forceinline__ void store(void* p, size_t i, const float (&f)[8]) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(f[0], f[1], f[2], f[3]);
    q[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};

// WPR warps share a row, each thread holding NCH chunks of 8 values.  With two
// chunks, registers for three CTAs per SM (two: T = 3000, H = 7088, bf16: 33.8 us
// instead of 27.6, f32: 37.2 instead of 31.6).
template <typename T, int WPR, int NCH>
__global__ void __launch_bounds__(WPR * 32, NCH == 2 ? 3 : 1) k_norm_fp8(NormFp8Args a) {
  __shared__ float part[WPR];
  pdl_wait();
  pdl_trigger();
  const int row = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t base = size_t(row) * a.H;
  float v[NCH][8];
  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int i = (c * WPR * 32 + int(threadIdx.x)) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[c][j] = 0.f;
    if (i < a.H) {
      Io<T>::load(a.x, base + i, v[c]);
      if (a.residual) {
        float r[8];
        Io<T>::load(a.residual, base + i, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[c][j] += r[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(v[c][j], v[c][j], ss);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
  if constexpr (WPR > 1) {
    if (lane == 0) part[warp] = ss;
    __syncthreads();
    ss = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) ss += part[w];
  }
  const float inv = rsqrtf(ss / float(a.H) + a.eps);
  const int nb = fp8_blocks(a.H);
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int i = (c * WPR * 32 + int(threadIdx.x)) * 8;
    const bool in = i < a.H;
    float2 n[4];
    float amax = 0.f;
    if (in) {
      if (a.residual_out) Io<T>::store(a.residual_out, base + i, v[c]);
      float w[8];
      Io<float>::load(a.weight, i, w);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        n[j] = mul2(mul2(make_float2(v[c][2 * j], v[c][2 * j + 1]), make_float2(inv, inv)),
                    make_float2(w[2 * j], w[2 * j + 1]));
        amax = fmaxf(amax, fmaxf(fabsf(n[j].x), fabsf(n[j].y)));
      }
      if (a.y) {
        const float y[8] = {n[0].x, n[0].y, n[1].x, n[1].y, n[2].x, n[2].y, n[3].x, n[3].y};
        Io<T>::store(a.y, base + i, y);
      }
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
    if (in) {
      const float s = fp8_scale(amax);
      uint32_t q[2];
      fp8_codes(n, s, q);
      *reinterpret_cast<uint2*>(a.q + base + i) = make_uint2(q[0], q[1]);
      if ((lane & 15) == 0) a.s[size_t(row) * nb + i / kFp8Block] = s;
    }
  }
}

template <typename T, int WPR, int NCH>
cudaError_t go(const NormFp8Args& a, cudaStream_t st) {
  return launch_pdl(k_norm_fp8<T, WPR, NCH>, dim3(a.rows), dim3(WPR * 32), 0, st, a);
}

template <typename T>
cudaError_t pick(const NormFp8Args& a, cudaStream_t st) {
  // one chunk per thread as far as 16 warps reach (bf16, T = 4096, H = 4096: 27.2
  // us with 16 warps and 1 chunk, 28.0 with 8 and 2, 31.3 with 4 and 4; T = 1:
  // 2.3, 2.7, 3.8 us; f16, T = 777, H = 7088: 7.2 us with 16 and 2, 7.7 with 8
  // and 4, 8.6 with 32 and 1)
  if (a.H <= 256) return go<T, 1, 1>(a, st);
  if (a.H <= 1024) return go<T, 4, 1>(a, st);
  if (a.H <= 2048) return go<T, 8, 1>(a, st);
  if (a.H <= 4096) return go<T, 16, 1>(a, st);
  if (a.H <= 8192) return go<T, 16, 2>(a, st);
  return go<T, 16, 4>(a, st);
}

}  // namespace

cudaError_t launch_norm_fp8(const NormFp8Args& a, cudaStream_t st) {
  if (a.rows == 0) return cudaSuccess;
  switch (a.dtype) {
    case MOE_DTYPE_BF16: return pick<__nv_bfloat16>(a, st);
    case MOE_DTYPE_F16: return pick<__half>(a, st);
    default: return pick<float>(a, st);
  }
}

}  // namespace moe

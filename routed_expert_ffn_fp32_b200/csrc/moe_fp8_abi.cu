// C-ABI entry points of the E4M3 operators (include/moe.h): argument checks,
// workspace carving and launches.  Nothing here allocates or synchronises.
#include <cstdint>
#include <initializer_list>

#include "moe_fp8.cuh"

using namespace moe;

namespace {

constexpr int kMaxDim = 65536;            // N, K
constexpr int64_t kMaxRows = 1 << 21;     // rows of any operand

bool ok_ptr(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool ok_opt(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool ok_ptrs(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!ok_ptr(p)) return false;
  return true;
}
bool ok_dtype(int32_t t) { return t == MOE_DTYPE_BF16 || t == MOE_DTYPE_F16 || t == MOE_DTYPE_F32; }

moe_status_t status_of(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  cudaGetLastError();
  return MOE_ERR_CUDA;
}

bool ok_k(int32_t K) { return K >= 16 && K <= kMaxDim && K % 16 == 0; }

moe_status_t check_groups(int32_t a_rows, int32_t n_pairs, int32_t E, int32_t N, int32_t K) {
  if (a_rows < 1 || a_rows > kMaxRows || n_pairs < 0 || n_pairs > kMaxRows) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (E < 1 || E > kMaxExperts || N < 1 || N > kMaxDim || !ok_k(K)) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

struct Fp8Ws {
  size_t hq, hs, total;
};
// status words, then the SwiGLU rows (codes, scales) of all pairs
Fp8Ws fp8_ws(const moe_shape_t& s, int has_shared) {
  const size_t rows = size_t(s.T) * s.k + (has_shared ? s.T : 0);
  Fp8Ws w;
  w.hq = 256;
  w.hs = align256(w.hq + rows * s.I);
  w.total = align256(w.hs + rows * fp8_blocks(s.I) * 4);
  return w;
}

moe_status_t check_ffn8(const moe_shape_t& s) {
  if (s.T < 1 || s.T > 65536 || s.E < 1 || s.E > kMaxExperts || s.k < 1 || s.k > kMaxTopK)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  for (int32_t d : {s.H, s.I})
    if (d < 32 || d > 16384 || d % 32) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

bool ok_experts(const moe_fp8_experts_t* e, int n) {
  return e != nullptr && e->n_experts == n &&
         ok_ptrs({e->gate_q, e->gate_s, e->up_q, e->up_s, e->down_q, e->down_s});
}

}  // namespace

extern "C" {

moe_status_t moe_rmsnorm_quant_fp8(const void* x, const void* residual, const float* weight,
                                   int32_t rows, int32_t H, int32_t dtype, float eps,
                                   void* residual_out, void* y_out, uint8_t* q_out, float* s_out,
                                   void* stream) {
  if (rows < 0 || rows > kMaxRows || H < 16 || H > 16384 || H % 16) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!ok_dtype(dtype) || !(eps >= 0.f)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!ok_ptrs({x, weight, q_out, s_out}) || !ok_opt(residual) || !ok_opt(residual_out) || !ok_opt(y_out))
    return MOE_ERR_INVALID_ARG;
  NormFp8Args a{x, residual, weight, residual_out, y_out, q_out, s_out, rows, H, dtype, eps};
  return status_of(launch_norm_fp8(a, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_gemm_fp8(const uint8_t* a_q, const float* a_s, const uint8_t* w_q, const float* w_s,
                          int32_t rows, int32_t N, int32_t K, int32_t out_dtype, void* out, void* ws,
                          size_t ws_bytes, void* stream) {
  if (rows < 0) return MOE_ERR_UNSUPPORTED_SHAPE;
  const moe_status_t st = check_groups(rows > 0 ? rows : 1, rows, 1, N, K);
  if (st != MOE_OK) return st;
  if (!ok_dtype(out_dtype)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!ok_ptrs({a_q, a_s, w_q, w_s, out, ws})) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < MOE_FP8_STATUS_BYTES) return MOE_ERR_WORKSPACE;
  Fp8GemmArgs a{};
  a.a_q = a_q;
  a.a_s = a_s;
  a.w_q[0] = a.w_q[1] = w_q;
  a.w_s[0] = a.w_s[1] = w_s;
  a.out = out;
  a.err = static_cast<int*>(ws);
  a.a_rows = a.P = rows;
  a.E = 1;
  a.N = N;
  a.K = K;
  a.out_type = out_dtype;
  return status_of(launch_gemm_fp8(a, false, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_grouped_gemm_fp8(const uint8_t* a_q, const float* a_s, int32_t a_rows,
                                  const uint8_t* w_q, const float* w_s, const int32_t* offsets,
                                  const int32_t* entries, int32_t n_pairs, int32_t E, int32_t N,
                                  int32_t K, int32_t a_div, int32_t scatter, int32_t out_dtype,
                                  void* out, void* ws, size_t ws_bytes, void* stream) {
  const moe_status_t st = check_groups(n_pairs == 0 ? 1 : a_rows, n_pairs, E, N, K);
  if (st != MOE_OK) return st;
  if (!ok_dtype(out_dtype) || a_div < 0) return MOE_ERR_INVALID_ARG;
  if (n_pairs == 0) return MOE_OK;
  if (!ok_ptrs({a_q, a_s, w_q, w_s, offsets, out, ws}) || !ok_opt(entries)) return MOE_ERR_INVALID_ARG;
  if ((a_div > 0 || scatter) && entries == nullptr) return MOE_ERR_INVALID_ARG;
  if (a_div == 0 && a_rows < n_pairs) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < MOE_FP8_STATUS_BYTES) return MOE_ERR_WORKSPACE;
  Fp8GemmArgs a{};
  a.a_q = a_q;
  a.a_s = a_s;
  a.w_q[0] = a.w_q[1] = w_q;
  a.w_s[0] = a.w_s[1] = w_s;
  a.offsets = offsets;
  a.entries = entries;
  a.out = out;
  a.err = static_cast<int*>(ws);
  a.a_rows = a_rows;
  a.P = n_pairs;
  a.E = E;
  a.N = N;
  a.K = K;
  a.a_div = a_div;
  a.scatter = scatter != 0;
  a.out_type = out_dtype;
  return status_of(launch_gemm_fp8(a, false, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_grouped_swiglu_fp8(const uint8_t* a_q, const float* a_s, int32_t a_rows,
                                    const uint8_t* gate_q, const float* gate_s, const uint8_t* up_q,
                                    const float* up_s, const int32_t* offsets,
                                    const int32_t* entries, int32_t n_pairs, int32_t E, int32_t I,
                                    int32_t H, int32_t a_div, uint8_t* q_out, float* s_out, void* ws,
                                    size_t ws_bytes, void* stream) {
  const moe_status_t st = check_groups(n_pairs == 0 ? 1 : a_rows, n_pairs, E, I, H);
  if (st != MOE_OK) return st;
  if (!ok_k(I)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (a_div < 0) return MOE_ERR_INVALID_ARG;
  if (n_pairs == 0) return MOE_OK;
  if (!ok_ptrs({a_q, a_s, gate_q, gate_s, up_q, up_s, q_out, s_out, ws}) || !ok_opt(offsets) ||
      !ok_opt(entries))
    return MOE_ERR_INVALID_ARG;
  if ((a_div > 0 && entries == nullptr) || (offsets == nullptr && E != 1)) return MOE_ERR_INVALID_ARG;
  if (a_div == 0 && a_rows < n_pairs) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < MOE_FP8_STATUS_BYTES) return MOE_ERR_WORKSPACE;
  Fp8GemmArgs a{};
  a.a_q = a_q;
  a.a_s = a_s;
  a.w_q[0] = gate_q;
  a.w_q[1] = up_q;
  a.w_s[0] = gate_s;
  a.w_s[1] = up_s;
  a.offsets = offsets;
  a.entries = entries;
  a.q_out = q_out;
  a.s_out = s_out;
  a.err = static_cast<int*>(ws);
  a.a_rows = a_rows;
  a.P = n_pairs;
  a.E = E;
  a.N = I;
  a.K = H;
  a.a_div = a_div;
  return status_of(launch_gemm_fp8(a, true, static_cast<cudaStream_t>(stream)));
}

size_t moe_expert_ffn_fp8_workspace_bytes(moe_shape_t shape, int32_t has_shared) {
  if (check_ffn8(shape) != MOE_OK) return 0;
  return fp8_ws(shape, has_shared != 0).total;
}

moe_status_t moe_expert_ffn_fp8(const moe_fp8_experts_t* experts, const moe_fp8_experts_t* shared,
                                const uint8_t* x_q, const float* x_s, const int32_t* offsets,
                                const int32_t* entries, moe_shape_t shape, float* partial_out,
                                void* ws, size_t ws_bytes, void* stream) {
  moe_status_t st = check_ffn8(shape);
  if (st != MOE_OK) return st;
  if (!ok_experts(experts, shape.E) || (shared && !ok_experts(shared, 1))) return MOE_ERR_INVALID_ARG;
  if (!ok_ptrs({x_q, x_s, offsets, entries, partial_out, ws})) return MOE_ERR_INVALID_ARG;
  const Fp8Ws L = fp8_ws(shape, shared != nullptr);
  if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
  const int P = shape.T * shape.k;
  uint8_t* hq = static_cast<uint8_t*>(ws) + L.hq;
  float* hs = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + L.hs);
  st = moe_grouped_swiglu_fp8(x_q, x_s, shape.T, experts->gate_q, experts->gate_s, experts->up_q,
                              experts->up_s, offsets, entries, P, shape.E, shape.I, shape.H, shape.k,
                              hq, hs, ws, ws_bytes, stream);
  if (st == MOE_OK)
    st = moe_grouped_gemm_fp8(hq, hs, P, experts->down_q, experts->down_s, offsets, entries, P, shape.E,
                              shape.H, shape.I, 0, 1, MOE_DTYPE_F32, partial_out, ws, ws_bytes, stream);
  if (st != MOE_OK || shared == nullptr) return st;
  // the shared expert: one group of all T rows, after the routed pairs' rows
  Fp8GemmArgs a{};
  a.a_q = x_q;
  a.a_s = x_s;
  a.w_q[0] = shared->gate_q;
  a.w_q[1] = shared->up_q;
  a.w_s[0] = shared->gate_s;
  a.w_s[1] = shared->up_s;
  a.q_out = hq + size_t(P) * shape.I;
  a.s_out = hs + size_t(P) * fp8_blocks(shape.I);
  a.err = static_cast<int*>(ws);
  a.a_rows = a.P = shape.T;
  a.E = 1;
  a.N = shape.I;
  a.K = shape.H;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_gemm_fp8(a, true, s);
  if (e != cudaSuccess) return status_of(e);
  a.a_q = a.q_out;
  a.a_s = a.s_out;
  a.w_q[0] = a.w_q[1] = shared->down_q;
  a.w_s[0] = a.w_s[1] = shared->down_s;
  a.out = partial_out + size_t(P) * shape.H;
  a.N = shape.H;
  a.K = shape.I;
  a.out_type = MOE_DTYPE_F32;
  return status_of(launch_gemm_fp8(a, false, s));
}

}  // extern "C"

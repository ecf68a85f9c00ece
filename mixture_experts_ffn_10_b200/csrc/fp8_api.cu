// fp8_api.cu -- the entry points of moe_fp8.h: argument checks and launches.
#include <algorithm>
#include <climits>
#include <cstdarg>
#include <cstdio>

#include "fp8.cuh"
#include "moe_fp8.h"

namespace moe {
namespace {

int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return set_error(code, buf);
}

int cuda_status(cudaError_t e, const char* what) {
  return e == cudaSuccess ? MOE_OK : fail(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// dtype, and sizes whose block count fits a launch
int check_quantize(int dtype, int64_t rows, int64_t K) {
  if (dtype != MOE_F32 && dtype != MOE_BF16) return fail(MOE_ERR_DTYPE, "dtype %d must be MOE_F32 or MOE_BF16", dtype);
  if (rows < 0 || K < 1 || K > INT_MAX - 256)
    return fail(MOE_ERR_SHAPE, "need rows >= 0 and 1 <= K < 2^31 (got %lld, %lld)", (long long)rows, (long long)K);
  return MOE_OK;
}

int check_pointers(int dtype, const void* x, const uint8_t* q, const float* scales) {
  if (!x || !q || !scales) return fail(MOE_ERR_NULL, "the input, q and scales are required");
  if (!aligned(x, dtype == MOE_BF16 ? 2 : 4) || !aligned(scales, 4))
    return fail(MOE_ERR_ALIGN, "the input and scales must be aligned to their elements");
  return MOE_OK;
}

int check_matmul(int64_t rows, int64_t E, int64_t N, int64_t K) {
  if (rows < 0 || rows > (1ll << 30) || E < 1 || N < 1 || K < 1 || N > (1ll << 30) || K > (1ll << 30))
    return fail(MOE_ERR_SHAPE, "need 0 <= rows, 1 <= E, N, K, each at most 2^30 (got %lld, %lld, %lld, %lld)",
                (long long)rows, (long long)E, (long long)N, (long long)K);
  if (E > kMaxE) return fail(MOE_ERR_UNSUPPORTED, "E=%lld exceeds %d groups", (long long)E, kMaxE);
  if (K % kFp8MinNK || N % 8) return fail(MOE_ERR_SHAPE, "K must be a multiple of 16 and N of 8 (16-byte rows)");
  if (rows > 0 && fp8_m_tiles(rows, E) * fp8_n_tiles(FP8_LINEAR, N) > INT_MAX / 16)
    return fail(MOE_ERR_SHAPE, "rows x N is too large for one call");
  return MOE_OK;
}

size_t matmul_workspace(int64_t rows, int64_t E, int64_t N, int64_t K, int* splits) {
  *splits = rows > 0 ? fp8_splits(FP8_LINEAR, rows, E, N, K, device_sms()) : 1;
  if (rows == 0) return 0;
  // the status word, then the partial sums
  return 256 + (*splits == 1 ? 0 : (size_t)*splits * rows * fp8_n_tiles(FP8_LINEAR, N) * 256 * sizeof(float));
}

}  // namespace
}  // namespace moe

extern "C" {

int moe_fp8_quantize(int dtype, int64_t rows, int64_t K, const void* x, int64_t pitch, uint8_t* q, float* scales,
                     void* stream) {
  using namespace moe;
  int rc = check_quantize(dtype, rows, K);
  if (rc) return rc;
  if (pitch < K) return fail(MOE_ERR_SHAPE, "pitch %lld is less than K=%lld", (long long)pitch, (long long)K);
  if (rows == 0) return MOE_OK;
  if (rows > (int64_t)INT_MAX * 8 / cdiv(K, 128)) return fail(MOE_ERR_SHAPE, "rows x K is too large for one call");
  if ((rc = check_pointers(dtype, x, q, scales))) return rc;
  return cuda_status(launch_fp8_quantize(dtype == MOE_BF16, rows, K, x, pitch, q, scales, static_cast<cudaStream_t>(stream)),
                     "FP8 quantisation");
}

int moe_fp8_quantize_weights(int dtype, int64_t E, int64_t N, int64_t K, const void* w, uint8_t* q, float* scales,
                             void* stream) {
  using namespace moe;
  int rc = check_quantize(dtype, E, K);
  if (rc) return rc;
  if (N < 1 || N > INT_MAX - 256) return fail(MOE_ERR_SHAPE, "need 1 <= N < 2^31 (got %lld)", (long long)N);
  if (E == 0) return MOE_OK;
  if (E > INT_MAX / cdiv(N, 128) / cdiv(K, 128)) return fail(MOE_ERR_SHAPE, "E x N x K is too large for one call");
  if ((rc = check_pointers(dtype, w, q, scales))) return rc;
  return cuda_status(launch_fp8_quantize_weights(dtype == MOE_BF16, E, N, K, w, q, scales, static_cast<cudaStream_t>(stream)),
                     "FP8 weight quantisation");
}

size_t moe_fp8_matmul_workspace_size(int64_t rows, int64_t E, int64_t N, int64_t K) {
  int splits;
  if (moe::check_matmul(rows, E, N, K) != MOE_OK) return 0;
  return moe::matmul_workspace(rows, E, N, K, &splits);
}

int moe_fp8_matmul(int64_t rows, int64_t E, int64_t N, int64_t K, const uint8_t* xq, const float* xs, const uint8_t* wq,
                   const float* ws, const int32_t* counts, void* y, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace moe;
  const int rc = check_matmul(rows, E, N, K);
  if (rc) return rc;
  if (rows == 0) return MOE_OK;
  if (!xq || !xs || !wq || !ws || !y) return fail(MOE_ERR_NULL, "xq, xs, wq, ws and y are required");
  if (!counts && E != 1) return fail(MOE_ERR_NULL, "counts is required for more than one group");
  if (!aligned(xq, 16) || !aligned(wq, 16) || !aligned(y, 16))
    return fail(MOE_ERR_ALIGN, "xq, wq and y must be 16-byte aligned");
  if (!aligned(xs, 4) || !aligned(ws, 4) || (counts && !aligned(counts, 4)))
    return fail(MOE_ERR_ALIGN, "xs, ws and counts must be 4-byte aligned");
  int splits;
  const size_t need = matmul_workspace(rows, E, N, K, &splits);
  if (!workspace || workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace ? workspace_bytes : 0);
  if (!aligned(workspace, 256)) return fail(MOE_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  Fp8GemmArgs a{};
  a.mode = FP8_LINEAR;
  a.E = (int)E;
  a.R = (int)rows;
  a.K = (int)K;
  a.N = (int)N;
  a.cnt = counts;
  a.a = xq;
  a.as = xs;
  a.as_row = cdiv(K, 128);
  a.as_kb = 1;
  a.w = wq;
  a.ws = ws;
  a.y = static_cast<uint16_t*>(y);
  a.splits = splits;
  a.status = static_cast<int*>(workspace);
  a.clear_status = 1;
  a.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + 256);
  a.pitch = fp8_n_tiles(FP8_LINEAR, N) * 256;
  a.max_tiles = (int)(fp8_m_tiles(rows, E) * fp8_n_tiles(FP8_LINEAR, N));
  a.num_sms = device_sms();
  cudaError_t e = launch_fp8_gemm(a, st);
  if (e != cudaSuccess) return cuda_status(e, "FP8 grouped GEMM");
  if (splits > 1) return cuda_status(launch_fp8_reduce_y(a, st), "FP8 reduction");
  return MOE_OK;
}

}  // extern "C"

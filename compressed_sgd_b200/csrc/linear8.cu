// The product of rows in 8 bits and its gradients.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace gs {
namespace {

constexpr int kTile = 16;

__device__ __forceinline__ float read_as(const void* p, int32_t dtype, int64_t at) {
  if (dtype == GSPARSE_F32) return static_cast<const float*>(p)[at];
  if (dtype == GSPARSE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at]);
  return __half2float(static_cast<const __half*>(p)[at]);
}

__device__ __forceinline__ void write_as(void* p, int32_t dtype, int64_t at, float v) {
  if (dtype == GSPARSE_F32) static_cast<float*>(p)[at] = v;
  else if (dtype == GSPARSE_BF16) static_cast<__nv_bfloat16*>(p)[at] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p)[at] = __float2half_rn(v);
}

struct SimpleArgs {
  const int8_t* x;
  const float* x_scale;
  const int8_t* w;
  const float* w_scale;
  const void* dout;
  void* out;
  int64_t x_stride, w_stride, dout_stride, out_stride;
  int tokens, channels, depth, dtype, out_dtype;
};

// OP 0: out[t][n] over k; 1: dx[t][k] over n; 2: dweight[n][k] over t. A block of 16 x 16 results, a thread each.
template <int OP>
__global__ void __launch_bounds__(kTile * kTile) simple_kernel(const __grid_constant__ SimpleArgs a) {
  pdl_begin();
  __shared__ float A[kTile][kTile + 1], B[kTile][kTile + 1];
  const int rows = OP == 2 ? a.channels : a.tokens, cols = OP == 0 ? a.channels : a.depth;
  const int sums = OP == 0 ? a.depth : OP == 1 ? a.channels : a.tokens;
  const int tx = threadIdx.x % kTile, ty = threadIdx.x / kTile;
  for (int64_t r0 = (int64_t)blockIdx.y * kTile; r0 < rows; r0 += (int64_t)gridDim.y * kTile) {
    const int64_t row = r0 + ty, col = (int64_t)blockIdx.x * kTile + tx;
    int whole = 0;
    float sum = 0.0f;
    for (int64_t s0 = 0; s0 < sums; s0 += kTile) {
      const int64_t ra = r0 + ty, sa = s0 + tx;          // A[ty][tx]: row ra at sum place sa
      float v = 0.0f;
      if (ra < rows && sa < sums) {
        if (OP == 0) v = (float)a.x[ra * a.x_stride + sa];
        if (OP == 1) v = read_as(a.dout, a.dtype, ra * a.dout_stride + sa);
        if (OP == 2) v = read_as(a.dout, a.dtype, sa * a.dout_stride + ra);
      }
      A[ty][tx] = v;
      const int64_t cb = (int64_t)blockIdx.x * kTile + tx, sb = s0 + ty;   // B[ty][tx]: sum place sb at column cb
      v = 0.0f;
      if (cb < cols && sb < sums) {
        if (OP == 0) v = (float)a.w[cb * a.w_stride + sb];
        if (OP == 1) v = (float)a.w[sb * a.w_stride + cb] * a.w_scale[sb];
        if (OP == 2) v = (float)a.x[sb * a.x_stride + cb] * a.x_scale[sb];
      }
      B[ty][tx] = v;
      __syncthreads();
      for (int i = 0; i < kTile; ++i) {
        if (OP == 0) whole += (int)A[ty][i] * (int)B[i][tx];
        else sum = __fmaf_rn(A[ty][i], B[i][tx], sum);
      }
      __syncthreads();
    }
    if (row < rows && col < cols) {
      if (OP == 0) sum = ((float)whole * a.x_scale[row]) * a.w_scale[col];
      write_as(a.out, a.out_dtype, row * a.out_stride + col, sum);
    }
  }
}

bool known(int32_t t) { return t == GSPARSE_F32 || t == GSPARSE_BF16 || t == GSPARSE_F16; }
size_t size_of(int32_t t) { return t == GSPARSE_F32 ? 4 : 2; }
bool at_multiple(const void* p, size_t of) { return (reinterpret_cast<uintptr_t>(p) % of) == 0; }

int sizes(int64_t tokens, int64_t channels, int64_t depth) {
  if (tokens < 0 || channels < 1 || depth < 1) return GSPARSE_ERR_INVALID_ARG;
  if (tokens > GSPARSE_MAX_ROWS || channels > GSPARSE_MAX_ROWS || depth > GSPARSE_MAX_DEPTH) return GSPARSE_ERR_UNSUPPORTED;
  return GSPARSE_OK;
}

bool rows8(const int8_t* q, int64_t stride, const float* scale, int64_t depth) {
  return q && scale && aligned16(q) && stride % 16 == 0 && stride >= depth && at_multiple(scale, 4);
}

bool matrix(const void* p, int64_t stride, int32_t dtype, int64_t rows, int64_t cols, bool write) {
  return known(dtype) && p && at_multiple(p, size_of(dtype)) && stride >= (write && rows > 1 ? cols : 0);
}

bool space(const void* workspace, size_t have, size_t need) { return workspace && at_multiple(workspace, 256) && have >= need; }

template <int OP>
int simple(const SimpleArgs& a, cudaStream_t st) {
  const int rows = OP == 2 ? a.channels : a.tokens, cols = OP == 0 ? a.channels : a.depth;
  const int64_t gy = cdiv(rows, kTile);
  launch(simple_kernel<OP>, dim3((unsigned)cdiv(cols, kTile), (unsigned)(gy < 65535 ? gy : 65535)), dim3(kTile * kTile), 0, st, a);
  return launch_status();
}

}  // namespace
}  // namespace gs

using namespace gs;

extern "C" {

size_t gsparse_linear_q8_workspace_size(int64_t tokens, int64_t channels, int64_t depth) {
  return sizes(tokens, channels, depth) == GSPARSE_OK ? 256 : 0;
}

int gsparse_linear_q8(const int8_t* x, int64_t x_stride, const float* x_scale, const int8_t* w, int64_t w_stride, const float* w_scale,
                      int64_t tokens, int64_t channels, int64_t depth, void* out, int32_t dtype, int64_t out_stride, void* workspace,
                      size_t workspace_bytes, int32_t* d_status, gsparse_stream stream) {
  const int st = sizes(tokens, channels, depth);
  if (st != GSPARSE_OK) return st;
  if (!known(dtype)) return GSPARSE_ERR_INVALID_ARG;
  if (tokens == 0) return GSPARSE_OK;
  if (!rows8(x, x_stride, x_scale, depth) || !rows8(w, w_stride, w_scale, depth) || !matrix(out, out_stride, dtype, tokens, channels, true))
    return GSPARSE_ERR_INVALID_ARG;
  if (!space(workspace, workspace_bytes, gsparse_linear_q8_workspace_size(tokens, channels, depth))) return GSPARSE_ERR_WORKSPACE;
  return simple<0>({x, x_scale, w, w_scale, nullptr, out, x_stride, w_stride, 0, out_stride, (int)tokens, (int)channels, (int)depth, 0, dtype},
                   (cudaStream_t)stream);
}

size_t gsparse_linear_q8_grad_input_workspace_size(const void* dout, int32_t dtype, int64_t dout_stride, int64_t tokens,
                                                   int64_t channels, int64_t depth) {
  return known(dtype) && sizes(tokens, channels, depth) == GSPARSE_OK ? 256 : 0;
}

int gsparse_linear_q8_grad_input(const void* dout, int32_t dtype, int64_t dout_stride, const int8_t* w, int64_t w_stride,
                                 const float* w_scale, int64_t tokens, int64_t channels, int64_t depth, void* dx, int32_t dx_dtype,
                                 int64_t dx_stride, void* workspace, size_t workspace_bytes, int32_t* d_status, gsparse_stream stream) {
  const int st = sizes(tokens, channels, depth);
  if (st != GSPARSE_OK) return st;
  if (!known(dtype) || !known(dx_dtype)) return GSPARSE_ERR_INVALID_ARG;
  if (tokens == 0) return GSPARSE_OK;
  if (!matrix(dout, dout_stride, dtype, tokens, channels, false) || !rows8(w, w_stride, w_scale, depth) ||
      !matrix(dx, dx_stride, dx_dtype, tokens, depth, true))
    return GSPARSE_ERR_INVALID_ARG;
  if (!space(workspace, workspace_bytes, gsparse_linear_q8_grad_input_workspace_size(dout, dtype, dout_stride, tokens, channels, depth)))
    return GSPARSE_ERR_WORKSPACE;
  return simple<1>({nullptr, nullptr, w, w_scale, dout, dx, 0, w_stride, dout_stride, dx_stride, (int)tokens, (int)channels, (int)depth, dtype, dx_dtype},
                   (cudaStream_t)stream);
}

size_t gsparse_linear_q8_grad_weight_workspace_size(const void* dout, int32_t dtype, int64_t dout_stride, int64_t tokens,
                                                    int64_t channels, int64_t depth) {
  return known(dtype) && sizes(tokens, channels, depth) == GSPARSE_OK ? 256 : 0;
}

int gsparse_linear_q8_grad_weight(const void* dout, int32_t dtype, int64_t dout_stride, const int8_t* x, int64_t x_stride,
                                  const float* x_scale, int64_t tokens, int64_t channels, int64_t depth, float* dweight,
                                  int64_t dweight_stride, void* workspace, size_t workspace_bytes, int32_t* d_status,
                                  gsparse_stream stream) {
  const int st = sizes(tokens, channels, depth);
  if (st != GSPARSE_OK) return st;
  if (!known(dtype) || !matrix(dweight, dweight_stride, GSPARSE_F32, channels, depth, true)) return GSPARSE_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  if (tokens == 0) {
    if (cudaMemset2DAsync(dweight, (size_t)(channels > 1 ? dweight_stride : depth) * 4, 0, (size_t)depth * 4, (size_t)channels, s) != cudaSuccess) {
      cudaGetLastError();
      return GSPARSE_ERR_CUDA;
    }
    return GSPARSE_OK;
  }
  if (!matrix(dout, dout_stride, dtype, tokens, channels, false) || !rows8(x, x_stride, x_scale, depth)) return GSPARSE_ERR_INVALID_ARG;
  if (!space(workspace, workspace_bytes, gsparse_linear_q8_grad_weight_workspace_size(dout, dtype, dout_stride, tokens, channels, depth)))
    return GSPARSE_ERR_WORKSPACE;
  return simple<2>({x, x_scale, nullptr, nullptr, dout, dweight, x_stride, 0, dout_stride, dweight_stride, (int)tokens, (int)channels, (int)depth, dtype, GSPARSE_F32},
                   s);
}

}  // extern "C"

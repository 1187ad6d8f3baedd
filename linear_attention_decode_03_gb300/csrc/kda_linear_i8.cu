// kda_linear_i8.cu -- the layer's projections on 8-bit operands on GB300
// (sm_103a): y[m, n] = sx[m] sw[n] sum_k x[m, k] W[n, k], int8 in, bf16 out
// (see include/kda_ops.h, kda_linear_i8).
//
// A 64 x 64 output tile a CTA of 256 threads, 64 k a step through shared memory, four-way byte dot
// products into 32-bit integers.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_ops.h"

namespace {

constexpr int TILE = 64, KS = 64;

__device__ unsigned g_i8_err;

struct I8Args {
  const int8_t *x, *w;
  const float *sx, *sw;
  __nv_bfloat16* y;
  long long M, N, K, ldx, ldy;
};

__global__ void __launch_bounds__(256) i8_tile_kernel(const I8Args a) {
  __shared__ int xs[TILE][KS / 4 + 1], ws[TILE][KS / 4 + 1];
  const long long n0 = (long long)blockIdx.x * TILE, m0 = (long long)blockIdx.y * TILE;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int acc[4][4] = {};
  for (long long k0 = 0; k0 < a.K; k0 += KS) {
    const int r = threadIdx.x >> 2, c = threadIdx.x & 3;
    const bool in = k0 + 16 * c < a.K;
    int4 vx = make_int4(0, 0, 0, 0), vw = vx;
    if (in && m0 + r < a.M) vx = *reinterpret_cast<const int4*>(a.x + (m0 + r) * a.ldx + k0 + 16 * c);
    if (in && n0 + r < a.N) vw = *reinterpret_cast<const int4*>(a.w + (n0 + r) * a.K + k0 + 16 * c);
    __syncthreads();
    xs[r][4 * c] = vx.x, xs[r][4 * c + 1] = vx.y, xs[r][4 * c + 2] = vx.z, xs[r][4 * c + 3] = vx.w;
    ws[r][4 * c] = vw.x, ws[r][4 * c + 1] = vw.y, ws[r][4 * c + 2] = vw.z, ws[r][4 * c + 3] = vw.w;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < KS / 4; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(xs[ty + 16 * i][k], ws[tx + 16 * j][k], acc[i][j]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const long long m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m < a.M && n < a.N) a.y[m * a.ldy + n] = __float2bfloat16_rn((float)acc[i][j] * a.sx[m] * a.sw[n]);
    }
}

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

}  // namespace

extern "C" int kda_linear_i8(const void* x, long long rows, long long ldx, const float* x_scales, const void* w,
                             const float* w_scales, long long N, long long K, void* y, long long ldy,
                             void* cuda_stream) {
  if (rows < 0 || N < 1 || K < 16 || K % 16 != 0) return KDA_EINVAL;
  if (rows == 0) return KDA_OK;
  if (!x || !x_scales || !w || !w_scales || !y || ldx < K || ldx % 16 != 0 || ldy < N) return KDA_EINVAL;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(y, 2) || !aligned(x_scales, 4) || !aligned(w_scales, 4))
    return KDA_EINVAL;
  if (K > 131072 || N > 0x7fffffffLL || rows > 65535LL * TILE) return KDA_EINVAL;
  I8Args a;
  a.x = static_cast<const int8_t*>(x);
  a.w = static_cast<const int8_t*>(w);
  a.sx = x_scales, a.sw = w_scales;
  a.y = static_cast<__nv_bfloat16*>(y);
  a.M = rows, a.N = N, a.K = K, a.ldx = ldx, a.ldy = ldy;
  const dim3 grid((unsigned)((N + TILE - 1) / TILE), (unsigned)((rows + TILE - 1) / TILE));
  i8_tile_kernel<<<grid, 256, 0, static_cast<cudaStream_t>(cuda_stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ECUDA;
}

extern "C" int kda_linear_i8_check(void* cuda_stream, unsigned* device_flags) {
  if (!device_flags) return KDA_EINVAL;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(cuda_stream)) != cudaSuccess) return KDA_ECUDA;
  unsigned v = 0;
  const unsigned zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_i8_err, sizeof(v)) != cudaSuccess ||
      cudaMemcpyToSymbol(g_i8_err, &zero, sizeof(zero)) != cudaSuccess)
    return KDA_ECUDA;
  *device_flags = v;
  return KDA_OK;
}

// kda_quant.cu -- residual addition, RMSNorm and int8 rows with one scale each
// on GB300 (sm_103a); see include/kda_ops.h, kda_quant_rows.
//
// With p = h w and n = 1 / sqrt(mean h^2 + eps), the row n p quantised to
// 127 steps of its largest magnitude is q_i = round(127 n p_i / (n max|p|)): the
// norm's factor cancels, so q needs max|p| alone and n enters the scale only.
// h and w are bf16, so p is exact in fp32 (16 bits), and so are 254 |p_i| and
// (2 m + 1) max|p| for m < 128 (24 bits): where the fp32 quotient lies next to a half,
// m + 1/2, comparing these two decides the rounding exactly.  q therefore
// does not depend on the order of any sum.
//
// One CTA a row, the row in registers (V vectors of 8 values a thread), one
// block reduction for max|p| and sum h^2 together.  The bound is the row's bytes:
// each value of x and residual is read once, h and q written once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_ops.h"

namespace {

constexpr int QUANT_THREADS = 512;  // at most, a CTA
static_assert(KDA_QUANT_MAX_COLS == QUANT_THREADS * 8 * 8, "8 vectors of 8 a thread");

struct QuantArgs {
  const __nv_bfloat16* x;
  __nv_bfloat16* res;
  const __nv_bfloat16* w;
  int8_t* q;
  float* scales;
  long long ldx, ldr, ldq;
  int cols;
  float eps;
};

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// max (as bits of non-negative floats, NaN above infinity above all) and sum over the block
__device__ __forceinline__ void block_reduce(unsigned& top, float& sum, unsigned* s_top, float* s_sum) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  top = __reduce_max_sync(0xffffffffu, top);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) s_top[warp] = top, s_sum[warp] = sum;
  __syncthreads();
  top = __reduce_max_sync(0xffffffffu, lane < warps ? s_top[lane] : 0u);
  sum = lane < warps ? s_sum[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
}

// round(127 p / top), ties to even, exactly; inv = 127 / top rounded
__device__ __forceinline__ int quantise(float p, float inv, float top) {
  const float t = p * inv;  // within 2^-22 |t| of 127 p / top
  const float r = rintf(t);
  int q = (int)r;
  if (fabsf(t - r) > 0.4999f) {  // next to a half: compare 254 |p| with (2 m + 1) top, both exact
    const int m = (int)fabsf(t);
    const float lhs = 254.0f * fabsf(p), rhs = (float)(2 * m + 1) * top;
    const int up = lhs > rhs ? 1 : (lhs < rhs ? 0 : (m & 1));
    q = p < 0.0f ? -(m + up) : m + up;
  }
  return q;
}

template <int V, bool RES, bool NORM>
__global__ void __launch_bounds__(QUANT_THREADS) quant_rows_kernel(const QuantArgs a) {
  __shared__ unsigned s_top[2][32];
  __shared__ float s_sum[2][32];
  const long long row = blockIdx.x;
  const int vecs = a.cols >> 3;
  const uint4* x = reinterpret_cast<const uint4*>(a.x + row * a.ldx);
  uint4* res = RES ? reinterpret_cast<uint4*>(a.res + row * a.ldr) : nullptr;
  const uint4* w = reinterpret_cast<const uint4*>(a.w);
  uint4 hx[V], hr[V], hw[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    const bool in = c < vecs;
    hx[i] = in ? __ldcs(x + c) : make_uint4(0, 0, 0, 0);
    if (RES) hr[i] = in ? __ldcs(res + c) : make_uint4(0, 0, 0, 0);
    if (NORM) hw[i] = in ? w[c] : make_uint4(0, 0, 0, 0);
  }
  unsigned top_bits = 0;
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    uint32_t* u = reinterpret_cast<uint32_t*>(&hx[i]);
    const uint32_t* r = reinterpret_cast<const uint32_t*>(&hr[i]);
    const uint32_t* g = reinterpret_cast<const uint32_t*>(&hw[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (RES) {
        const __nv_bfloat162 h2 = __floats2bfloat162_rn(bf_lo(u[j]) + bf_lo(r[j]), bf_hi(u[j]) + bf_hi(r[j]));
        u[j] = *reinterpret_cast<const uint32_t*>(&h2);
      }
      const float h0 = bf_lo(u[j]), h1 = bf_hi(u[j]);
      if (NORM) sum = fmaf(h0, h0, fmaf(h1, h1, sum));
      top_bits = max(top_bits, __float_as_uint(fabsf(NORM ? h0 * bf_lo(g[j]) : h0)));
      top_bits = max(top_bits, __float_as_uint(fabsf(NORM ? h1 * bf_hi(g[j]) : h1)));
    }
    if (RES) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c < vecs) __stcs(res + c, hx[i]);
    }
  }
  block_reduce(top_bits, sum, s_top[0], s_sum[0]);
  float scale;      // of the row
  float up = 1.0f;  // p is computed with h and w times this
  // value j of vector i of p
  auto p_of = [&](int i, int j) {
    const uint32_t u = reinterpret_cast<const uint32_t*>(&hx[i])[j >> 1];
    const uint32_t g = reinterpret_cast<const uint32_t*>(&hw[i])[j >> 1];
    const float h = ((j & 1) ? bf_hi(u) : bf_lo(u)) * up;
    return NORM ? h * (((j & 1) ? bf_hi(g) : bf_lo(g)) * up) : h;
  };
  float inv, top = __uint_as_float(top_bits);
  if (top_bits >= 0x7f800000u) {  // a NaN or an infinity: the row says so
    scale = __uint_as_float(0x7fc00000u);
    inv = 0.0f;
  } else if (top_bits == 0) {
    scale = inv = 0.0f;
  } else {
    float n = 1.0f, unit = 1.0f;
    if (top < 0x1p-100f || (NORM && sum > 0x1p120f)) {
      // magnitudes whose products or squares leave fp32's range: once more with h (and w) times a power of two
      if (top < 0x1p-100f) up = 0x1p64f;
      const float down = NORM && sum > 0x1p120f ? 0x1p-80f : 1.0f;
      top_bits = 0, sum = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint32_t* u = reinterpret_cast<const uint32_t*>(&hx[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float h = ((j & 1) ? bf_hi(u[j >> 1]) : bf_lo(u[j >> 1])) * down;
          top_bits = max(top_bits, __float_as_uint(fabsf(p_of(i, j))));
          sum = fmaf(h, h, sum);
        }
      }
      block_reduce(top_bits, sum, s_top[1], s_sum[1]);
      top = __uint_as_float(top_bits);
      unit = 1.0f / up;
      if (NORM) n = down / sqrtf(sum / (float)a.cols + a.eps * down * down);
    } else if (NORM) {
      n = 1.0f / sqrtf(sum / (float)a.cols + a.eps);
    }
    scale = n * (top / 127.0f) * unit;
    if (NORM) scale *= unit;
    inv = 127.0f / top;
  }
  if (threadIdx.x == 0) a.scales[row] = scale;
  int8_t* q = a.q + row * a.ldq;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (c >= vecs) continue;
    uint32_t o[2] = {0u, 0u};
    if (inv != 0.0f) {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j >> 2] |= ((uint32_t)quantise(p_of(i, j), inv, top) & 0xffu) << (8 * (j & 3));
    }
    *reinterpret_cast<uint2*>(q + 8 * (long long)c) = make_uint2(o[0], o[1]);
  }
}

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

template <int V>
int quant_launch(const QuantArgs& a, long long rows, int threads, cudaStream_t st) {
  const unsigned grid = (unsigned)rows;
  if (a.res && a.w)
    quant_rows_kernel<V, true, true><<<grid, threads, 0, st>>>(a);
  else if (a.res)
    quant_rows_kernel<V, true, false><<<grid, threads, 0, st>>>(a);
  else if (a.w)
    quant_rows_kernel<V, false, true><<<grid, threads, 0, st>>>(a);
  else
    quant_rows_kernel<V, false, false><<<grid, threads, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ECUDA;
}

}  // namespace

extern "C" int kda_quant_rows(const void* x, long long rows, long long ldx, long long cols, void* residual,
                              long long ldr, const void* norm_weight, float eps, void* q, long long ldq,
                              float* scales, void* cuda_stream) {
  if (rows < 0 || rows > 0x7fffffffLL || cols < 16 || cols % 16 != 0 || cols > KDA_QUANT_MAX_COLS) return KDA_EINVAL;
  if (rows == 0) return KDA_OK;
  if (!x || !q || !scales || ldx < cols || ldx % 8 || ldq < cols || ldq % 8) return KDA_EINVAL;
  if (residual && (ldr < cols || ldr % 8)) return KDA_EINVAL;
  if (norm_weight && !(eps >= 0.0f)) return KDA_EINVAL;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(norm_weight, 16) || !aligned(q, 8) || !aligned(scales, 4))
    return KDA_EINVAL;
  QuantArgs a;
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.res = static_cast<__nv_bfloat16*>(residual);
  a.w = static_cast<const __nv_bfloat16*>(norm_weight);
  a.q = static_cast<int8_t*>(q);
  a.scales = scales;
  a.ldx = ldx, a.ldr = ldr, a.ldq = ldq;
  a.cols = (int)cols;
  a.eps = eps;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const int vecs = (int)(cols / 8);
  const int v = vecs <= QUANT_THREADS ? 1 : vecs <= 2 * QUANT_THREADS ? 2 : vecs <= 4 * QUANT_THREADS ? 4 : 8;
  const int threads = ((vecs + v - 1) / v + 31) / 32 * 32;
  if (v == 1) return quant_launch<1>(a, rows, threads, st);
  if (v == 2) return quant_launch<2>(a, rows, threads, st);
  if (v == 4) return quant_launch<4>(a, rows, threads, st);
  return quant_launch<8>(a, rows, threads, st);
}

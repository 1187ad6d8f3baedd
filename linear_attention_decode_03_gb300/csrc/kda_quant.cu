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
// A CTA takes rows in turn (as many CTAs as are resident), a row in registers (V vectors of 8
// values a thread, the same columns each time, so the weight stays there too), one block reduction a
// row for max|p| and sum h^2 together.  The bound is the rows' bytes, each read or written once; a row
// by itself would load, wait, reduce and store one after the other, so the next rows are on their
// way into shared memory meanwhile (asynchronous 16-byte copies; each thread reads back its own, so
// they need no barrier).  8191 x 7168 with norm and residual: 411 MB in 64 us, 0.94 of the measured copy
// bandwidth (a CTA a row, without the copies ahead: 87 us); 4 vectors a thread in 224 threads against 2 in 448: 64
// and 84 us; a ring of three rows and fewer registers for more CTAs were no faster.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_ops.h"

namespace {

// rows of a CTA in flight or in use (the longest rows leave shared memory for one)
__host__ __device__ constexpr int depth_of(int v) { return v == 8 ? 1 : 2; }

struct QuantArgs {
  const __nv_bfloat16* x;
  __nv_bfloat16* res;
  const __nv_bfloat16* w;
  int8_t* q;
  float* scales;
  long long rows, ldx, ldr, ldq;
  int cols;
  float eps;
};

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

constexpr int MAX_WARPS = 16;

// max (as bits of non-negative floats, NaN above infinity above all) and sum over the block; s_top and
// s_sum hold a value a warp, zeros behind the last
__device__ __forceinline__ void block_reduce(unsigned& top, float& sum, unsigned* s_top, float* s_sum) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  top = __reduce_max_sync(0xffffffffu, top);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) s_top[warp] = top, s_sum[warp] = sum;
  __syncthreads();
  top = 0, sum = 0.0f;
#pragma unroll
  for (int i = 0; i < MAX_WARPS; i += 4) {
    if (i >= warps) break;
    const uint4 m = *reinterpret_cast<const uint4*>(s_top + i);
    const float4 s = *reinterpret_cast<const float4*>(s_sum + i);
    top = max(max(top, m.x), max(m.y, max(m.z, m.w)));
    sum += (s.x + s.y) + (s.z + s.w);
  }
}

// round(127 p / top), ties to even, exactly, for t = p inv (inv = 127 / top rounded) next to a half: t is
// within 2^-22 |t| of the quotient, so the whole part is right, and 254 |p| and (2 m + 1) top decide.
__device__ __forceinline__ int round_exact(float p, float t, float top) {
  const int m = (int)fabsf(t);
  const float lhs = 254.0f * fabsf(p), rhs = (float)(2 * m + 1) * top;
  const int up = lhs > rhs ? 1 : (lhs < rhs ? 0 : (m & 1));
  return p < 0.0f ? -(m + up) : m + up;
}

// Eight values of p as bytes.  Adding 1.5 x 2^23 leaves the rounded integer in a float's low bits, two's
// complement, so neither the rounding nor the conversion takes the slow conversion unit; quotients within
// 5e-5 of a half (127 x 2^-22 = 3e-5) are decided again.
__device__ __forceinline__ uint2 quantise8(const float (&p)[8], float inv, float top) {
  constexpr float MAGIC = 12582912.0f;
  uint32_t u[8];
  float far = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float t = p[j] * inv, m = t + MAGIC;
    far = fmaxf(far, fabsf(t - (m - MAGIC)));
    u[j] = __float_as_uint(m);
  }
  if (far > 0.49995f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float t = p[j] * inv;
      if (fabsf(t - (__uint_as_float(u[j]) - MAGIC)) > 0.49995f) u[j] = (uint32_t)round_exact(p[j], t, top);
    }
  }
  const uint32_t a = __byte_perm(u[0], u[1], 0x0040), b = __byte_perm(u[2], u[3], 0x0040);
  const uint32_t c = __byte_perm(u[4], u[5], 0x0040), d = __byte_perm(u[6], u[7], 0x0040);
  return make_uint2(__byte_perm(a, b, 0x5410), __byte_perm(c, d, 0x5410));
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}

template <int V, bool RES, bool NORM, int MAXT>
__global__ void __launch_bounds__(MAXT) quant_rows_kernel(const QuantArgs a) {
  constexpr int DEPTH = depth_of(V);
  extern __shared__ __align__(16) unsigned char ring[];  // DEPTH rows of x and residual
  __shared__ __align__(16) unsigned s_top[3][MAX_WARPS];
  __shared__ __align__(16) float s_sum[3][MAX_WARPS];
  for (int i = threadIdx.x; i < 3 * MAX_WARPS; i += blockDim.x)
    s_top[i / MAX_WARPS][i % MAX_WARPS] = 0, s_sum[i / MAX_WARPS][i % MAX_WARPS] = 0.0f;
  __syncthreads();
  const int vecs = a.cols >> 3;
  const int row_bytes = a.cols * 2, slot_bytes = row_bytes * (RES ? 2 : 1);
  const uint32_t base = (uint32_t)__cvta_generic_to_shared(ring);
  // one copy group a row, empty behind the last
  auto fetch = [&](long long row, int slot) {
    if (row < a.rows) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c < vecs) {
          copy16(base + slot * slot_bytes + 16 * c, a.x + row * a.ldx + 8 * c);
          if (RES) copy16(base + slot * slot_bytes + row_bytes + 16 * c, a.res + row * a.ldr + 8 * c);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int d = 0; d < DEPTH - 1; ++d) fetch(blockIdx.x + (long long)d * gridDim.x, d);
  uint4 hw[V];
  // NaN if this thread's weights are not all finite: added to the sum, it sends every row the careful way
  float w_bad = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    hw[i] = NORM && c < vecs ? reinterpret_cast<const uint4*>(a.w)[c] : make_uint4(0, 0, 0, 0);
    const uint32_t g[4] = {hw[i].x, hw[i].y, hw[i].z, hw[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if ((g[j] & 0x7f80u) == 0x7f80u || (g[j] & 0x7f800000u) == 0x7f800000u) w_bad = __uint_as_float(0x7fc00000u);
  }
  int slot = 0, turn = 0;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    fetch(row + (long long)(DEPTH - 1) * gridDim.x, slot == 0 ? DEPTH - 1 : slot - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
    const uint32_t at = base + slot * slot_bytes;
    slot = slot + 1 == DEPTH ? 0 : slot + 1;
    // vector i of h
    auto load_h = [&](int i, float (&h)[8], bool store) {
      const int c = threadIdx.x + i * blockDim.x;
      uint4 h4 = make_uint4(0, 0, 0, 0);
      if (c < vecs) {
        h4 = lds16(at + 16 * c);
        if (RES) {
          const uint4 r4 = lds16(at + row_bytes + 16 * c);
          auto sum2 = [](uint32_t u, uint32_t r) {
            const __nv_bfloat162 h2 = __floats2bfloat162_rn(bf_lo(u) + bf_lo(r), bf_hi(u) + bf_hi(r));
            return *reinterpret_cast<const uint32_t*>(&h2);
          };
          h4 = make_uint4(sum2(h4.x, r4.x), sum2(h4.y, r4.y), sum2(h4.z, r4.z), sum2(h4.w, r4.w));
          if (store) __stcs(reinterpret_cast<uint4*>(a.res + row * a.ldr) + c, h4);
        }
      }
      h[0] = bf_lo(h4.x), h[1] = bf_hi(h4.x), h[2] = bf_lo(h4.y), h[3] = bf_hi(h4.y);
      h[4] = bf_lo(h4.z), h[5] = bf_hi(h4.z), h[6] = bf_lo(h4.w), h[7] = bf_hi(h4.w);
    };
    auto load_w = [&](int i, float (&w)[8]) {
      w[0] = bf_lo(hw[i].x), w[1] = bf_hi(hw[i].x), w[2] = bf_lo(hw[i].y), w[3] = bf_hi(hw[i].y);
      w[4] = bf_lo(hw[i].z), w[5] = bf_hi(hw[i].z), w[6] = bf_lo(hw[i].w), w[7] = bf_hi(hw[i].w);
    };
    float p[V][8];
    float top = 0.0f, sum = NORM ? w_bad : 0.0f;
    unsigned top_bits = 0;  // without a norm: the largest magnitude's bits, where a NaN is above all
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float h[8], w[8];
      load_h(i, h, true);
      load_w(i, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        p[i][j] = NORM ? h[j] * w[j] : h[j];
        if (NORM) {
          sum = fmaf(h[j], h[j], sum);
          top = fmaxf(top, fabsf(p[i][j]));  // (drops a NaN; one in h shows in the sum)
        } else {
          top_bits = max(top_bits, __float_as_uint(fabsf(p[i][j])));
        }
      }
    }
    if (NORM) top_bits = __float_as_uint(top);
    // (by turns: a warp may be at the next row's before another has read this one's)
    block_reduce(top_bits, sum, s_top[turn], s_sum[turn]);
    top = __uint_as_float(top_bits);
    float scale, inv;
    if (top >= 0x1p-100f && top < 0x1p119f && (!NORM || (sum <= 0x1p120f && (sum >= 0x1p-80f || a.eps >= 0x1p-60f)))) {
      scale = (NORM ? 1.0f / sqrtf(sum / (float)a.cols + a.eps) : 1.0f) * (top / 127.0f);
      inv = 127.0f / top;
    } else {
      // The careful way, for rows of zeros, with values that are not finite, or whose products or squares leave
      // fp32's range: once more with h (and w) times a power of two for p, and h times another for the sum.  Whatever that
      // pushes out of range is too small to count.
      const float up = top < 0x1p-100f ? 0x1p90f : top >= 0x1p119f ? 0x1p-72f : 1.0f;
      const float down = !NORM ? 1.0f : sum > 0x1p120f ? 0x1p-80f : sum < 0x1p-80f && a.eps < 0x1p-60f ? 0x1p90f : 1.0f;
      top_bits = 0, sum = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float h[8], w[8];
        load_h(i, h, false);
        load_w(i, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          // (a zero times anything finite stays one, whatever the other's size)
          p[i][j] = !NORM ? h[j] * up : h[j] == 0.0f || w[j] == 0.0f ? h[j] * w[j] : (h[j] * up) * (w[j] * up);
          top_bits = max(top_bits, __float_as_uint(fabsf(p[i][j])));
          sum = fmaf(h[j] * down, h[j] * down, sum);
        }
      }
      block_reduce(top_bits, sum, s_top[2], s_sum[2]);
      top = __uint_as_float(top_bits);
      inv = 0.0f;
      if (top_bits >= 0x7f800000u) {  // a NaN or an infinity: the row says so
        scale = __uint_as_float(0x7fc00000u);
      } else if (top_bits == 0) {
        scale = 0.0f;
      } else {
        const float unit = 1.0f / up;
        scale = (top / 127.0f) * unit;
        if (NORM) scale = (top / 127.0f) / sqrtf(sum / (float)a.cols + a.eps * down * down) * (down * unit) * unit;
        inv = 127.0f / top;
      }
    }
    if (threadIdx.x == 0) a.scales[row] = scale;
    int8_t* q = a.q + row * a.ldq;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c < vecs)
        *reinterpret_cast<uint2*>(q + 8 * (long long)c) = inv != 0.0f ? quantise8(p[i], inv, top) : make_uint2(0, 0);
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

template <int V, bool RES, bool NORM, int MAXT>
int quant_run(const QuantArgs& a, int threads, cudaStream_t st) {
  auto kernel = quant_rows_kernel<V, RES, NORM, MAXT>;
  const int smem = depth_of(V) * a.cols * 2 * (RES ? 2 : 1);
  int dev = 0, sms = 0, per_sm = 1;
  if (smem > 46 * 1024 &&  // (48 KB with the static part)
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return KDA_ECUDA;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return KDA_ECUDA;
  if (a.rows > sms &&
      (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem) != cudaSuccess || per_sm < 1))
    return KDA_ECUDA;
  const long long resident = (long long)sms * per_sm;
  kernel<<<(unsigned)(a.rows < resident ? a.rows : resident), threads, smem, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ECUDA;
}

template <int V, int MAXT>
int quant_launch(const QuantArgs& a, int threads, cudaStream_t st) {
  if (a.res && a.w) return quant_run<V, true, true, MAXT>(a, threads, st);
  if (a.res) return quant_run<V, true, false, MAXT>(a, threads, st);
  if (a.w) return quant_run<V, false, true, MAXT>(a, threads, st);
  return quant_run<V, false, false, MAXT>(a, threads, st);
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
  a.rows = rows, a.ldx = ldx, a.ldr = ldr, a.ldq = ldq;
  a.cols = (int)cols;
  a.eps = eps;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  // vectors of 8 a thread: as few as make a CTA of at most 512 threads
  const int vecs = (int)(cols / 8);
  const int v = vecs <= 256 ? 1 : vecs <= 512 ? 2 : vecs <= 2048 ? 4 : 8;
  static_assert(KDA_QUANT_MAX_COLS == 512 * 8 * 8, "8 vectors a thread at most");
  const int threads = ((vecs + v - 1) / v + 31) / 32 * 32;
  if (v == 1) return quant_launch<1, 512>(a, threads, st);
  if (v == 2) return quant_launch<2, 512>(a, threads, st);
  if (v == 4) return quant_launch<4, 512>(a, threads, st);
  return quant_launch<8, 512>(a, threads, st);
}

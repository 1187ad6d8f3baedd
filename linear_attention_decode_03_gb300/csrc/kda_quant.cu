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
// and 84 us; a ring of three rows 73 us.  With fewer bytes a value the instructions count too: products, squares and
// roundings two at a time (f32x2), and without a norm the row stays packed and its maximum is
// taken on bf16 bit patterns (51 registers instead of 59: three CTAs an SM), 1024 x 12288 12.9 -> 11.5 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_ops.h"
#include "tc.cuh"

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

// Two floats in a register pair, for the instructions that work on two at a time.
using F2 = unsigned long long;
__device__ __forceinline__ F2 pack2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpack2(F2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ F2 bf2(uint32_t u) { return pack2(bf_lo(u), bf_hi(u)); }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// the largest magnitude (drops NaNs)
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float r;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

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
// 5e-5 of a half (127 x 2^-24 = 8e-6) are decided again.
__device__ __forceinline__ uint2 quantise8(const F2 (&p)[4], float inv, float top) {
  constexpr float MAGIC = 12582912.0f;
  const F2 inv2 = pack2(inv, inv), magic2 = pack2(MAGIC, MAGIC), minus2 = pack2(-1.0f, -1.0f);
  uint32_t u[8];
  float far = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const F2 m = fma2(p[j], inv2, magic2);
    const float2 off = unpack2(fma2(p[j], inv2, fma2(m, minus2, magic2)));
    far = max_abs(far, off.x, off.y);
    const float2 r = unpack2(m);
    u[2 * j] = __float_as_uint(r.x), u[2 * j + 1] = __float_as_uint(r.y);
  }
  if (far > 0.49995f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 two = unpack2(p[j >> 1]);
      const float x = (j & 1) ? two.y : two.x, t = x * inv;
      if (fabsf(t - (__uint_as_float(u[j]) - MAGIC)) > 0.49994f) u[j] = (uint32_t)round_exact(x, t, top);
    }
  }
  const uint32_t a = __byte_perm(u[0], u[1], 0x0040), b = __byte_perm(u[2], u[3], 0x0040);
  const uint32_t c = __byte_perm(u[4], u[5], 0x0040), d = __byte_perm(u[6], u[7], 0x0040);
  return make_uint2(__byte_perm(a, b, 0x5410), __byte_perm(c, d, 0x5410));
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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
  after_previous();
  const int vecs = a.cols >> 3;
  const int row_bytes = a.cols * 2, slot_bytes = row_bytes * (RES ? 2 : 1);
  const uint32_t base = smem_addr(ring);
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
    auto load_h = [&](int i, bool store) {
      const int c = threadIdx.x + i * blockDim.x;
      uint4 h4 = make_uint4(0, 0, 0, 0);
      if (c < vecs) {
        h4 = lds128(at + 16 * c);
        if (RES) {
          const uint4 r4 = lds128(at + row_bytes + 16 * c);
          auto sum2 = [](uint32_t u, uint32_t r) { return pack_bf(bf_lo(u) + bf_lo(r), bf_hi(u) + bf_hi(r)); };
          h4 = make_uint4(sum2(h4.x, r4.x), sum2(h4.y, r4.y), sum2(h4.z, r4.z), sum2(h4.w, r4.w));
          if (store) __stcs(reinterpret_cast<uint4*>(a.res + row * a.ldr) + c, h4);
        }
      }
      return h4;
    };
    // p: with a norm as fp32 pairs, else h's bf16 pairs themselves
    F2 p[V][4];
    uint4 kept[V];
    float top = 0.0f, sum = NORM ? w_bad : 0.0f;
    unsigned top_bits = 0;  // the largest magnitude's bits (without a norm a NaN is above all)
    if (NORM) {
      F2 sum2 = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint4 h4 = load_h(i, true);
        const uint32_t h[4] = {h4.x, h4.y, h4.z, h4.w}, w[4] = {hw[i].x, hw[i].y, hw[i].z, hw[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const F2 h2 = bf2(h[j]);
          p[i][j] = mul2(h2, bf2(w[j]));
          sum2 = fma2(h2, h2, sum2);
          const float2 two = unpack2(p[i][j]);
          top = max_abs(top, two.x, two.y);  // (drops a NaN; one in h shows in the sum)
        }
      }
      const float2 two = unpack2(sum2);
      sum += two.x + two.y;
      top_bits = __float_as_uint(top);
    } else {
      uint32_t top2 = 0;  // bits of bf16 magnitudes, the same order
#pragma unroll
      for (int i = 0; i < V; ++i) {
        kept[i] = load_h(i, true);
        constexpr uint32_t ABS = 0x7fff7fffu;
        top2 = __vimax3_u16x2(top2, kept[i].x & ABS, kept[i].y & ABS);
        top2 = __vimax3_u16x2(top2, kept[i].z & ABS, kept[i].w & ABS);
      }
      top_bits = max(top2 << 16, top2 & 0xffff0000u);
    }
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
        const uint4 h4 = load_h(i, false);
        const uint32_t h[4] = {h4.x, h4.y, h4.z, h4.w}, w[4] = {hw[i].x, hw[i].y, hw[i].z, hw[i].w};
        uint32_t k[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float hx = bf_lo(h[j]), hy = bf_hi(h[j]), wx = bf_lo(w[j]), wy = bf_hi(w[j]);
          // (a zero times anything finite stays one, whatever the other's size)
          auto scaled = [&](float u, float v) { return u == 0.0f || v == 0.0f ? u * v : (u * up) * (v * up); };
          const float x = NORM ? scaled(hx, wx) : hx * up, y = NORM ? scaled(hy, wy) : hy * up;
          p[i][j] = pack2(x, y);
          k[j] = pack_bf(x, y);  // (exact where it counts, as h is)
          top_bits = max(top_bits, max(__float_as_uint(fabsf(x)), __float_as_uint(fabsf(y))));
          sum = fmaf(hx * down, hx * down, fmaf(hy * down, hy * down, sum));
        }
        kept[i] = make_uint4(k[0], k[1], k[2], k[3]);
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
      if (c < vecs) {
        if (!NORM) p[i][0] = bf2(kept[i].x), p[i][1] = bf2(kept[i].y), p[i][2] = bf2(kept[i].z), p[i][3] = bf2(kept[i].w);
        *reinterpret_cast<uint2*>(q + 8 * (long long)c) = inv != 0.0f ? quantise8(p[i], inv, top) : make_uint2(0, 0);
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int V, bool RES, bool NORM, int MAXT>
int quant_run(const QuantArgs& a, int threads, cudaStream_t st) {
  auto kernel = quant_rows_kernel<V, RES, NORM, MAXT>;
  const int smem = depth_of(V) * a.cols * 2 * (RES ? 2 : 1);
  int dev = 0, per_sm = 1;
  if (smem > 46 * 1024 &&  // (48 KB with the static part)
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return KDA_ECUDA;
  if (cudaGetDevice(&dev) != cudaSuccess) return KDA_ECUDA;
  const int sms = sm_count(dev);
  if (sms <= 0) return KDA_ECUDA;
  if (a.rows > sms &&
      (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem) != cudaSuccess || per_sm < 1))
    return KDA_ECUDA;
  const long long resident = (long long)sms * per_sm;
  return launch(kernel, a.rows < resident ? a.rows : resident, threads, smem, 1, st, a);
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
  if (!ptr_aligned(x, 16) || !ptr_aligned(residual, 16) || !ptr_aligned(norm_weight, 16) || !ptr_aligned(q, 8) || !ptr_aligned(scales, 4))
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

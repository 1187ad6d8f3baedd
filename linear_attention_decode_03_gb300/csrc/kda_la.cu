// kda_la.cu -- linear attention with a decay a head on GB300 (sm_103a): the
// single-token step and the prompt form (see include/kda_ops.h).
//
//   S_t = e^{g_t} S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t,   S [128 (v), 128 (k)]
//
// Step.  Every v row of S is independent of the others (o[v] = S[v, :] . q), so the
// unit of work is 16 v rows of one (row, head), held by one warp in registers:
// 64 state values a lane, 8 KiB a warp, all loads in flight before the first
// use.  The dot products of the 16 rows are summed over the lanes together by
// halving the rows a lane carries at each exchange (16 shuffles for 16 rows
// instead of 5 a row).  A CTA is four warps, 64 v rows.  The bound is the state's
// bytes, read and written once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_ops.h"

namespace {

constexpr int D = 128;          // head size (k and v)
constexpr int STEP_WARPS = 4;   // a CTA of the step: 4 warps x 16 v rows
constexpr int STEP_ROWS = 16 * STEP_WARPS;
constexpr int STEP_SPLIT = D / STEP_ROWS;  // CTAs a (row, head)

// Device error bits of la_step and la_prefill, read and cleared by kda_la_check.
__device__ unsigned g_la_err;

struct LaArgs {
  const __nv_bfloat16 *q, *k, *v;
  const float* g;
  __nv_bfloat16* out;
  void* state;
  const int *slots, *cu, *has_state;
  long long ldq, ldk, ldv, ldg, ldo;
  long long rows, seqs, max_len, pool;
  int heads, share;  // share: value heads a query / key head
  float scale;
};

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// A warp's 16 v rows of a state: KL k values a lane, RL rows a lane.  fp32: lane l has
// k = 4 l .. + 3 of every row (a row is one 512-byte access of the warp); bf16: the
// half-warps take 8 rows each, 8 k a lane (16-byte accesses either way).
template <bool BF>
struct Slice {
  static constexpr int KL = BF ? 8 : 4, RL = BF ? 8 : 16;
  float s[RL][KL];

  __device__ static int k0(int lane) { return BF ? (lane & 15) * 8 : lane * 4; }
  __device__ static int row(int lane, int i) { return BF ? (lane >> 4) * 8 + i : i; }
  // p: the slice's first element in the pool
  __device__ __forceinline__ void load(const void* p, int lane) {
#pragma unroll
    for (int i = 0; i < RL; ++i) {
      const long long at = row(lane, i) * D + k0(lane);
      if (BF) {
        const uint4 u = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + at));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][(2 * j) % KL] = bf_lo(w[j]), s[i][(2 * j + 1) % KL] = bf_hi(w[j]);
      } else {
        const float4 u = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(p) + at));
        s[i][0] = u.x, s[i][1] = u.y, s[i][2] = u.z, s[i][3] = u.w;
      }
    }
  }
  __device__ __forceinline__ void store(void* p, int lane) const {
#pragma unroll
    for (int i = 0; i < RL; ++i) {
      const long long at = row(lane, i) * D + k0(lane);
      if (BF)
        __stcs(reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + at),
               make_uint4(pack_bf(s[i][0], s[i][1]), pack_bf(s[i][2], s[i][3]), pack_bf(s[i][4 % KL], s[i][5 % KL]),
                          pack_bf(s[i][6 % KL], s[i][7 % KL])));
      else
        __stcs(reinterpret_cast<float4*>(static_cast<float*>(p) + at),
               make_float4(s[i][0], s[i][1], s[i][2], s[i][3]));
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < RL; ++i)
#pragma unroll
      for (int j = 0; j < KL; ++j) s[i][j] = 0.0f;
  }
  // KL bf16 of a row of q or k
  __device__ static void load_k(float (&x)[KL], const __nv_bfloat16* p, int lane) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(p + k0(lane));
    uint32_t u[KL / 2];
    if (BF) {
      const uint4 t = *reinterpret_cast<const uint4*>(w);
      u[0] = t.x, u[1] = t.y, u[2 % (KL / 2)] = t.z, u[3 % (KL / 2)] = t.w;
    } else {
      const uint2 t = *reinterpret_cast<const uint2*>(w);
      u[0] = t.x, u[1] = t.y;
    }
#pragma unroll
    for (int j = 0; j < KL / 2; ++j) x[2 * j] = bf_lo(u[j]), x[2 * j + 1] = bf_hi(u[j]);
  }
  // S <- d S + v k^T; returns S q of v row lane / 2 (the same on both lanes of a pair).
  // v: the slice's 16 values as 8 packed pairs
  __device__ __forceinline__ float update(float d, const uint32_t (&v)[8], const float (&k)[KL],
                                          const float (&q)[KL], int lane) {
    float acc[RL];
#pragma unroll
    for (int i = 0; i < RL; ++i) {
      // the value of row row(lane, i): RL = 8 rows start at pair 0 or 4
      const uint32_t u = BF ? (lane < 16 ? v[i >> 1] : v[(4 + (i >> 1)) & 7]) : v[i >> 1];
      const float vi = (i & 1) ? bf_hi(u) : bf_lo(u);
      float t = 0.0f;
#pragma unroll
      for (int j = 0; j < KL; ++j) {
        s[i][j] = fmaf(vi, k[j], d * s[i][j]);
        t = fmaf(s[i][j], q[j], t);
      }
      acc[i] = t;
    }
    // each exchange halves the rows: after it a lane holds those whose next index bit is its own
#pragma unroll
    for (int n = RL / 2, bit = BF ? 8 : 16; n >= 1; n >>= 1, bit >>= 1) {
      const bool up = lane & bit;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float keep = up ? acc[i + n] : acc[i], send = up ? acc[i] : acc[i + n];
        acc[i] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
      }
    }
    return acc[0] + __shfl_xor_sync(0xffffffffu, acc[0], 1);
  }
};

__device__ __forceinline__ void load_v16(uint32_t (&v)[8], const __nv_bfloat16* p) {
  const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

__device__ __forceinline__ void* state_at(const LaArgs& a, bool bf, int slot, int h, int v0) {
  const long long e = ((long long)slot * a.heads + h) * (D * D) + v0 * D;
  return static_cast<unsigned char*>(a.state) + e * (bf ? 2 : 4);
}

template <bool BF>
__global__ void __launch_bounds__(32 * STEP_WARPS) la_step_kernel(const LaArgs a) {
  const int lane = threadIdx.x & 31;
  const long long task = blockIdx.x / STEP_SPLIT;
  const int v0 = (blockIdx.x % STEP_SPLIT) * STEP_ROWS + (threadIdx.x >> 5) * 16;
  const long long b = task / a.heads;
  const int h = (int)(task % a.heads), hk = h / a.share;
  const int slot = a.slots[b];
  __nv_bfloat16* o = a.out + b * a.ldo + h * D + v0 + (lane >> 1);
  if (slot < 0 || slot >= a.pool) {
    if (slot == -1) {
      if (!(lane & 1)) *o = __float2bfloat16_rn(0.0f);
    } else if (threadIdx.x == 0) {
      atomicOr(&g_la_err, KDA_ERR_SLOT);
    }
    return;
  }
  void* st = state_at(a, BF, slot, h, v0);
  Slice<BF> S;
  S.load(st, lane);
  float q[Slice<BF>::KL], k[Slice<BF>::KL];
  uint32_t v[8];
  Slice<BF>::load_k(q, a.q + b * a.ldq + hk * D, lane);
  Slice<BF>::load_k(k, a.k + b * a.ldk + hk * D, lane);
  load_v16(v, a.v + b * a.ldv + h * D + v0);
  const float d = expf(a.g[b * a.ldg + h]);
  const float t = S.update(d, v, k, q, lane);
  S.store(st, lane);
  if (!(lane & 1)) *o = __float2bfloat16_rn(a.scale * t);
}

// The prompt form token by token: a warp keeps its 16 v rows over the sequence.
template <bool BF>
__global__ void __launch_bounds__(32 * STEP_WARPS) la_scan_kernel(const LaArgs a) {
  const int lane = threadIdx.x & 31;
  const long long task = blockIdx.x / STEP_SPLIT;
  const int v0 = (blockIdx.x % STEP_SPLIT) * STEP_ROWS + (threadIdx.x >> 5) * 16;
  const long long i = task / a.heads;
  const int h = (int)(task % a.heads), hk = h / a.share;
  const long long begin = a.cu[i], end = a.cu[i + 1];
  if (begin < 0 || end < begin || end > a.rows || end - begin > a.max_len) {
    if (threadIdx.x == 0) atomicOr(&g_la_err, KDA_ERR_SEQ);
    return;
  }
  const int slot = a.slots[i];
  const bool pad = slot == -1;
  if (!pad && (slot < 0 || slot >= a.pool)) {
    if (threadIdx.x == 0) atomicOr(&g_la_err, KDA_ERR_SLOT);
    return;
  }
  __nv_bfloat16* o = a.out + h * D + v0 + (lane >> 1);
  if (pad) {
    for (long long t = begin; t < end; ++t)
      if (!(lane & 1)) o[t * a.ldo] = __float2bfloat16_rn(0.0f);
    return;
  }
  void* st = state_at(a, BF, slot, h, v0);
  Slice<BF> S;
  if (a.has_state && a.has_state[i])
    S.load(st, lane);
  else
    S.zero();
  for (long long t = begin; t < end; ++t) {
    float q[Slice<BF>::KL], k[Slice<BF>::KL];
    uint32_t v[8];
    Slice<BF>::load_k(q, a.q + t * a.ldq + hk * D, lane);
    Slice<BF>::load_k(k, a.k + t * a.ldk + hk * D, lane);
    load_v16(v, a.v + t * a.ldv + h * D + v0);
    const float d = expf(a.g[t * a.ldg + h]);
    const float r = S.update(d, v, k, q, lane);
    if (!(lane & 1)) o[t * a.ldo] = __float2bfloat16_rn(a.scale * r);
  }
  S.store(st, lane);
}

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

// The checks that step and prefill share.  Without rows (a prompt call of empty
// sequences) there is nothing behind the rows' pointers.
bool la_args_ok(long long rows, const void* q, long long ldq, const void* k, long long ldk, const void* v,
                long long ldv, int heads, int qk_heads, const float* g, long long ldg, const void* state, int dtype,
                long long pool, const int* slots, const void* out, long long ldo) {
  if (heads < 1 || heads > 65535 || qk_heads < 1 || heads % qk_heads != 0) return false;
  if (dtype != KDA_STATE_F32 && dtype != KDA_STATE_BF16) return false;
  if (rows > 0 && (!q || !k || !v || !g || !out)) return false;
  if (!state || !slots || pool < 1 || pool > 0x7fffffffLL) return false;
  const long long nq = (long long)qk_heads * D, nv = (long long)heads * D;
  if (ldq < nq || ldk < nq || ldv < nv || ldo < nv || ldq % 8 || ldk % 8 || ldv % 8 || ldo % 8) return false;
  if (ldg != 0 && ldg < heads) return false;
  return aligned(q, 16) && aligned(k, 16) && aligned(v, 16) && aligned(out, 16) && aligned(state, 16) &&
         aligned(g, 4) && aligned(slots, 4);
}

LaArgs la_args(const void* q, long long ldq, const void* k, long long ldk, const void* v, long long ldv,
               long long rows, int heads, int qk_heads, const float* g, long long ldg, float scale, void* state,
               long long pool, const int* slots, void* out, long long ldo) {
  LaArgs a = {};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.g = g;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.state = state;
  a.slots = slots;
  a.ldq = ldq, a.ldk = ldk, a.ldv = ldv, a.ldg = ldg, a.ldo = ldo;
  a.rows = rows, a.pool = pool, a.heads = heads, a.share = heads / qk_heads, a.scale = scale;
  return a;
}

int launched() { return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ECUDA; }

}  // namespace

extern "C" int kda_la_step(const void* q, long long ldq, const void* k, long long ldk, const void* v, long long ldv,
                           long long rows, int heads, int qk_heads, const float* g, long long ldg, float scale,
                           void* state_pool, int state_dtype, long long pool_slots, const int* slots, void* out,
                           long long ldo, void* cuda_stream) {
  if (rows < 0) return KDA_EINVAL;
  if (rows == 0) return KDA_OK;
  if (!la_args_ok(rows, q, ldq, k, ldk, v, ldv, heads, qk_heads, g, ldg, state_pool, state_dtype, pool_slots, slots,
                  out, ldo))
    return KDA_EINVAL;
  if (rows > 0x7fffffffLL / STEP_SPLIT / heads) return KDA_EINVAL;
  const LaArgs a = la_args(q, ldq, k, ldk, v, ldv, rows, heads, qk_heads, g, ldg, scale, state_pool, pool_slots,
                           slots, out, ldo);
  const unsigned grid = (unsigned)(rows * heads * STEP_SPLIT);
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (state_dtype == KDA_STATE_BF16)
    la_step_kernel<true><<<grid, 32 * STEP_WARPS, 0, st>>>(a);
  else
    la_step_kernel<false><<<grid, 32 * STEP_WARPS, 0, st>>>(a);
  return launched();
}

extern "C" long long kda_la_prefill_workspace(long long rows, int heads, long long seqs, long long max_len) {
  (void)rows, (void)heads, (void)seqs, (void)max_len;
  return 0;
}

extern "C" int kda_la_prefill(const void* q, long long ldq, const void* k, long long ldk, const void* v,
                              long long ldv, long long rows, int heads, int qk_heads, const float* g, long long ldg,
                              float scale, const int* cu_seqlens, long long seqs, long long max_len,
                              const int* has_state, void* state_pool, int state_dtype, long long pool_slots,
                              const int* slots, void* out, long long ldo, void* workspace, long long workspace_bytes,
                              void* cuda_stream) {
  if (rows < 0 || rows > 0x7fffffffLL || seqs < 0 || max_len < 0) return KDA_EINVAL;
  if (seqs == 0) return KDA_OK;
  if (!la_args_ok(rows, q, ldq, k, ldk, v, ldv, heads, qk_heads, g, ldg, state_pool, state_dtype, pool_slots, slots,
                  out, ldo) ||
      !cu_seqlens || !aligned(cu_seqlens, 4) || !aligned(has_state, 4))
    return KDA_EINVAL;
  if (seqs > 0x7fffffffLL / STEP_SPLIT / heads) return KDA_EINVAL;
  const long long need = kda_la_prefill_workspace(rows, heads, seqs, max_len);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16))) return KDA_EINVAL;
  LaArgs a = la_args(q, ldq, k, ldk, v, ldv, rows, heads, qk_heads, g, ldg, scale, state_pool, pool_slots, slots,
                     out, ldo);
  a.cu = cu_seqlens, a.has_state = has_state, a.seqs = seqs, a.max_len = max_len;
  const unsigned grid = (unsigned)(seqs * heads * STEP_SPLIT);
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (state_dtype == KDA_STATE_BF16)
    la_scan_kernel<true><<<grid, 32 * STEP_WARPS, 0, st>>>(a);
  else
    la_scan_kernel<false><<<grid, 32 * STEP_WARPS, 0, st>>>(a);
  return launched();
}

extern "C" int kda_la_check(void* cuda_stream, unsigned* device_flags) {
  if (!device_flags) return KDA_EINVAL;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(cuda_stream)) != cudaSuccess) return KDA_ECUDA;
  unsigned v = 0;
  const unsigned zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_la_err, sizeof(v)) != cudaSuccess ||
      cudaMemcpyToSymbol(g_la_err, &zero, sizeof(zero)) != cudaSuccess)
    return KDA_ECUDA;
  *device_flags = v;
  return KDA_OK;
}

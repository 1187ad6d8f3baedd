// kda_linear_i8.cu -- the layer's projections on 8-bit operands on GB300
// (sm_103a): y[m, n] = sx[m] sw[n] sum_k x[m, k] W[n, k], int8 in, bf16 out
// (see include/kda_ops.h, kda_linear_i8).
//
// This GPU's integer matrix rate is a small fraction of its fp16 rate, and tcgen05 has no
// integer kind here.  Every int8 is a value of fp16, a product of two is below 2^14, and fp32
// sums of whole numbers are exact below 2^24: so the operands become fp16 on the way to the tensor
// core and the accumulator is the exact integer sum (rounded to fp32 where it passes 2^24).
// Widening four bytes is five instructions: flip the sign bits, put 0x64 above each byte (1024 + u
// in fp16), subtract 1024 + 128.
//
// Where the widened operands go decides the speed, because shared memory feeds everything
// (128 bytes a cycle).  The weight is the MMA's A operand and goes to tensor memory, straight from the
// registers that widened it; only the token rows (B) are written back to shared memory.  So a
// tile is 128 or 256 weight rows (lanes) by TN <= 192 tokens (columns); a 256 x 160 x 64 step is 640
// cycles of MMA against about 850 of shared memory.  Widened units (64 k) have three buffers where tensor
// memory has the room (TN <= 160), else two: with two the way from one unit's last MMA to the first on
// the same buffer (store, fence, barriers: 850 cycles) shows, 0.64 against 0.52 us a step.
//
// 4111 x 7168 x 6284: 294 us, 1260 TFLOP/s (cuBLAS bf16 here: 1914 in a burst, 1723 sustained), the tensor pipe
// busy 56 %; 512 rows 45 us; 64 x 1536 x 7168 9.0 us.
//
// Roles: two groups of warps widen the even and the odd units of 64 k (one alone took 1000
// cycles a unit, wait, read, widen and store one after the other), 4 or 8 of them W (a weight row a
// thread), 4 x; one warp issues the TMA copies (128 k a stage, 128-byte swizzle, zeros behind
// every edge), one the MMAs.  With few tiles K is
// split over a cluster of up to 8 CTAs, whose fp32 partial tiles are summed in rank order through
// distributed shared memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_ops.h"
#include "tc.cuh"

namespace {

constexpr int MAX_SPLIT = 8;   // portable cluster size
constexpr int MAX_TN = 192;    // tokens of a tile
constexpr int MAX_BUFS = 3;    // of widened units
constexpr int MAX_TN3 = 160;   // tokens of a tile with 3 of them: 2 x 160 + 3 x 64 columns of tensor memory (2 x 192 + 2 x 64)
constexpr int KSTAGE = 128;    // k a copy stage: the swizzle's 128 bytes
constexpr int I8_MAX_STAGES = 6;
constexpr int I8_MISC = 2048;
constexpr int I8_SMEM = 227 * 1024;
constexpr int X_WARPS = 4;     // of each of the two groups
constexpr int X_CHUNKS = MAX_TN * 4 / (32 * X_WARPS);  // 16-byte chunks of 64 k of x that a thread widens

// Device error bits, read and cleared by kda_linear_i8_check.
__device__ unsigned g_i8_err;

struct I8Args {
  const float *sx, *sw;
  __nv_bfloat16* y;
  long long M, N, K, ldy;
  int tn;       // tokens of a tile, a multiple of 16
  int tiles_m;  // token tiles
  int stages;   // of the copy ring
  int bufs;     // of widened units
  int vec;      // y's rows take 8-byte stores
};

struct I8Misc {
  float sx[MAX_TN];
  uint32_t tmem;
  int dead;
  unsigned long long bars[2 * I8_MAX_STAGES + 2 * MAX_BUFS + 1];
};
static_assert(sizeof(I8Misc) <= I8_MISC, "misc area");

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ unsigned cluster_size() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ unsigned cluster_id() {
  unsigned r;
  asm volatile("mov.u32 %0, %%clusterid.x;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 peer_f32x4(uint32_t local, unsigned rank) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(remote));
  return v;
}

// four int8 as two pairs of fp16
__device__ __forceinline__ void widen(uint32_t w, uint32_t& lo, uint32_t& hi) {
  w ^= 0x80808080u;
  const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
  const uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
  const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), bias);
  const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), bias);
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}

template <int MH>
__global__ void __launch_bounds__(32 * (2 * (4 * MH + X_WARPS) + 2), 1)
    i8_kernel(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap tw, const I8Args a) {
  constexpr int W_WARPS = 4 * MH, GROUP = W_WARPS + X_WARPS, TM = 128 * MH, THREADS = 32 * (2 * GROUP + 2);
  extern __shared__ __align__(1024) unsigned char dyn[];
  const uint32_t base = (smem_addr(dyn) + 1023u) & ~1023u;
  unsigned char* base_p = dyn + (base - smem_addr(dyn));
  I8Misc& sm = *reinterpret_cast<I8Misc*>(base_p);
  const uint32_t xbytes = (uint32_t)a.tn * 128u;         // 128 k of int8, and 64 k of fp16
  const uint32_t xc = base + I8_MISC, ring = xc + a.bufs * xbytes;
  const uint32_t stage_bytes = TM * 128 + xbytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned split = cluster_size(), rank = cluster_rank();
  const long long grp = cluster_id();
  // the token tiles of one weight tile are neighbours in launch order: all but the first find it in L2
  const long long m0 = (grp % a.tiles_m) * a.tn, n0 = (grp / a.tiles_m) * TM;
  const int total = (int)((a.K + KSTAGE - 1) / KSTAGE);
  const int s_begin = (int)((long long)total * rank / split);
  const int stages = (int)((long long)total * (rank + 1) / split) - s_begin;  // >= 1
  const uint32_t bars = smem_addr(sm.bars);
  auto full = [&](int i) { return bars + 8u * i; };
  auto empty = [&](int i) { return bars + 8u * (I8_MAX_STAGES + i); };
  auto conv_full = [&](int i) { return bars + 8u * (2 * I8_MAX_STAGES + i); };
  auto conv_empty = [&](int i) { return bars + 8u * (2 * I8_MAX_STAGES + MAX_BUFS + i); };
  const uint32_t done = bars + 8u * (2 * I8_MAX_STAGES + 2 * MAX_BUFS);
  if (threadIdx.x == 0) {
    prefetch_map(&tx);
    prefetch_map(&tw);
    for (int i = 0; i < I8_MAX_STAGES; ++i) bar_init(full(i), 1), bar_init(empty(i), 2 * GROUP);
    for (int i = 0; i < MAX_BUFS; ++i) bar_init(conv_full(i), GROUP), bar_init(conv_empty(i), 1);
    bar_init(done, 1);
    sm.dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2 * GROUP + 1) tmem_alloc(smem_addr(&sm.tmem), 512);
  after_previous();
  for (int i = threadIdx.x; i < a.tn; i += THREADS) sm.sx[i] = m0 + i < a.M ? a.sx[m0 + i] : 0.0f;
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *static_cast<volatile uint32_t*>(&sm.tmem);
  volatile int* dead = &sm.dead;
  const uint32_t acc_cols = a.bufs == 3 ? MAX_TN3 : MAX_TN;
  auto t_acc = [&](int half) { return tmem + acc_cols * half; };
  auto t_a = [&](int buf, int half) { return tmem + 2 * acc_cols + 64 * buf + 32 * half; };
  bool ok = true;

  const int grp2 = warp >= GROUP ? 1 : 0;        // the group, and its half of each stage's k
  const int gw = warp - grp2 * GROUP;            // the warp in its group
  if (warp < 2 * GROUP) {
    // Each unit is read and (W) widened before the wait for its buffer: what lies between one unit's MMAs
    // and the next one's on the same buffer is only the store.  (x widened there too measured slower, 122
    // against 81 us for 1024 x 7168 x 6284: twice the registers for it.)
    const int row = gw * 32 + lane;              // of the weight tile
    const int e0 = (gw - W_WARPS) * 32 + lane;   // of the x tile's 16-byte chunks, 32 X_WARPS apart
    int slot = 0, buf = grp2;              // of the ring; of the widened units (2 s + the group, mod bufs)
    unsigned round = 0, use = 0;           // parities of their uses
    auto arrive = [&](uint32_t bar) {
      __syncwarp();
      if (lane == 0) bar_arrive(bar);
    };
    for (int s = 0; s < stages; ++s) {
      if (!(ok = warp_wait(full(slot), round, dead))) break;
      const uint32_t st = ring + slot * stage_bytes;
      if (gw < W_WARPS) {
        uint32_t v[32];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 b = lds128(st + swz128(row, 4 * grp2 + i));
          widen(b.x, v[8 * i], v[8 * i + 1]);
          widen(b.y, v[8 * i + 2], v[8 * i + 3]);
          widen(b.z, v[8 * i + 4], v[8 * i + 5]);
          widen(b.w, v[8 * i + 6], v[8 * i + 7]);
        }
        arrive(empty(slot));
        if (2 * s + grp2 >= a.bufs && !(ok = warp_wait(conv_empty(buf), use ^ 1, dead))) break;
        tc_after();
        tmem_st(t_a(buf, gw >> 2) + ((uint32_t)((gw & 3) * 32) << 16), v);
        tmem_wait_st();
        tc_before();
      } else {
        const uint32_t xs = st + TM * 128, xd = xc + buf * xbytes;
        // eight rows' chunks at a time: no bank conflicts
        auto row_of = [](int e) { return (e >> 5) * 8 + (e & 7); };
        uint4 b[X_CHUNKS];
#pragma unroll
        for (int j = 0; j < X_CHUNKS; ++j) {
          const int e = e0 + 32 * X_WARPS * j;
          if (e < a.tn * 4) b[j] = lds128(xs + swz128(row_of(e), 4 * grp2 + ((e >> 3) & 3)));
        }
        arrive(empty(slot));
        if (2 * s + grp2 >= a.bufs && !(ok = warp_wait(conv_empty(buf), use ^ 1, dead))) break;
#pragma unroll
        for (int j = 0; j < X_CHUNKS; ++j) {
          const int e = e0 + 32 * X_WARPS * j;
          if (e < a.tn * 4) {
            uint4 c, d;
            widen(b[j].x, c.x, c.y);
            widen(b[j].y, c.z, c.w);
            widen(b[j].z, d.x, d.y);
            widen(b[j].w, d.z, d.w);
            sts128(xd + swz128(row_of(e), 2 * ((e >> 3) & 3)), c);
            sts128(xd + swz128(row_of(e), 2 * ((e >> 3) & 3) + 1), d);
          }
        }
        fence_async();
      }
      arrive(conv_full(buf));
      if (++slot == a.stages) slot = 0, round ^= 1;
      if ((buf += 2) >= a.bufs) buf -= a.bufs, use ^= 1;
    }
  } else if (warp == 2 * GROUP) {  // copies
    int slot = 0;
    unsigned round = 1;
    for (int s = 0; s < stages; ++s) {
      if (s >= a.stages && !(ok = warp_wait(empty(slot), round, dead))) break;
      if (elect()) {
        const uint32_t st = ring + slot * stage_bytes;
        const int k = (s_begin + s) * KSTAGE;
        bar_expect(full(slot), stage_bytes);
        tma_load(st, &tw, k, (int)n0, full(slot));
        tma_load(st + TM * 128, &tx, k, (int)m0, full(slot));
      }
      __syncwarp();
      if (++slot == a.stages) slot = 0, round ^= 1;
    }
  } else {  // matrix products
    const uint32_t id = idesc_f16(128, a.tn);
    int buf = 0;
    unsigned use = 0;
    for (int u = 0; u < 2 * stages; ++u) {  // 64 k each
      if (!(ok = warp_wait(conv_full(buf), use, dead))) break;
      tc_after();
      if (elect()) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint64_t b = desc_k(xc + buf * xbytes + 32 * k);
#pragma unroll
          for (int half = 0; half < MH; ++half) mma_ts(t_acc(half), t_a(buf, half) + 8 * k, b, id, u > 0 || k > 0);
        }
        mma_commit(conv_empty(buf));
        if (u + 1 == 2 * stages) mma_commit(done);
      }
      __syncwarp();
      if (++buf == a.bufs) buf = 0, use ^= 1;
    }
    if (!ok && elect()) mma_commit(done);
  }
  if (!ok) {
    *dead = 1;
    if (lane == 0) atomicOr(&g_i8_err, KDA_ERR_TIMEOUT);
  }
  __syncwarp();
  // everyone: the accumulators are final
  if (!warp_wait(done, 0, dead) && lane == 0) atomicOr(&g_i8_err, KDA_ERR_TIMEOUT);
  tc_after();
  __syncthreads();
  if (*dead) {
    // copies that were issued and not waited for land before the memory goes (~10 ms)
    const long long c0 = clock64();
    while (clock64() - c0 < 20000000ll) {
    }
  }
  __syncthreads();

  // Read-out, by W's warps of both groups (16 columns in turn): thread = weight row (an output column), accumulator columns = tokens.  The tile goes
  // through shared memory (the drained ring) so that the stores are along y's rows.
  const int rows = a.M - m0 < a.tn ? (int)(a.M - m0) : a.tn;      // tokens of this tile
  const int cols = a.N - n0 < TM ? (int)(a.N - n0) : TM;
  if (split == 1) {
    constexpr int LD = TM + 8;  // bf16 a row
    __nv_bfloat16* tile = reinterpret_cast<__nv_bfloat16*>(base_p + I8_MISC);
    if (warp < 2 * GROUP && gw < W_WARPS) {
      const int n = gw * 32 + lane;
      const float sw = n < cols ? a.sw[n0 + n] : 0.0f;
      for (int c = 16 * grp2; c < rows; c += 32) {
        uint32_t v[16];
        tmem_ld(t_acc(gw >> 2) + ((uint32_t)((warp & 3) * 32) << 16) + c, v);
        tmem_wait_ld(v);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          tile[(c + i) * LD + n] = __float2bfloat16_rn(__uint_as_float(v[i]) * sm.sx[c + i] * sw);
      }
      tc_before();
    }
    __syncthreads();
    for (int r = warp; r < rows; r += THREADS / 32) {
      __nv_bfloat16* y = a.y + (m0 + r) * a.ldy + n0;
      for (int c = 4 * lane; c < cols; c += 128) {
        const uint2 v = *reinterpret_cast<const uint2*>(tile + r * LD + c);
        if (a.vec && c + 4 <= cols) {
          *reinterpret_cast<uint2*>(y + c) = v;
        } else {
          const __nv_bfloat16* e = tile + r * LD + c;
          for (int i = 0; i < 4 && c + i < cols; ++i) y[c + i] = e[i];
        }
      }
    }
  } else {
    constexpr int LD = TM + 4, QUADS = TM / 4;  // fp32 a row; groups of four columns
    static_assert(I8_MISC + 4 * MAX_TN * LD <= I8_SMEM - 1024, "partial tile");
    float* red = reinterpret_cast<float*>(base_p + I8_MISC);
    if (warp < 2 * GROUP && gw < W_WARPS) {
      const int n = gw * 32 + lane;
      for (int c = 16 * grp2; c < rows; c += 32) {
        uint32_t v[16];
        tmem_ld(t_acc(gw >> 2) + ((uint32_t)((warp & 3) * 32) << 16) + c, v);
        tmem_wait_ld(v);
#pragma unroll
        for (int i = 0; i < 16; ++i) red[(c + i) * LD + n] = __uint_as_float(v[i]);
      }
      tc_before();
    }
    cluster_sync();
    // this CTA's share: groups of four columns, row by row
    const int e_end = (int)((long long)rows * QUADS * (rank + 1) / split);
    for (int e = (int)((long long)rows * QUADS * rank / split) + threadIdx.x; e < e_end; e += THREADS) {
      const int r = e / QUADS, n = (e % QUADS) * 4;
      if (n >= cols) continue;
      const uint32_t at = smem_addr(red + r * LD + n);
      float4 t[MAX_SPLIT];
#pragma unroll
      for (int q = 0; q < MAX_SPLIT; ++q)
        t[q] = (unsigned)q < split ? peer_f32x4(at, q) : make_float4(0.f, 0.f, 0.f, 0.f);
      float4 v = t[0];
#pragma unroll
      for (int q = 1; q < MAX_SPLIT; ++q) v.x += t[q].x, v.y += t[q].y, v.z += t[q].z, v.w += t[q].w;
      const float sx = sm.sx[r];
      const float f[4] = {v.x, v.y, v.z, v.w};
      __nv_bfloat16* y = a.y + (m0 + r) * a.ldy + n0 + n;
      if (a.vec && n + 4 <= cols) {
        const float* sw = a.sw + n0 + n;
        *reinterpret_cast<uint2*>(y) =
            make_uint2(pack_bf(f[0] * sx * sw[0], f[1] * sx * sw[1]), pack_bf(f[2] * sx * sw[2], f[3] * sx * sw[3]));
      } else {
        for (int i = 0; i < 4 && n + i < cols; ++i) y[i] = __float2bfloat16_rn(f[i] * sx * a.sw[n0 + n + i]);
      }
    }
    cluster_sync();  // the peers have read this CTA's partials
  }
  __syncthreads();
  if (warp == 2 * GROUP + 1) {
    tc_after();
    tmem_free(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// Few rows: mma.sync (m16n8k16, fp16) with 16 weight rows as M and 8 NT tokens as N, operands straight
// from global memory into fragments.  The product sums over k in any order, so a thread's 16
// contiguous bytes of a row serve as its four k of four steps (lane l: rows l / 4 and + 8, bytes
// 16 (l % 4) of 64), for W and x alike: no shared memory, no shuffles.  The 8 warps of a CTA take the
// 64-k chunks in turn and add their partial tiles through shared memory, in warp order.  The
// bound is the weight's bytes; UNROLL chunks of it are in flight a warp, and the CTAS resident
// CTAs cover each other's latency (loading ahead of the products measured slower, 12.2 against
// 10.5 us for 1 x 7168 x 6284: the registers cost more CTAs than that hides; asynchronous copies into rings of 3 to 8 chunks a
// warp, with two to four CTAs an SM, 11.3 to 13.1 against 11.6 there, 4.5 to 5.5 against 4.0 for 1 x 1536 x 7168).  45 MB
// in 11.6 us from a cold L2, 1 x 7168 x 49376 in 57.1: 6.8 TB/s for what lies between, 5 us for start and end.
constexpr int ROWS_WARPS = 8;

// 16 bytes, zeros where `in` is false; KEEP: in L1 (x, which every CTA of the SM reads).
template <bool KEEP>
__device__ __forceinline__ uint4 load16(const int8_t* p, bool in) {
  uint4 v;
  if (KEEP)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@p ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(p), "r"((uint32_t)in));
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@p ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(p), "r"((uint32_t)in));
  return v;
}

template <int NT, int UNROLL, int CTAS>
__global__ void __launch_bounds__(32 * ROWS_WARPS, CTAS)
    i8_rows_kernel(const int8_t* __restrict__ x, long long ldx, const int8_t* __restrict__ w, const I8Args a) {
  __shared__ float red[ROWS_WARPS][128 * NT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const long long n0 = (long long)blockIdx.x * 16;
  const int chunks = (int)((a.K + 63) / 64);
  const bool in0 = n0 + g < a.N, in1 = n0 + g + 8 < a.N;
  const int8_t* w0 = w + (n0 + g) * a.K + 16 * t;
  const int8_t* w1 = w0 + 8 * a.K;
  const int8_t* xp = x + g * ldx + 16 * t;
  after_previous();
  float acc[NT][4] = {};
  for (int c0 = warp; c0 < chunks; c0 += ROWS_WARPS * UNROLL) {
    uint4 wa[UNROLL], wb[UNROLL], xb[UNROLL][NT];
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) {
      const long long k = 64ll * (c0 + ROWS_WARPS * j);
      const bool in = k + 16 * t < a.K;
      wa[j] = load16<false>(w0 + k, in && in0);
      wb[j] = load16<false>(w1 + k, in && in1);
#pragma unroll
      for (int i = 0; i < NT; ++i) xb[j][i] = load16<true>(xp + 8 * i * ldx + k, in && g + 8 * i < a.M);
    }
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) {
      const uint32_t pa[4] = {wa[j].x, wa[j].y, wa[j].z, wa[j].w}, pb[4] = {wb[j].x, wb[j].y, wb[j].z, wb[j].w};
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        uint32_t a0, a1, a2, a3;
        widen(pa[s], a0, a2);
        widen(pb[s], a1, a3);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const uint32_t px[4] = {xb[j][i].x, xb[j][i].y, xb[j][i].z, xb[j][i].w};
          uint32_t b0, b1;
          widen(px[s], b0, b1);
          asm volatile(
              "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
              "{%0, %1, %2, %3};"
              : "+f"(acc[i][0]), "+f"(acc[i][1]), "+f"(acc[i][2]), "+f"(acc[i][3])
              : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
        }
      }
    }
  }
  // accumulator: 0, 1 at weight row g, tokens 2 t, + 1; 2, 3 eight weight rows down
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) red[warp][(8 * i + 2 * t + (j & 1)) * 16 + g + 8 * (j >> 1)] = acc[i][j];
  __syncthreads();
  for (int e = threadIdx.x; e < 128 * NT; e += 32 * ROWS_WARPS) {
    const int m = e >> 4;
    const long long n = n0 + (e & 15);
    if (m >= a.M || n >= a.N) continue;
    float v = 0.0f;
#pragma unroll
    for (int q = 0; q < ROWS_WARPS; ++q) v += red[q][e];
    a.y[m * a.ldy + n] = __float2bfloat16_rn(v * a.sx[m] * a.sw[n]);
  }
}

template <int NT, int UNROLL, int CTAS>
int i8_rows_launch(const void* x, long long ldx, const void* w, const I8Args& a, cudaStream_t st) {
  return launch(i8_rows_kernel<NT, UNROLL, CTAS>, (a.N + 15) / 16, 32 * ROWS_WARPS, 0, 1, st,
                static_cast<const int8_t*>(x), ldx, static_cast<const int8_t*>(w), a);
}

// A launch: weight-row halves, tokens a tile, K split.
struct I8Plan {
  int mh = 1, tn = 16, split = 1;
  double cost = 1e300;
};

int bufs_of(int tn) { return tn <= MAX_TN3 ? 3 : 2; }

int ring_stages(int mh, int tn) {
  const int room = I8_SMEM - 1024 - I8_MISC - bufs_of(tn) * tn * 128;
  const int n = room / ((128 * mh + tn) * 128);
  return n < I8_MAX_STAGES ? n : I8_MAX_STAGES;
}

template <int MH>
constexpr int i8_threads() {
  return 32 * (2 * (4 * MH + X_WARPS) + 2);
}

// Clusters of c CTAs that the device holds at once (a cluster stays within one GPC, so fewer
// than SMs / c), looked up once per device; 0 if that fails.
template <int MH>
int clusters_held(int dev, int c) {
  static std::atomic<int> cache[64][MAX_SPLIT + 1];
  int held = dev < 64 ? cache[dev][c].load(std::memory_order_relaxed) : 0;
  if (held <= 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)c, 1, 1);
    cfg.blockDim = dim3(i8_threads<MH>(), 1, 1);
    cfg.dynamicSmemBytes = I8_SMEM;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)c;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // the shared-memory attribute is per device
    if (cudaFuncSetAttribute(i8_kernel<MH>, cudaFuncAttributeMaxDynamicSharedMemorySize, I8_SMEM) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&held, i8_kernel<MH>, &cfg) != cudaSuccess)
      return 0;
    const int cap = sm_count(dev) / c;
    if (held > cap) held = cap;
    if (held > 0 && dev < 64) cache[dev][c].store(held, std::memory_order_relaxed);
  }
  return held;
}

// Time model of these tiles, in us, for 1 and 2 halves (fitted to 26 shapes of 17 to 4111 tokens, 256 to 12288 k
// and 512 to 49376 columns, every TN and C of each, 1200 launches; its pick is within 0.5 % of the
// fastest on average): a CTA runs its units of 64 k in max(low, base + per_token TN) (base2, per_token2
// with two buffers), or in its share of what the running CTAs' bytes take at `mb_per_us`, plus a fixed part,
// plus the split's sum; a last wave costs 1 - tail of a whole one and `tail` by its share.
struct I8Model {
  double low[2], base[2], per_token[2], base2[2], per_token2[2], mb_per_us, fixed[2], per_cell, split, split_cell, tail;
};
constexpr I8Model I8_MODEL = {{0.296, 0.450},     {0.244, 0.420}, {0.00078, 0.00061}, {0.273, 0.43},
                              {0.00094, 0.00096}, 18.6,           {4.12, 4.61},       0.0134,
                              0.75,               0.00607,        0.133};

// The launch that the model rates fastest.
I8Plan i8_plan(long long M, long long N, long long K, int dev) {
  constexpr I8Model t = I8_MODEL;
  I8Plan best;
  const long long units = (K + 63) / 64, stages = (K + KSTAGE - 1) / KSTAGE;
  for (int mh = 1; mh <= 2; ++mh) {
    const long long tiles_n = (N + 128 * mh - 1) / (128 * mh);
    for (int parts = 0; parts < 8; ++parts) {
      // tokens in the fewest tiles and up to 7 more, all of about one size
      const long long want = (M + MAX_TN - 1) / MAX_TN + parts;
      const int tn = (int)(((M + want - 1) / want + 15) / 16 * 16);
      const long long groups = tiles_n * ((M + tn - 1) / tn);
      double step = bufs_of(tn) == 3 ? t.base[mh - 1] + t.per_token[mh - 1] * tn
                                     : t.base2[mh - 1] + t.per_token2[mh - 1] * tn;
      if (step < t.low[mh - 1]) step = t.low[mh - 1];
      const double mb = (128.0 * mh + tn) * 64e-6;
      for (int c = 1; c <= MAX_SPLIT && c <= stages; ++c) {
        const int held = mh == 2 ? clusters_held<2>(dev, c) : clusters_held<1>(dev, c);
        if (held <= 0) continue;
        const double w = (double)groups / held, whole = (double)((groups + held - 1) / held);
        const double waves = w <= 1.0 ? 1.0 : whole - t.tail * (whole - w);
        const double running = (double)(groups < held ? groups : held) * c, feed = running * mb / t.mb_per_us;
        const double cost =
            waves * ((double)units / c * (step > feed ? step : feed) + t.fixed[mh - 1] + t.per_cell * tn * mh +
                     (c > 1 ? t.split + t.split_cell * tn * mh : 0.0));
        if (cost < best.cost * (1.0 - 1e-9)) best.cost = cost, best.mh = mh, best.tn = tn, best.split = c;
      }
      if (tn <= 16) break;
    }
  }
  return best;
}

template <int MH>
int i8_launch(const void* x, long long ldx, const void* w, I8Args a, const I8Plan& p, cudaStream_t st) {
  CUtensorMap tx, tw;
  const CUtensorMapDataType t = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const CUtensorMapSwizzle s = CU_TENSOR_MAP_SWIZZLE_128B;
  if (!encode_2d(&tx, t, x, a.M, a.K, ldx, KSTAGE, p.tn, s) ||
      !encode_2d(&tw, t, w, a.N, a.K, a.K, KSTAGE, 128 * MH, s))
    return KDA_ECUDA;
  a.tn = p.tn;
  a.tiles_m = (int)((a.M + p.tn - 1) / p.tn);
  a.stages = ring_stages(MH, p.tn);
  a.bufs = bufs_of(p.tn);
  const long long groups = (a.N + 128 * MH - 1) / (128 * MH) * a.tiles_m;
  if (groups * p.split > 0x7fffffffLL) return KDA_EINVAL;
  return launch(i8_kernel<MH>, groups * p.split, i8_threads<MH>(), I8_SMEM, p.split, st, tx, tw, a);
}

}  // namespace

extern "C" int kda_linear_i8(const void* x, long long rows, long long ldx, const float* x_scales, const void* w,
                             const float* w_scales, long long N, long long K, void* y, long long ldy,
                             void* cuda_stream) {
  if (rows < 0 || N < 1 || K < 16 || K % 16 != 0) return KDA_EINVAL;
  if (rows == 0) return KDA_OK;
  if (!x || !x_scales || !w || !w_scales || !y || ldx < K || ldx % 16 != 0 || ldy < N) return KDA_EINVAL;
  if (!ptr_aligned(x, 16) || !ptr_aligned(w, 16) || !ptr_aligned(y, 2) || !ptr_aligned(x_scales, 4) ||
      !ptr_aligned(w_scales, 4))
    return KDA_EINVAL;
  // tensor-map coordinates fit 32 bits
  if (K > 0x7fffff00LL || N > 0x7fffff00LL || rows > 0x7fffff00LL) return KDA_EINVAL;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KDA_ECUDA;
  if (!on_device(x, dev) || !on_device(w, dev) || !on_device(y, dev)) return KDA_EINVAL;
  I8Args a = {};
  a.sx = x_scales, a.sw = w_scales;
  a.y = static_cast<__nv_bfloat16*>(y);
  a.M = rows, a.N = N, a.K = K, a.ldy = ldy;
  a.vec = ptr_aligned(y, 8) && ldy % 4 == 0;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (rows <= 8) return i8_rows_launch<1, 3, 4>(x, ldx, w, a, st);
  if (rows <= 16) return i8_rows_launch<2, 2, 3>(x, ldx, w, a, st);
  const I8Plan p = i8_plan(rows, N, K, dev);
  if (p.cost >= 1e300) return KDA_ECUDA;
  // 17 to 32 rows: the fragments kernel where few k make the tiles' fixed part count (32 x 1536 x 7168: 6.1
  // against 9.8 us; 32 x 7168 x 1154: 13.5 against 10.7).  Its time: a start, and 8 warps' 512 k
  // at a time, longer as more CTAs share an SM.
  if (rows <= 32) {
    const double per_sm = (double)((N + 15) / 16) / sm_count(dev);
    if (2.5 + (double)((K + 511) / 512) * (0.75 + (per_sm > 1.0 ? 0.26 * (per_sm - 1.0) : 0.0)) < p.cost)
      return i8_rows_launch<4, 1, 3>(x, ldx, w, a, st);
  }
  return p.mh == 2 ? i8_launch<2>(x, ldx, w, a, p, st) : i8_launch<1>(x, ldx, w, a, p, st);
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

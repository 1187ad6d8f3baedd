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
// bytes, read and written once: 512 rows x 12 heads, fp32, 812 MB in 120.4 us, 0.99 of the measured
// copy bandwidth; one row of 2 heads takes 2.2 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_ops.h"
#include "tc.cuh"

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
  after_previous();
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

// ---------------------------------------------------------------------------
// Prompts.  With G_i the sum of the log decays of tokens 0..i of a chunk (C = 128
// tokens), R_j that of the tokens behind j, and S the state before the chunk,
//   o_i = scale (e^{G_i} S q_i + sum_{j <= i} e^{G_i - G_j} (q_i . k_j) v_j)
//   S'  = e^{G_C} S + sum_j v_j (e^{R_j} k_j)^T
// so a chunk is matrix products: scores Q K^T, their decayed lower triangle P times V, Q S^T, and
// K'^T V with K' the decayed keys.  One CTA takes a segment (a run of chunks of one
// sequence and head) and carries S from chunk to chunk in fp32 registers; the
// products run on tcgen05.  Every exponent is at most 0.
//
// What is rounded: P and, as an operand of Q S^T, S to bf16 (an output of bf16
// anyway).  The state itself is summed from exact parts: K' = hi + mid + lo in bf16 (24
// bits; hi + mid where only bf16 comes of it), each chunk's sum added to S in fp32
// registers, so that nothing accumulates in the tensor pipe over chunks.
//
// What bounds it is shared memory's 128 bytes a cycle: a 128 x 128 x 16 MMA takes 8 KB of
// operands in its 64 cycles.  So the A operands that threads make themselves, P and K'^T, go
// to tensor memory: 128 columns of scores that become P (64) and lo (64), 128 of hi and
// mid, 128 of outputs (Q S^T, scaled there by e^{G_i}, PV added on top), 128 of K'^T V.
//
// Measured: 8192 tokens x 12 heads 43 us in a replayed graph (segments of 6 chunks; 101 MB, 14.9 us at the
// copy bandwidth): OWN 15 us, the join 7, OUTPUT's chunks 19.  A chunk takes 3.2 us in the DIRECT kernel, about 6200 cycles
// of which 3950 are MMAs, 1.6 in OWN and 2.9 in OUTPUT; one chunk by itself 7.8 us.  (Keys on eight warps of their own:
// 5 % less a chunk in DIRECT, no less where 132 CTAs run, and 2 us more for short prompts.)
//
// Roles (warps): 0-15 compute, 16 TMA copies (two stages of Q, K, V) and the decays, 17 MMAs.
//   MMA:     QK QS | mid, hi | lo PV                | QK ...
//   compute: scores -> P; QS * e^G | K -> K' of the next chunk | S += K'^T V | outputs
//
// A long sequence is split into segments to fill the GPU: la_chunk_kernel<OWN> computes each
// segment's own contribution to the state, la_join_kernel turns these into the states the segments
// start from and the one behind the last, and la_chunk_kernel<OUTPUT> runs all segments at once for their
// outputs (its states end as bf16 operands, so hi and mid will do).  la_chunk_kernel<DIRECT> does all of it for a sequence
// that is not split: for all of them if none is, else in a fourth launch, whose CTAs take the SMs that OUTPUT's leave
// (16384 tokens and 255 x 64 of 12 heads: 256 us; all in segments 712, none 423).
constexpr int CHUNK = 128;
constexpr int BOX = 64 * 128 * 2;          // 64 columns of 128 rows, bf16
constexpr int TILE = 2 * BOX;              // a 128 x 128 bf16 operand
constexpr int COMPUTE_WARPS = 16;          // four for each quarter of an accumulator's 128 rows
constexpr int CHUNK_THREADS = 32 * (COMPUTE_WARPS + 2);
constexpr int MISC = 2048;                 // ChunkMisc
constexpr int CHUNK_SMEM = 7 * TILE + MISC + 1024;  // (1024: the alignment of the swizzled tiles)
static_assert(CHUNK_SMEM <= 227 * 1024, "shared memory of one CTA");
constexpr float LOG2E = 1.4426950408889634f;
constexpr float G_MIN = -104.0f;  // e^-104 is below fp32's smallest step

// segments of a sequence of `len` tokens: runs of m chunks; an empty one has one, without chunks
__device__ __forceinline__ long long seg_count(long long len, int m) {
  const long long per = (long long)m * CHUNK;
  return len <= per ? 1 : (len + per - 1) / per;
}
__device__ __forceinline__ bool seq_ok(const LaArgs& a, long long begin, long long end) {
  return begin >= 0 && end >= begin && end <= a.rows && end - begin <= a.max_len;
}

struct Segment {
  int seq, index, count;  // which sequence; which of its `count` segments
  long long begin, end;   // the sequence's rows
};
struct ChunkArgs {
  LaArgs a;
  float* ws;        // [parts, heads, 128 (v), 128 (k)]: a segment's own state, then the one it starts from
  float* decays;    // [parts, heads]: log2 of the decay over a segment
  int m;            // chunks a segment
  int least;        // sequences of so many segments are split: 2, 1 (every one), or 0: none is
  long long parts;  // the split sequences' segments, at most
};
// A warp looks for a part, a segment of a split sequence, by its number among all parts (by_seq false), or for the first
// part of a split sequence, by the sequence's number among its like (by_seq true).  False if there is none, or if the
// rest of its sequence passes the limit: ascending cu_seqlens never get there, and overlapping ones
// stay within the workspace.
__device__ bool find_part(const ChunkArgs& p, long long want, bool by_seq, Segment* s, long long* number) {
  const LaArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  long long before = 0, split_before = 0;
  for (long long i0 = 0; i0 < a.seqs; i0 += 32) {
    const long long i = i0 + lane;
    long long b = 0, e = 0;
    int n = 0;
    if (i < a.seqs) {
      b = a.cu[i], e = a.cu[i + 1];
      if (seq_ok(a, b, e)) n = (int)seg_count(e - b, p.m);
      if (n < p.least) n = 0;
    }
    long long upto = n;  // parts of the sequences i0 .. i
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += t;
    }
    const unsigned split = __ballot_sync(0xffffffffu, n > 0);
    const long long first = before + upto - n;
    const bool here = by_seq ? n > 0 && split_before + __popc(split & ((1u << lane) - 1)) == want
                             : first <= want && want < first + n;
    const unsigned who = __ballot_sync(0xffffffffu, here);
    if (who) {
      const int l = __ffs(who) - 1;
      const long long f = __shfl_sync(0xffffffffu, first, l);
      s->seq = (int)(i0 + l);
      s->count = __shfl_sync(0xffffffffu, n, l);
      s->begin = __shfl_sync(0xffffffffu, b, l);
      s->end = __shfl_sync(0xffffffffu, e, l);
      s->index = by_seq ? 0 : (int)(want - f);
      *number = f + s->index;
      return f + s->count <= p.parts;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
    split_before += __popc(split);
  }
  return false;
}
// Sequence `seq` by itself, if it is not split.
__device__ bool find_whole(const ChunkArgs& p, long long seq, Segment* s) {
  const long long b = p.a.cu[seq], e = p.a.cu[seq + 1];
  *s = Segment{(int)seq, 0, 1, b, e};
  return seq_ok(p.a, b, e) && (p.least == 0 || seg_count(e - b, p.m) < p.least);
}

// the upper 16 bits of two floats, and a float without its lower 16: bf16 parts cut off, not rounded
__device__ __forceinline__ uint32_t top_halves(float lo, float hi) {
  return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}
__device__ __forceinline__ float bf_cut(float x) { return bf_hi(__float_as_uint(x)); }

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

enum {  // barriers: completed by copies and MMAs (one arrival), two stages of each, ...
  FULL_Q, FULL_K = FULL_Q + 2, FULL_V = FULL_K + 2, EMPTY_V = FULL_V + 2,
  SCORES = EMPTY_V + 2, FROM_S, HI_DONE, DELTA, OUT, DRAIN,
  DECAY_W, DECAY_G,                         // ... by the decays' warp, ...
  EMPTY_K, EMPTY_Q = EMPTY_K + 2,           // ... by the compute warps (EMPTY_K: and QK's commit), two stages, ...
  KP = EMPTY_Q + 2, P_IN, S_IN, O_READ,     // ... by the compute warps, ...
  QUARTER, BARS = QUARTER + 4               // ... by the four warps of a quarter of the rows
};
struct ChunkMisc {
  float G[CHUNK];  // G_i (log2)
  float W[CHUNK];  // e^{R_j}, used up to the sequence's end
  float E[CHUNK];  // e^{G_b - G_j}, G_b the last G of j's block of 16
  float total;     // G_C (log2)
  int found, dead, slot, resumed;
  uint32_t tmem;
  long long number;
  Segment seg;
  unsigned long long bars[BARS];
};
static_assert(sizeof(ChunkMisc) <= MISC, "misc area");

enum Mode { DIRECT, OWN, OUTPUT };

// BF: a bf16 pool (DIRECT; the other two read and write the workspace's fp32 only)
template <Mode MODE, bool BF>
__global__ void __launch_bounds__(CHUNK_THREADS, 1)
    la_chunk_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                    const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap to,
                    const ChunkArgs p) {
  constexpr bool LOCAL = MODE == OWN, LO = MODE == OWN || (MODE == DIRECT && !BF);  // with the third part of K'
  const LaArgs& a = p.a;
  extern __shared__ __align__(1024) unsigned char dyn[];
  // (all shared memory is dynamic: the seven operand tiles leave no room for a second alignment)
  const uint32_t base = (smem_addr(dyn) + 1023u) & ~1023u;
  const uint32_t ss = base + 6 * TILE;  // S for Q S^T; before it two stages of Q, K, V
  ChunkMisc& sm = *reinterpret_cast<ChunkMisc*>(dyn + (base - smem_addr(dyn)) + 7 * TILE);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = (int)(blockIdx.x % a.heads), hk = h / a.share;
  const uint32_t bars = smem_addr(sm.bars);
  auto bar = [&](int i) { return bars + 8u * i; };
  // which segment, the barriers and the tensor memory, each by a warp, then one barrier
  // The first kernel of a call reads nothing before the stream's work before it has ended; those behind it are
  // launched when it has passed this, so they wait where they read another's results, or as they end.
  const bool first = LOCAL || (MODE == DIRECT && p.least == 0);
  // What ends behind a kernel that it has not waited for: this one does not end before it, for which one CTA's wait will
  // do where the kernel before takes long (every CTA's would keep the SMs from the others: 8192 tokens of 4 sequences
  // and 12 heads 50 us).
  const bool ends_after = !first && (MODE == OUTPUT || blockIdx.x == gridDim.x - 1);
  if (warp == 0) {
    if (first) asm volatile("griddepcontrol.wait;" ::: "memory");
    Segment s;
    long long number = 0;
    const long long task = blockIdx.x / a.heads;
    const bool found = MODE == DIRECT ? find_whole(p, task, &s) : find_part(p, task, false, &s, &number);
    if (lane == 0) {
      sm.found = found, sm.dead = 0;
      if (found) {
        sm.seg = s, sm.number = number;
        sm.slot = a.slots[s.seq];
        sm.resumed = MODE == OUTPUT || (MODE == DIRECT && a.has_state && a.has_state[s.seq]);
      }
    }
    if ((MODE == DIRECT || (MODE == OUTPUT && p.least == 1)) && blockIdx.x == 0) {  // bad pairs of cu_seqlens: once
      bool bad = false;
      long long parts = 0;
      for (long long i = lane; i < a.seqs; i += 32) {
        const long long b = a.cu[i], e = a.cu[i + 1];
        if (!seq_ok(a, b, e)) {
          bad = true;
        } else if (p.least > 0) {
          const long long n = seg_count(e - b, p.m);
          parts += n < p.least ? 0 : n;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) parts += __shfl_xor_sync(0xffffffffu, parts, o);
      if (bad || parts > p.parts) atomicOr(&g_la_err, KDA_ERR_SEQ);
    }
  } else if (warp == COMPUTE_WARPS) {
    if (lane == 0) {
      for (int i = 0; i < BARS; ++i)
        bar_init(bar(i), i >= QUARTER                         ? 4
                         : i == EMPTY_K || i == EMPTY_K + 1 ? COMPUTE_WARPS + (LOCAL ? 0 : 1)
                         : i >= EMPTY_Q                     ? COMPUTE_WARPS
                                                            : 1);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      if (!LOCAL) prefetch_map(&tq), prefetch_map(&to);
      prefetch_map(&tk);
      prefetch_map(&tv);
    }
  } else if (warp == COMPUTE_WARPS + 1) {
    tmem_alloc(smem_addr(&sm.tmem), 512);
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *static_cast<volatile uint32_t*>(&sm.tmem);
  if (first) after_previous();
  // (the sequences that are not split need nothing of these kernels: they may start while OUTPUT waits for the join)
  if (MODE == OUTPUT) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // A CTA without work: no segment, a padding sequence (its rows zero), a bad slot, an empty sequence (its
  // state stays, or is zeros; the join's where there is one).
  const Segment sg = sm.seg;
  const long long number = sm.number;
  const int slot = sm.slot;
  const bool resumed = sm.resumed;  // starts from a state
  const long long row0 = sg.begin + (long long)sg.index * p.m * CHUNK;
  const long long left = sg.end - row0;
  const int tokens = (int)(left < (long long)p.m * CHUNK ? left : (long long)p.m * CHUNK);
  const int chunks = (tokens + CHUNK - 1) / CHUNK;
  const bool slot_ok = slot >= 0 && slot < a.pool;
  unsigned char* pool = static_cast<unsigned char*>(a.state) + ((long long)slot * a.heads + h) * (D * D) * (BF ? 2 : 4);
  if (!sm.found || !slot_ok || chunks == 0) {
    if (sm.found && !LOCAL) {
      if (slot == -1) {
        for (int e = threadIdx.x; e < tokens * (D / 8); e += CHUNK_THREADS)
          *reinterpret_cast<uint4*>(a.out + (row0 + e / (D / 8)) * a.ldo + h * D + 8 * (e % (D / 8))) =
              make_uint4(0, 0, 0, 0);
      } else if (!slot_ok) {
        if (threadIdx.x == 0) atomicOr(&g_la_err, KDA_ERR_SLOT);
      } else if (MODE == DIRECT && !resumed) {
        for (int e = threadIdx.x; e < D * D * (BF ? 2 : 4) / 16; e += CHUNK_THREADS)
          reinterpret_cast<uint4*>(pool)[e] = make_uint4(0, 0, 0, 0);
      }
    }
    if (warp == COMPUTE_WARPS + 1) tmem_free(tmem, 512);
    // (a kernel behind this one waits for this one alone)
    if (ends_after) after_previous();
    return;
  }
  float* wsp = p.ws + (number * a.heads + h) * (D * D);
  // tensor memory: scores, then P and lo; hi and mid; outputs; K'^T V.  (LOCAL: two sets of hi, mid, lo; K'^T V)
  const uint32_t t_sc = tmem, t_p = tmem, t_o = tmem + 256, t_ds = tmem + 384;
  auto t_hi = [&](int c) { return LOCAL ? tmem + 192 * (c & 1) : tmem + 128; };
  auto t_mid = [&](int c) { return t_hi(c) + 64; };
  auto t_lo = [&](int c) { return LOCAL ? t_hi(c) + 128 : tmem + 64; };
  auto sq = [&](int c) { return base + 3 * TILE * (c & 1); };
  auto sk = [&](int c) { return sq(c) + TILE; };
  auto sv = [&](int c) { return sq(c) + 2 * TILE; };
  volatile int* dead = &sm.dead;
  auto wait = [&](int i, unsigned ph) { return warp_wait(bar(i), ph, dead); };  // whole warps only
  // the state behind the segment's last chunk is wanted: by the pool, or (OWN) by the join
  constexpr bool want_last = MODE != OUTPUT;
  bool ok = true;

  if (warp < COMPUTE_WARPS) {
    const int quarter = warp & 3, part = warp >> 2;
    const int r = quarter * 32 + lane;  // this thread's row of every accumulator: a token, or a k of the state ...
    const int c0 = 32 * part;           // ... and its 32 columns
    const uint32_t lane_at = (uint32_t)(quarter * 32) << 16;
    // 16-byte chunk i (0..3) of these columns in a 128-byte-swizzled tile of bf16
    auto chunk_at = [&](int i) { return (part >> 1) * BOX + swz128(r, 4 * (part & 1) + i); };
    auto arrive = [&](int i) {
      __syncwarp();
      if (lane == 0) bar_arrive(bar(i));
    };
    // All of the above and the first copies overlap the join; the state the segment starts from is its result.
    if (MODE == OUTPUT) after_previous();
    float S[32];  // S[v = c0 ..][k = r]
    if (resumed) {
      const long long at = (long long)c0 * D + r;
      if (MODE == DIRECT && BF) {
        const uint16_t* f = reinterpret_cast<const uint16_t*>(pool) + at;
#pragma unroll
        for (int i = 0; i < 32; ++i) S[i] = __uint_as_float((uint32_t)f[i * D] << 16);
      } else {
        const float* f = reinterpret_cast<const float*>(MODE == OUTPUT ? reinterpret_cast<unsigned char*>(wsp) : pool) + at;
#pragma unroll
        for (int i = 0; i < 32; ++i) S[i] = __ldcg(f + i * D);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) S[i] = 0.0f;
    }
    // S as the bf16 operand of Q S^T: rows k, 64 v a box
    auto put_state = [&]() {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        sts128(ss + chunk_at(i),
               make_uint4(pack_bf(S[8 * i], S[8 * i + 1]), pack_bf(S[8 * i + 2], S[8 * i + 3]),
                          pack_bf(S[8 * i + 4], S[8 * i + 5]), pack_bf(S[8 * i + 6], S[8 * i + 7])));
      fence_async();
    };
    auto wanted = [&](int c) { return want_last || c + 1 < chunks; };
    auto count_of = [&](int c) { return tokens - c * CHUNK < CHUNK ? tokens - c * CHUNK : CHUNK; };
    uint32_t lo[2][8];
    float total = 0.0f;  // of the chunk whose K' was made last

    // K'^T = hi + mid + lo of chunk c: k quarter * 32 .. + 31, tokens c0 .. + 31, two a column.  The
    // transpose is ldmatrix's, whose fragments are what tensor memory takes in 16 x 128-bit form:
    // thread l has k = l / 4 + 8 i, tokens 2 (l % 4), + 1 (+ 8 g).  Cutting bits off (not rounding)
    // gives three parts of 8 bits that add up to all 24.
    auto keys = [&](int c) {
      const int n = count_of(c) - c0 - 2 * (lane & 3);  // the thread's first token is in its chunk if > 0, ...
      if (!wait(DECAY_W, c & 1) || !wait(FULL_K + (c & 1), (c >> 1) & 1)) return false;
      total = sm.total;
      if (wanted(c)) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // 16 k
          uint32_t hi[8], mid[8];
#pragma unroll
          for (int g2 = 0; g2 < 4; g2 += 2) {  // 16 tokens
            uint32_t u[4];
            const int j = c0 + 8 * (g2 + (lane >> 4)) + (lane & 7);
            const int k8 = quarter * 4 + half * 2 + ((lane >> 3) & 1);  // 8 k: a 16-byte chunk
            ldsm_x4_trans(u, sk(c) + (k8 >> 3) * BOX + swz128(j, k8 & 7));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int g = g2 + e;
              const float2 w = *reinterpret_cast<const float2*>(sm.W + c0 + 8 * g + 2 * (lane & 3));
              // rows behind the sequence's end are somebody else's: not even times zero
              const uint32_t live = n > 8 * g + 1 ? 0xffffffffu : n > 8 * g ? 0xffffu : 0u;
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int o = 2 * g + i;
                const uint32_t x = u[2 * e + i] & live;
                float f0 = bf_lo(x) * w.x, f1 = bf_hi(x) * w.y;
                hi[o] = top_halves(f0, f1);
                f0 -= bf_cut(f0), f1 -= bf_cut(f1);
                if (!LO) {
                  mid[o] = pack_bf(f0, f1);
                } else {
                  mid[o] = top_halves(f0, f1);
                  f0 -= bf_cut(f0), f1 -= bf_cut(f1);
                  lo[half][o] = top_halves(f0, f1);
                }
              }
            }
          }
          const uint32_t at = lane_at + ((uint32_t)(16 * half) << 16) + c0 / 2;
          tmem_st_frag(t_hi(c) + at, hi);
          tmem_st_frag(t_mid(c) + at, mid);
          if (LOCAL) tmem_st_frag(t_lo(c) + at, lo[half]);
        }
        tmem_wait_st();
        tc_before();
      }
      arrive(EMPTY_K + (c & 1));
      if (count_of(c) < CHUNK) {  // nor are their values multiplied by the zeros of P and K'
        if (!wait(FULL_V + (c & 1), (c >> 1) & 1)) return false;
        if (r >= count_of(c))
#pragma unroll
          for (int i = 0; i < 4; ++i) sts128(sv(c) + chunk_at(i), make_uint4(0, 0, 0, 0));
        fence_async();
      }
      arrive(KP);
      return true;
    };

    put_state();
    arrive(S_IN);
    float seg_decay = 0.0f;
    ok = keys(0);
    for (int c = 0; c < chunks && ok; ++c) {
      const unsigned ph = c & 1;
      const bool from_state = resumed || c > 0;
      if (!LOCAL) {
        // the scores' lower triangle, decayed: row i = r
        if (!(ok = wait(DECAY_G, ph))) break;
        const float gi = sm.G[r];
        if (!(ok = wait(SCORES, ph))) break;
        tc_after();
        uint32_t pk[16];
        if (part <= quarter) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int j0 = c0 + 16 * q;
            uint32_t x[16];
            tmem_ld(t_sc + lane_at + j0, x);
            tmem_wait_ld(x);
            const float s = ex2(gi - sm.G[j0 + 15]);
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              float f[4];
              if (part < quarter) {  // all of these tokens are before all of the warp's
                const float4 e = *reinterpret_cast<const float4*>(sm.E + j0 + j);
                f[0] = e.x * s, f[1] = e.y * s, f[2] = e.z * s, f[3] = e.w * s;
              } else {
                const float4 g = *reinterpret_cast<const float4*>(sm.G + j0 + j);
                f[0] = ex2(gi - g.x), f[1] = ex2(gi - g.y), f[2] = ex2(gi - g.z), f[3] = ex2(gi - g.w);
              }
#pragma unroll
              for (int i = 0; i < 4; ++i)
                f[i] = part < quarter || 16 * q + j + i <= lane ? f[i] * __uint_as_float(x[j + i]) : 0.0f;
              pk[8 * q + j / 2] = pack_bf(f[0], f[1]);
              pk[8 * q + j / 2 + 1] = pack_bf(f[2], f[3]);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) pk[i] = 0u;
        }
        // P and lo take the scores' place, once all four warps of these lanes have read theirs
        tc_before();
        arrive(QUARTER + quarter);
        if (!(ok = wait(QUARTER + quarter, ph))) break;
        tc_after();
        tmem_st(t_p + lane_at + c0 / 2, pk);
        if (LO && wanted(c)) {
          tmem_st_frag(t_lo(c) + lane_at + c0 / 2, lo[0]);
          tmem_st_frag(t_lo(c) + lane_at + (16u << 16) + c0 / 2, lo[1]);
        }
        if (from_state) {  // Q S^T times e^{G_i}: PV adds to it
          if (!(ok = wait(FROM_S, ph))) break;
          tc_after();
          const float eg = ex2(gi);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t x[16];
            tmem_ld(t_o + lane_at + c0 + 16 * q, x);
            tmem_wait_ld(x);
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * eg);
            tmem_st(t_o + lane_at + c0 + 16 * q, x);
          }
        }
        tmem_wait_st();
        tc_before();
        arrive(P_IN);
        if (c > 0) {  // the chunk before's outputs have left its Q
          if (lane == 0) tma_store_read();
          arrive(EMPTY_Q + (ph ^ 1));
        }
      }
      const float decay = total;
      if (c + 1 < chunks) {
        if (!LOCAL && !(ok = wait(HI_DONE, ph))) break;
        if (!(ok = keys(c + 1))) break;
      }
      if (wanted(c)) {
        if (!(ok = wait(DELTA, ph))) break;
        tc_after();
        seg_decay += decay;
        const float d = ex2(decay);
        uint32_t y[32];
        tmem_ld(t_ds + lane_at + c0, y);
        tmem_wait_ld(y);
#pragma unroll
        for (int i = 0; i < 32; ++i) S[i] = fmaf(d, S[i], __uint_as_float(y[i]));
        if (!LOCAL && c + 1 < chunks) put_state();
        tc_before();
      }
      arrive(S_IN);
      if (!LOCAL) {
        const int n = count_of(c);
        if (!(ok = wait(OUT, ph))) break;
        tc_after();
        // by way of shared memory, 2 KB of Q (which nobody reads any more) a warp: rows of 64 bytes,
        // 64-byte swizzle (16-byte chunk i of row r at i ^ (r / 2) % 4), sent as one box if all 32 are the sequence's
        const uint32_t stage = sq(c) + warp * 2048;
        auto at64 = [&](int row, int i) { return stage + row * 64 + ((i ^ ((row >> 1) & 3)) << 4); };
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t y[16];
          tmem_ld(t_o + lane_at + c0 + 16 * q, y);
          tmem_wait_ld(y);
          uint32_t w[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            w[j] = pack_bf(a.scale * __uint_as_float(y[2 * j]), a.scale * __uint_as_float(y[2 * j + 1]));
          sts128(at64(lane, 2 * q), make_uint4(w[0], w[1], w[2], w[3]));
          sts128(at64(lane, 2 * q + 1), make_uint4(w[4], w[5], w[6], w[7]));
        }
        tc_before();
        arrive(O_READ);
        const long long row = row0 + (long long)c * CHUNK + quarter * 32;
        fence_async();
        __syncwarp();
        if (n >= quarter * 32 + 32) {
          if (lane == 0) tma_store(&to, h * D + c0, (int)row, stage);
        } else {
          __nv_bfloat16* o = a.out + row * a.ldo + h * D + c0 + 8 * (lane & 3);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = 8 * i + (lane >> 2);
            const uint4 u = lds128(at64(t, lane & 3));
            if (quarter * 32 + t < n) *reinterpret_cast<uint4*>(o + t * a.ldo) = u;
          }
        }
      }
    }
    if (MODE == DIRECT && ends_after) after_previous();
    if (!LOCAL && lane == 0) tma_store_read();  // before the memory goes
    if (ok && want_last) {
      const long long at = (long long)c0 * D + r;
      if (MODE == DIRECT && BF) {
        __nv_bfloat16* f = reinterpret_cast<__nv_bfloat16*>(pool) + at;
#pragma unroll
        for (int i = 0; i < 32; ++i) f[i * D] = __float2bfloat16_rn(S[i]);
      } else {
        float* f = reinterpret_cast<float*>(LOCAL ? reinterpret_cast<unsigned char*>(wsp) : pool) + at;
#pragma unroll
        for (int i = 0; i < 32; ++i) f[i * D] = S[i];
        if (LOCAL && threadIdx.x == 0) p.decays[number * a.heads + h] = seg_decay;
      }
    }
  } else if (warp == COMPUTE_WARPS) {  // copies, and the decays (four tokens a lane)
    for (int c = 0; c < chunks; ++c) {
      const int row = (int)(row0 + (long long)c * CHUNK);
      const long long t0 = row0 + (long long)c * CHUNK + 4 * lane;
      const int n = tokens - c * CHUNK;
      float g[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) g[j] = 4 * lane + j < n ? a.g[(t0 + j) * a.ldg + h] : 0.0f;
      auto load = [&](int full, int empty, uint32_t dst, const CUtensorMap* map, int col) {
        if (c > 1 && !(ok = wait(empty + (c & 1), ((c >> 1) & 1) ^ 1))) return;  // its reader two chunks ago
        if (elect()) {
          const uint32_t b = bar(full + (c & 1));
          bar_expect(b, TILE);
          tma_load(dst, map, col, row, b);
          tma_load(dst + BOX, map, col + 64, row, b);
        }
        __syncwarp();
      };
      load(FULL_K, EMPTY_K, sk(c), &tk, hk * D);
      if (ok) load(FULL_V, EMPTY_V, sv(c), &tv, h * D);
      if (!ok) break;
#pragma unroll
      for (int j = 0; j < 4; ++j) g[j] = (g[j] < G_MIN ? G_MIN : g[j]) * LOG2E;
      float pre[4], suf[4];  // sums up to and behind each token, each from its own end: the near ones exact
      pre[0] = g[0], pre[1] = pre[0] + g[1], pre[2] = pre[1] + g[2], pre[3] = pre[2] + g[3];
      suf[3] = 0.0f, suf[2] = g[3], suf[1] = suf[2] + g[2], suf[0] = suf[1] + g[1];
      float up = pre[3], down = suf[0] + g[0];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float x = __shfl_up_sync(0xffffffffu, up, o), y = __shfl_down_sync(0xffffffffu, down, o);
        if (lane >= o) up += x;
        if (lane + o < 32) down += y;
      }
      float before = __shfl_up_sync(0xffffffffu, up, 1), behind = __shfl_down_sync(0xffffffffu, down, 1);
      if (lane == 0) before = 0.0f;
      if (lane == 31) behind = 0.0f;
      const float total = __shfl_sync(0xffffffffu, down, 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) pre[j] += before, suf[j] += behind;
      const float ref = __shfl_sync(0xffffffffu, pre[3], lane | 3);
      const unsigned prev = (c & 1) ^ 1;  // the phase of chunk c - 1, whose readers have to be done
      if (c > 0 && !(ok = wait(KP, prev))) break;
      *reinterpret_cast<float4*>(sm.W + 4 * lane) = make_float4(ex2(suf[0]), ex2(suf[1]), ex2(suf[2]), ex2(suf[3]));
      if (lane == 0) sm.total = total;
      __syncwarp();
      if (lane == 0) bar_arrive(bar(DECAY_W));
      if (!LOCAL) {
        load(FULL_Q, EMPTY_Q, sq(c), &tq, hk * D);  // (the last of the three to come free)
        if (!ok) break;
        if (c > 0 && !(ok = wait(P_IN, prev))) break;
        *reinterpret_cast<float4*>(sm.G + 4 * lane) = make_float4(pre[0], pre[1], pre[2], pre[3]);
        *reinterpret_cast<float4*>(sm.E + 4 * lane) =
            make_float4(ex2(ref - pre[0]), ex2(ref - pre[1]), ex2(ref - pre[2]), ex2(ref - pre[3]));
        __syncwarp();
        if (lane == 0) bar_arrive(bar(DECAY_G));
      }
    }
  } else {  // matrix products
    constexpr uint32_t id_kk = idesc_bf16(128, 128, false, false), id_kmn = idesc_bf16(128, 128, false, true);
    for (int c = 0; c < chunks; ++c) {
      const unsigned ph = c & 1, ph2 = (c >> 1) & 1;
      const bool want = want_last || c + 1 < chunks, from_state = resumed || c > 0;
      // K'^T's parts times V
      auto delta = [&](uint32_t keys, bool first) {
#pragma unroll
        for (int k = 0; k < 8; ++k) mma_ts(t_ds, keys + 8 * k, desc_mn(sv(c) + 2048 * k, BOX), id_kmn, !first || k > 0);
      };
      if (!LOCAL) {
        if (!(ok = wait(FULL_Q + ph, ph2) && wait(FULL_K + ph, ph2))) break;
        tc_after();
        if (elect()) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t at = (k >> 2) * BOX + 32 * (k & 3);
            mma_ss(t_sc, desc_k(sq(c) + at), desc_k(sk(c) + at), id_kk, k > 0);
          }
          mma_commit(bar(SCORES));
          mma_commit(bar(EMPTY_K + ph));
        }
        __syncwarp();
      }
      // (S_IN: the threads have read the chunk before's K'^T V, too)
      if (!(ok = wait(S_IN, ph) && (LOCAL || c == 0 || wait(O_READ, ph ^ 1)))) break;
      tc_after();
      if (!LOCAL && elect()) {
        if (from_state) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_ss(t_o, desc_k(sq(c) + (k >> 2) * BOX + 32 * (k & 3)), desc_mn(ss + 2048 * k, BOX), id_kmn, k > 0);
        }
        mma_commit(bar(FROM_S));  // (every chunk: its phases count them)
      }
      __syncwarp();
      if (!(ok = wait(KP, ph) && wait(FULL_V + ph, ph2))) break;
      tc_after();
      if (want && elect()) {
        if (LOCAL) delta(t_lo(c), true);  // smallest first
        delta(t_mid(c), !LOCAL);
        delta(t_hi(c), false);
        if (LOCAL) {
          mma_commit(bar(EMPTY_V + ph));
          mma_commit(bar(DELTA));
        } else {
          mma_commit(bar(HI_DONE));
        }
      }
      __syncwarp();
      if (!LOCAL) {
        if (!(ok = wait(P_IN, ph))) break;
        tc_after();
        if (elect()) {
          if (want) {
            if (LO) delta(t_lo(c), false);
            mma_commit(bar(DELTA));
          }
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_ts(t_o, t_p + 8 * k, desc_mn(sv(c) + 2048 * k, BOX), id_kmn, from_state || k > 0);
          mma_commit(bar(EMPTY_V + ph));
          mma_commit(bar(OUT));
        }
        __syncwarp();
      }
    }
  }
  if (!ok) {
    *dead = 1;
    if (lane == 0) atomicOr(&g_la_err, KDA_ERR_TIMEOUT);
  }
  __syncwarp();
  tc_before();
  __syncthreads();
  tc_after();
  if (*dead && warp == COMPUTE_WARPS + 1 && elect()) {
    // what is still in flight lands before the memory goes: the MMAs, then the copies nobody has
    // waited for (they take microseconds; ~10 ms)
    int never = 0;
    mma_commit(bar(DRAIN));
    bar_wait(bar(DRAIN), 0, &never);
    const long long c0 = clock64();
    while (clock64() - c0 < 20000000ll) {
    }
  }
  __syncthreads();
  if (warp == COMPUTE_WARPS + 1) tmem_free(tmem, 512);
}

// From the segments' own states to the states they start from, elementwise and in place in
// the workspace, and to the one behind the last segment, in the pool: four values a thread, JOIN_PARTS CTAs a state, the
// loads of JOIN_AHEAD segments in flight together.  Between the two passes it is all latency: small CTAs, which find
// room on every SM, 8192 x 1 head 18 -> 16 us for the whole call against 16 of 256 threads; 16 segments ahead and one load
// a lane for their decays, 8192 x 12 heads 45.5 -> 42.6 against 8 and a load a segment.
constexpr int JOIN_PARTS = 64, JOIN_AHEAD = 16, JOIN_THREADS = D * D / 4 / JOIN_PARTS;
template <bool BF>
__global__ void __launch_bounds__(JOIN_THREADS) la_join_kernel(const ChunkArgs p) {
  const LaArgs& a = p.a;
  __shared__ Segment s_seg;
  __shared__ long long s_number;
  __shared__ int s_found;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const long long task = blockIdx.x / JOIN_PARTS;
  const int h = (int)(task % a.heads), lane = threadIdx.x & 31;
  if (threadIdx.x < 32) {
    Segment s;
    long long number = 0;
    const bool found = find_part(p, task / a.heads, true, &s, &number);
    if (threadIdx.x == 0) s_seg = s, s_number = number, s_found = found;
  }
  __syncthreads();
  const int seq = s_found ? s_seg.seq : 0, slot = a.slots[seq];
  if (!s_found || slot < 0 || slot >= a.pool) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const int count = s_seg.end > s_seg.begin ? s_seg.count : 0;  // (without tokens the state is the start's)
  const int at = (int)(blockIdx.x % JOIN_PARTS) * (D * D / JOIN_PARTS) + 4 * threadIdx.x;
  const long long e = ((long long)slot * a.heads + h) * (D * D) + at;
  float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.has_state && a.has_state[seq]) {
    if (BF) {
      const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a.state) + e);
      S = make_float4(bf_lo(u.x), bf_hi(u.x), bf_lo(u.y), bf_hi(u.y));
    } else {
      S = *reinterpret_cast<const float4*>(static_cast<const float*>(a.state) + e);
    }
  }
  const long long step = (long long)a.heads * (D * D / 4);
  float4* w = reinterpret_cast<float4*>(p.ws + (s_number * a.heads + h) * (D * D) + at);
  const float* decays = p.decays + s_number * a.heads + h;
  // the segments' states are the kernel before's
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int s0 = 0; s0 < count; s0 += JOIN_AHEAD, w += JOIN_AHEAD * step, decays += (long long)JOIN_AHEAD * a.heads) {
    float4 own[JOIN_AHEAD];
#pragma unroll
    for (int i = 0; i < JOIN_AHEAD; ++i) {
      if (s0 + i >= count) break;
      own[i] = __ldcg(w + i * step);
    }
    // a segment's decay a lane
    const float mine = ex2(lane < JOIN_AHEAD && s0 + lane < count ? __ldcg(decays + (long long)lane * a.heads) : 0.0f);
#pragma unroll
    for (int i = 0; i < JOIN_AHEAD; ++i) {
      if (s0 + i >= count) break;
      w[i * step] = S;
      const float d = __shfl_sync(0xffffffffu, mine, i);
      S = make_float4(fmaf(d, S.x, own[i].x), fmaf(d, S.y, own[i].y), fmaf(d, S.z, own[i].z), fmaf(d, S.w, own[i].w));
    }
  }
  if (BF)
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.state) + e) = make_uint2(pack_bf(S.x, S.y), pack_bf(S.z, S.w));
  else
    *reinterpret_cast<float4*>(static_cast<float*>(a.state) + e) = S;
}

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
  return ptr_aligned(q, 16) && ptr_aligned(k, 16) && ptr_aligned(v, 16) && ptr_aligned(out, 16) && ptr_aligned(state, 16) &&
         ptr_aligned(g, 4) && ptr_aligned(slots, 4);
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
  return launch(state_dtype == KDA_STATE_BF16 ? la_step_kernel<true> : la_step_kernel<false>, rows * heads * STEP_SPLIT,
                32 * STEP_WARPS, 0, 1, static_cast<cudaStream_t>(cuda_stream), a);
}

namespace {

// How a prompt call is cut.
struct Cut {
  int m;                     // chunks a segment
  int least;                 // ChunkArgs::least
  long long splits, parts;   // split sequences and their segments, at most
};

// Time model in us (fitted to 20 shapes, 37 to 32704 rows of 1 to 96 heads, 1 to 1024 sequences of like and of very unlike
// lengths, each at up to 14 values of m; its pick takes 1 % longer than the best m on average): a chunk and a CTA's
// start without a split; with one a chunk in both passes, the three kernels' start, another wave, a segment's states through the
// join, and the launch for the sequences that are not split, which fill the SMs that the parts leave.
constexpr double T_CHUNK = 3.2, T_START = 6.8, T_CHUNK2 = 4.08, T_START2 = 8.8, T_WAVE2 = 3.8, T_JOIN2 = 0.066,
                 T_WHOLE2 = 8.5;

Cut la_cut(long long rows, int heads, long long seqs, long long max_len, int sms) {
  const long long bound = max_len < rows ? max_len : rows;
  long long longest = (bound + CHUNK - 1) / CHUNK;  // chunks
  if (longest < 1) longest = 1;
  const double per_sm = (double)heads / sms;
  auto waves_of = [&](double tasks) {
    const double w = tasks * per_sm;
    return w <= 1.0 ? 1.0 : (double)(long long)(w + 0.999);
  };
  // `n` sequences of `tokens` together that are not split, half of a chunk of each empty: a CTA each and head
  auto whole = [&](double n, double tokens) {
    return waves_of(n) * ((tokens / CHUNK / n + 0.5) * T_CHUNK + T_START);
  };
  Cut best = {};
  double least = 1e300;
  for (long long m = 1;; m = m < 8 ? m + 1 : m + m / 8) {
    const bool last = m >= longest;
    if (last) m = longest;
    double t;
    if (last) {
      const double chain = (double)m * T_CHUNK + T_START, all = whole((double)seqs, (double)rows);
      t = chain > all ? chain : all;
    } else {
      // the lengths are not known here: all alike if that makes them longer than a segment, else one of the longest
      const bool alike = (double)rows > (double)seqs * (double)m * CHUNK;
      const double n = alike ? (double)seqs : 1.0, tokens = (double)(alike ? rows : bound);
      const double chunks = tokens / CHUNK + 0.5 * n, segs = tokens / CHUNK / (double)m + 0.5 * n;
      const double waves = waves_of(segs), per = chunks / segs < (double)m ? chunks / segs : (double)m;
      const double run = (per * waves > (double)m ? per * waves : (double)m) * T_CHUNK2;
      t = run + T_START2 + (waves - 1.0) * T_WAVE2 + segs * heads * T_JOIN2;
      if (seqs > 1) t += T_WHOLE2;
      if ((double)seqs > n) {
        const double left = 1.0 - segs * per_sm;
        const double rest = whole((double)seqs - n, (double)rows - tokens) - (left > 0.0 ? left : 0.0) * run;
        if (rest > 0.0) t += rest;
      }
    }
    if (t < least * 0.999) {
      least = t;
      best.m = (int)(m > 0x1000000 ? 0x1000000 : m);
      best.least = last ? 0 : seqs > 1 ? 2 : 1;
    }
    if (last) break;
  }
  const long long per = (long long)best.m * CHUNK;
  if (best.least > 0) {  // (with 2 a split sequence is longer than `per`)
    best.splits = rows / per < seqs ? rows / per : seqs;
    best.parts = rows / per + best.splits;
  }
  return best;
}

bool la_sizes_ok(long long rows, int heads, long long seqs, long long max_len) {
  return rows >= 0 && rows <= 0x7fffffffLL && heads >= 1 && heads <= 65535 && seqs >= 0 && seqs <= 0x7fffffffLL &&
         max_len >= 0;
}

template <bool BF>
int la_prefill_launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& to,
                      const ChunkArgs& p, const Cut& cut, cudaStream_t st) {
  // the shared-memory attribute is per device and cheap: set on every call
  auto chunks = [&](auto* kernel, long long segments) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, CHUNK_SMEM) != cudaSuccess)
      return KDA_ECUDA;
    return launch(kernel, segments * p.a.heads, CHUNK_THREADS, CHUNK_SMEM, 1, st, tq, tk, tv, to, p);
  };
  if (cut.least == 0) return chunks(la_chunk_kernel<DIRECT, BF>, p.a.seqs);
  int rc = chunks(la_chunk_kernel<OWN, false>, cut.parts);
  if (rc == KDA_OK) rc = launch(la_join_kernel<BF>, cut.splits * p.a.heads * JOIN_PARTS, JOIN_THREADS, 0, 1, st, p);
  if (rc == KDA_OK) rc = chunks(la_chunk_kernel<OUTPUT, false>, cut.parts);
  return rc == KDA_OK && cut.least == 2 ? chunks(la_chunk_kernel<DIRECT, BF>, p.a.seqs) : rc;
}

}  // namespace

extern "C" long long kda_la_prefill_workspace(long long rows, int heads, long long seqs, long long max_len) {
  if (!la_sizes_ok(rows, heads, seqs, max_len) || seqs == 0) return 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  const int sms = sm_count(dev);
  if (sms <= 0) return 0;
  const Cut cut = la_cut(rows, heads, seqs, max_len, sms);
  if (cut.least == 0) return 0;
  return (cut.parts * heads * (D * D + 1) * 4 + 15) / 16 * 16;
}

extern "C" int kda_la_prefill(const void* q, long long ldq, const void* k, long long ldk, const void* v,
                              long long ldv, long long rows, int heads, int qk_heads, const float* g, long long ldg,
                              float scale, const int* cu_seqlens, long long seqs, long long max_len,
                              const int* has_state, void* state_pool, int state_dtype, long long pool_slots,
                              const int* slots, void* out, long long ldo, void* workspace, long long workspace_bytes,
                              void* cuda_stream) {
  if (!la_sizes_ok(rows, heads, seqs, max_len)) return KDA_EINVAL;
  if (seqs == 0) return KDA_OK;
  if (!la_args_ok(rows, q, ldq, k, ldk, v, ldv, heads, qk_heads, g, ldg, state_pool, state_dtype, pool_slots, slots,
                  out, ldo) ||
      !cu_seqlens || !ptr_aligned(cu_seqlens, 4) || !ptr_aligned(has_state, 4))
    return KDA_EINVAL;
  if ((rows / CHUNK + seqs) > 0x7fffffffLL / heads) return KDA_EINVAL;  // the largest grid: a CTA a segment and head
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KDA_ECUDA;
  const int sms = sm_count(dev);
  if (sms <= 0) return KDA_ECUDA;
  const Cut cut = la_cut(rows, heads, seqs, max_len, sms);
  if (cut.splits > 0x7fffffffLL / JOIN_PARTS / heads) return KDA_EINVAL;
  const long long need = cut.least > 0 ? (cut.parts * heads * (D * D + 1) * 4 + 15) / 16 * 16 : 0;
  if (need > 0 && (!workspace || workspace_bytes < need || !ptr_aligned(workspace, 16))) return KDA_EINVAL;
  CUtensorMap tq = {}, tk = {}, tv = {}, to = {};
  if (rows > 0) {
    if (!on_device(q, dev) || !on_device(k, dev) || !on_device(v, dev) || !on_device(out, dev)) return KDA_EINVAL;
    const CUtensorMapDataType t = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const CUtensorMapSwizzle s = CU_TENSOR_MAP_SWIZZLE_128B;
    if (!encode_2d(&tq, t, q, rows, (long long)qk_heads * D, ldq * 2, 64, CHUNK, s) ||
        !encode_2d(&tk, t, k, rows, (long long)qk_heads * D, ldk * 2, 64, CHUNK, s) ||
        !encode_2d(&tv, t, v, rows, (long long)heads * D, ldv * 2, 64, CHUNK, s) ||
        !encode_2d(&to, t, out, rows, (long long)heads * D, ldo * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B))
      return KDA_ECUDA;
  }
  ChunkArgs p;
  p.a = la_args(q, ldq, k, ldk, v, ldv, rows, heads, qk_heads, g, ldg, scale, state_pool, pool_slots, slots, out, ldo);
  p.a.cu = cu_seqlens, p.a.has_state = has_state, p.a.seqs = seqs, p.a.max_len = max_len;
  p.ws = static_cast<float*>(workspace);
  p.decays = p.ws + cut.parts * heads * (D * D);
  p.m = cut.m;
  p.least = cut.least, p.parts = cut.parts;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  return state_dtype == KDA_STATE_BF16 ? la_prefill_launch<true>(tq, tk, tv, to, p, cut, st)
                                       : la_prefill_launch<false>(tq, tk, tv, to, p, cut, st);
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

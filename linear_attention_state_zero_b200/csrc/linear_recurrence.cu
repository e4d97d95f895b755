// linear_recurrence.cu -- the gated linear recurrence per channel, over packed sequences:
//
//   forward   h_t = a_t h_{t-1} + x_t,                  y_t = h_t
//   backward  u_t = a_t (dy_t + u_{t+1})                (u behind a sequence's last token: dh_final)
//             dx_t = dy_t + u_{t+1},  d(log a_t) = u_t h_{t-1},  dh0 = u at the first token
//
// with a = exp(gate) or a = exp(-softplus(gate)) = 1 / (1 + e^gate) (then d(gate) =
// -(1 - a) d(log a)).  Both are one scan of maps u -> A u + B, in time and against it.
//
// One pass over HBM: a cluster of up to 8 CTAs owns a tile of channels and walks the tokens;
// in a round each warp (or each of G groups of its lanes) holds a segment of consecutive tokens
// of its lanes' channels in registers (the next rounds' loads already in flight), reduces it to
// one map (A, B) per channel, and the segments are joined in time order: those of a CTA through
// shared memory, the CTAs of the cluster through each other's shared memory (stores that count
// their bytes on the receiver's mbarrier; a cluster barrier in each round, whose release waits
// for the loads and stores in flight, took half as long again).  Every lane then knows the state
// in front of its segment and replays the segment from registers.  Nothing is read twice, nothing
// passes through global memory, and the order of every sum is fixed, so results are bitwise
// reproducible.
//
// HBM bounds it where the runs of sequences fill the GPU: 65536 x 4096 bf16 in 64 sequences takes
// 252 us with exponential gates and 264-270 with logits (98% and 91-93% of the measured copy rate;
// up to 307 us on another GPU), backward 453 and 480 (90% and 85%: segments of 4 tokens, a join
// for every 64), backward 16384 x 4096 fp32 in 40 sequences 213 us (96%).  One long sequence is
// bound by the join of its cluster each round (65536 x 1024 bf16: 153-163 us, 40%; backward
// 32768 x 2048, bf16 with fp32 gates: 235 us, 61%), a few thousand tokens by the latency of a few
// rounds of about 2 us, and rows that are not 4-byte (bf16) or 8-byte (fp32) aligned by one channel
// a lane (35-70%).
//
// The packed tokens are scanned as one long sequence that starts over where a sequence
// begins.  That is a selection, not a product with a = 0, so infinities or NaN of one
// sequence never reach the next.  All states, products and sums are fp32; outputs are rounded
// once.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstddef>

#include "fp8_ptx.cuh"
#include "layer_ops.h"
#include "tr_internal.h"

namespace tr {
namespace {

constexpr int kW = 8;             // warps of a CTA
constexpr int kMaxParts = 64;     // independent runs of whole sequences (grid.y)
constexpr int kMaxCluster = 8;

struct Parts {
  int32_t lo[kMaxParts], hi[kMaxParts];           // tokens of each run, the longest first
  int32_t seq_lo[kMaxParts], seq_hi[kMaxParts];   // its sequences: cu[seq_lo] = lo, cu[seq_hi] = hi
  int some_empty;                                 // some sequence has no token
};

template <int V> struct alignas(4 * V) Floats { float f[V]; };

// V channels of one token as loaded
template <typename T, int V> struct Raw;
template <> struct Raw<__nv_bfloat16, 1> { unsigned short u; };
template <> struct Raw<__nv_bfloat16, 2> { uint32_t u[1]; };
template <> struct alignas(8) Raw<__nv_bfloat16, 4> { uint32_t u[2]; };
template <int V> struct Raw<float, V> : Floats<V> {};

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> ld_raw(const T *p) {
  return *reinterpret_cast<const Raw<T, V> *>(p);
}
__device__ __forceinline__ void to_f32(const Raw<__nv_bfloat16, 1> &r, float (&f)[1]) {
  f[0] = __uint_as_float((uint32_t)r.u << 16);
}
template <int V>
__device__ __forceinline__ void to_f32(const Raw<__nv_bfloat16, V> &r, float (&f)[V]) {
#pragma unroll
  for (int v = 0; v < V; v += 2) {
    f[v] = __uint_as_float(r.u[v / 2] << 16);
    f[v + 1] = __uint_as_float(r.u[v / 2] & 0xffff0000u);
  }
}
template <int V>
__device__ __forceinline__ void to_f32(const Raw<float, V> &r, float (&f)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) f[v] = r.f[v];
}
__device__ __forceinline__ void st_f32(__nv_bfloat16 *p, const float (&f)[1]) { *p = __float2bfloat16_rn(f[0]); }
template <int V>
__device__ __forceinline__ void st_f32(__nv_bfloat16 *p, const float (&f)[V]) {
  Raw<__nv_bfloat16, V> r;
#pragma unroll
  for (int v = 0; v < V; v += 2) r.u[v / 2] = pack_bf16x2(f[v], f[v + 1]);
  *reinterpret_cast<Raw<__nv_bfloat16, V> *>(p) = r;
}
template <int V>
__device__ __forceinline__ void st_f32(float *p, const float (&f)[V]) {
  Floats<V> r;
#pragma unroll
  for (int v = 0; v < V; ++v) r.f[v] = f[v];
  *reinterpret_cast<Floats<V> *>(p) = r;
}

// d = a b + c, a b and a + b of V channels, two to an instruction (each rounds as the scalar one).
template <int V>
__device__ __forceinline__ void vfma(float (&d)[V], const float (&a)[V], const float (&b)[V], const float (&c)[V]) {
  if constexpr (V == 1) {
    d[0] = fmaf(a[0], b[0], c[0]);
  } else {
#pragma unroll
    for (int v = 0; v < V; v += 2) {
      const uint64_t r = fma_f32x2(pair_f32(a[v], a[v + 1]), pair_f32(b[v], b[v + 1]), pair_f32(c[v], c[v + 1]));
      split_f32(r, d[v], d[v + 1]);
    }
  }
}
template <int V>
__device__ __forceinline__ void vmul(float (&d)[V], const float (&a)[V], const float (&b)[V]) {
  if constexpr (V == 1) {
    d[0] = a[0] * b[0];
  } else {
#pragma unroll
    for (int v = 0; v < V; v += 2) {
      const uint64_t r = mul_f32x2(pair_f32(a[v], a[v + 1]), pair_f32(b[v], b[v + 1]));
      split_f32(r, d[v], d[v + 1]);
    }
  }
}
template <int V>
__device__ __forceinline__ void vadd(float (&d)[V], const float (&a)[V], const float (&b)[V]) {
  if constexpr (V == 1) {
    d[0] = a[0] + b[0];
  } else {
#pragma unroll
    for (int v = 0; v < V; v += 2) {
      uint64_t r;
      asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair_f32(a[v], a[v + 1])), "l"(pair_f32(b[v], b[v + 1])));
      split_f32(r, d[v], d[v + 1]);
    }
  }
}

__device__ __forceinline__ float ex2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_ftz(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float min_nan(float a, float b) {   // (a NaN stays)
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// a by ex2 and rcp (approximate, 2^-22 each) of a rounded argument: off by at most 2^-22 + 2^-23 |gate|
// of itself (2^-21 + 2^-23 |gate| for a logit; measured next to a = 1: 1.4 x 2^-24, as expf).  e^gate
// may be infinite: a is 0 then, as where it is below 2^-126.  GRAD: also q = h d(log a) / d(gate),
// with d(log a) / d(gate) = 1, or -(1 - a) = -a e^gate for a logit, e^gate held finite there (a is 0
// before it is not, and so is the product).
// Without LOGITS, l += log2 a.
template <bool LOGITS, bool GRAD, int V>
__device__ __forceinline__ void decay(float (&g)[V], float (&a)[V], const float (&h)[V], float (&q)[V], float (&l)[V]) {
  float e[V], one[V], log2e[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    one[v] = 1.f;
    log2e[v] = 1.4426950408889634f;
  }
  vmul(e, g, log2e);
  if (!LOGITS) vadd(l, l, e);
#pragma unroll
  for (int v = 0; v < V; ++v) e[v] = ex2_ftz(e[v]);
  if (!LOGITS) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      a[v] = e[v];
      if (GRAD) q[v] = h[v];
    }
    return;
  }
  vadd(a, e, one);
#pragma unroll
  for (int v = 0; v < V; ++v) a[v] = rcp_ftz(a[v]);
  if (GRAD) {
#pragma unroll
    for (int v = 0; v < V; ++v) e[v] = min_nan(e[v], 3.4028235e38f);
    vmul(e, e, a);
#pragma unroll
    for (int v = 0; v < V; ++v) e[v] = -e[v];
    vmul(q, e, h);
  }
}
template <bool LOGITS, int V>
__device__ __forceinline__ void decay(float (&g)[V], float (&a)[V], float (&l)[V]) {
  float none[V] = {};
  decay<LOGITS, false>(g, a, none, none, l);
}

// The decays of a map u -> A u + B.  exp(gate) may be above 1, and their product then leave fp32's
// range, on the way or at its end, where the values that it is for do not: a zero in front would
// become inf * 0, a tiny value infinite, one that shrinks and grows again 0.  So without LOGITS a map
// keeps F = sqrt(A), from the sum of its decays' logarithms.  Its ends are those of A = 2^254, which
// takes the least normal fp32 past the largest, and of 2^-252, which takes the largest below 2^-124.
// With LOGITS (a <= 1) it keeps A itself.  (Backward 32768 x 2048: 237 us with products of such
// decays too, 236 with F; 285 with A as a logarithm that the joining threads apply in three factors.)
template <bool LOGITS>
struct Decays {
  // a segment's, from the product or the sum of log2 a
  static __device__ __forceinline__ float of(float p) {
    if (LOGITS) return p;
    return ex2_ftz(min_nan(0.5f * p, 127.f));
  }
  static __device__ __forceinline__ float both(float a, float b) {
    return LOGITS ? a * b : min_nan(a * b, 3.4028235e38f);
  }
  static __device__ __forceinline__ float apply(float A, float v, float B) {
    return LOGITS ? fmaf(A, v, B) : fmaf(A * v, A, B);
  }
};

// What a thread reads of one operand, V channels of LS tokens a round, a few rounds ahead: a ring
// in shared memory that the thread alone fills and reads, by asynchronous copies, so that it
// waits for nothing but its own copies, and the data in flight take no registers (but for one
// channel of two bytes, see there).
template <typename T, int V, int LS>
struct Slots {
  static constexpr int TOKEN = kW * 32 * V * (int)sizeof(T);   // of a CTA
  static constexpr int BYTES = LS * TOKEN;                     // a stage
  uint8_t *mine;                                               // this thread's slot of token 0
  __device__ explicit Slots(uint8_t *smem) : mine(smem + threadIdx.x * V * sizeof(T)) {}
  __device__ __forceinline__ Raw<T, V> *at(int stage, int i) const {
    return reinterpret_cast<Raw<T, V> *>(mine + stage * BYTES + i * TOKEN);
  }
  __device__ __forceinline__ Raw<T, V> get(int stage, int i) const { return *at(stage, i); }
};
template <typename T, int V, int LS>
struct Ring : Slots<T, V, LS> {
  using Slots<T, V, LS>::Slots;
  // tokens p, p + step, ... of which the first `left` exist (the others read as 0)
  __device__ __forceinline__ void issue(int stage, const T *p, int64_t step, int left) {
    const uint32_t dst = smem_u32(this->at(stage, 0));
    if (left >= LS) {
#pragma unroll
      for (int i = 0; i < LS; ++i) copy(dst + i * this->TOKEN, p + i * step);
    } else {
#pragma unroll
      for (int i = 0; i < LS; ++i)
        if (i < left) copy(dst + i * this->TOKEN, p + i * step);
        else *this->at(stage, i) = Raw<T, V>{};
    }
  }
  static __device__ __forceinline__ void copy(uint32_t dst, const T *p) {
    if constexpr (V * sizeof(T) == 16) {   // (past the L1 cache, which smaller copies go through)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(p) : "memory");
    } else {
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(p), "n"(V * (int)sizeof(T)) : "memory");
    }
  }
};
// Two bytes are too few for an asynchronous copy: the loads of a stage wait in registers until
// the next stage is issued, so that one stage is in flight at a time whatever the ring holds.
template <int LS>
struct Ring<__nv_bfloat16, 1, LS> : Slots<__nv_bfloat16, 1, LS> {
  Raw<__nv_bfloat16, 1> next[LS];
  int held = -1;
  using Slots<__nv_bfloat16, 1, LS>::Slots;
  __device__ __forceinline__ void issue(int stage, const __nv_bfloat16 *p, int64_t step, int left) {
    if (held >= 0) {
#pragma unroll
      for (int i = 0; i < LS; ++i) *this->at(held, i) = next[i];
    }
    held = stage;
#pragma unroll
    for (int i = 0; i < LS; ++i)
      next[i] = i < left ? ld_raw<__nv_bfloat16, 1>(p + i * step) : Raw<__nv_bfloat16, 1>{};
  }
};
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Rounds in the rings (the one in hand among them), for stages of `bytes`.  Two CTAs run on an
// SM, and copies of less than 16 bytes need the L1 cache while they are in flight: with rings
// of 96 KB instead of 64 the forward pass over 65536 x 4096 took 360 us instead of 262.
constexpr int stages_of(int bytes) { return 65536 / bytes > 4 ? 4 : 65536 / bytes < 2 ? 2 : 65536 / bytes; }

// The maps u -> A u + B of a round's segments, per channel, and the values in front of them.
// `start`: a sequence begins inside a segment, so u does not count.  The CTAs' maps of a cluster
// are two sets, used in turn: a CTA sends those of a round only after it has those of the round
// before from every CTA, each of which sent them when it had read the set in use now.
template <int V, int G>
struct Shared {
  static constexpr int C = 32 / G * V, SEGS = kW * G;
  float A[SEGS][C], B[SEGS][C];    // (the value in front of a segment then takes its A's place)
  float start[SEGS];
  uint64_t bar[2];                 // every CTA's maps of a set are here
  int abort;                       // a wait ran out
  int gave_up;                     // the last round that bar was armed for, then
  struct Cta {                     // (not allocated without a cluster)
    float A[C], B[C];
    float start;
  } cta[2][kMaxCluster];
};
template <int V, int G>
size_t shared_bytes(int S) {
  typedef Shared<V, G> Sh;
  return S > 1 ? sizeof(Sh) : offsetof(Sh, cta);
}

// What a CTA starts with; with a cluster, every CTA's barriers are ready before any sends to it.
template <int V, int G>
__device__ __forceinline__ void begin(Shared<V, G> &sh, uint32_t S, bool hold_back) {
  if (S == 1) return;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&sh.bar[0]), 1);
    mbar_init(smem_u32(&sh.bar[1]), 1);
    sh.abort = hold_back;   // (as if it had given up in front of the first round)
    sh.gave_up = -1;
    fence_mbar_init();
  }
  __syncwarp();
  cluster_sync_all();
}

// Arms the set of maps of round `round`: every CTA's bytes are to come.
template <int V, int G>
__device__ __forceinline__ uint32_t expect_maps(Shared<V, G> &sh, int round, uint32_t S) {
  const uint32_t bar = smem_u32(&sh.bar[round & 1]);
  mbar_arrive_expect_tx(bar, S * (8 * Shared<V, G>::C + 4));
  return bar;
}
__device__ __forceinline__ uint32_t parity_of(int round) { return (uint32_t)(round >> 1) & 1u; }

// No CTA of a cluster leaves before all have sent what they send.  One that gave up then lets arrive
// what may be on its way to it: the maps of the round that it gave up in, and those of CTAs that got
// through that round and sent the next one's (each wait bounded).
template <int V, int G>
__device__ __forceinline__ void leave(Shared<V, G> &sh, uint32_t S) {
  if (S == 1) return;
  __syncwarp();
  cluster_sync_all();
  if (threadIdx.x != 0 || !sh.abort) return;
  const int round = sh.gave_up;
  if (round >= 0) mbar_wait_drain(smem_u32(&sh.bar[round & 1]), parity_of(round));
  mbar_wait_drain(expect_maps(sh, round + 1, S), parity_of(round + 1));
}

// The sequence that holds token t0 (the last with cu <= t0: seq, its tokens from .. to - 1), and
// where sequences begin in the tokens [t0, t0 + n], n < 31: bit i for a cu entry equal to t0 + i
// (cu[N] = T among them).  lookup_up starts from a sequence `seq` that begins at or before t0,
// lookup_down from an entry `top` that is past t0 + n or the last such (and cu[low] <= t0).  The
// whole warp calls them with the same arguments; one load of 32 entries is the rule.  (Offsets on
// the device that are not the host's give a wrong result, but neither a walk without end nor a
// sequence that does not exist.)
__device__ __forceinline__ uint32_t bits_of(int v, int t0, int n) {
  return v >= t0 && v - t0 <= n ? 1u << (v - t0) : 0u;
}
__device__ __forceinline__ uint32_t lookup_up(const int32_t *__restrict__ cu, int n_seqs, int t0, int n, int &seq,
                                              int &from, int &to) {
  const int lane = threadIdx.x & 31;
  int at = seq, v;
  uint32_t le;
  for (;; at += 31) {
    v = __ldg(cu + (at + lane < n_seqs ? at + lane : n_seqs));
    le = __ballot_sync(0xffffffffu, v <= t0);   // lanes 0 .. k
    if (le != 0xffffffffu || at >= n_seqs) break;
  }
  const int k = min(max(__popc(le) - 1, 0), 30);
  seq = min(at + k, n_seqs - 1);
  from = __shfl_sync(0xffffffffu, v, k);
  to = __shfl_sync(0xffffffffu, v, k + 1);
  uint32_t m = bits_of(v, t0, n);
  while (__shfl_sync(0xffffffffu, v, 31) <= t0 + n && at + 31 < n_seqs) {
    at += 31;
    v = __ldg(cu + (at + lane < n_seqs ? at + lane : n_seqs));
    m |= bits_of(v, t0, n);
  }
  return __reduce_or_sync(0xffffffffu, m);
}
__device__ __forceinline__ uint32_t lookup_down(const int32_t *__restrict__ cu, int low, int top, int t0, int n,
                                                int &seq, int &from, int &to) {
  const int lane = threadIdx.x & 31;
  uint32_t m = 0;
  for (;;) {
    const int at = top - 31 > low ? top - 31 : low;
    const int v = __ldg(cu + (at + lane < top ? at + lane : top));
    m |= bits_of(v, t0, n);
    const uint32_t le = __ballot_sync(0xffffffffu, v <= t0);
    if (le || at <= low) {
      const int k = min(max(__popc(le) - 1, 0), 30);
      seq = min(at + k, max(top - 1, low));
      from = __shfl_sync(0xffffffffu, v, k);
      to = __shfl_sync(0xffffffffu, v, k + 1);
      return __reduce_or_sync(0xffffffffu, m);
    }
    top = at;
  }
}

// Joins the maps of a round.  In: the map of this lane's segment.  Out: the value in front of
// it (A: the product of its decays, or without LOGITS the sum of their logarithms to base 2).  The
// first 32 V / G threads own a channel each: they walk the segments' maps, and keep the
// value in front of the round (`carry`) for the next.  (Every warp walking the maps before its
// own for its own channels took a fifth of the kernel's instructions.)
// A thread whose wait for the other CTAs gave up arms no barrier again, sends nothing (`sends`) and
// waits no more: the rounds go on with undefined values to their end, where leave() meets the other
// CTAs.  (Leaving the rounds took a test in each, 1-3% of a call's time.)
template <bool LOGITS, int V, int G>
__device__ __forceinline__ void join(Shared<V, G> &sh, int round, uint32_t S, uint32_t r, uint32_t &sends,
                                     const Waits &waits, int seg, int li, const float (&A)[V], const float (&B)[V],
                                     bool start, float &carry, float (&u)[V]) {
  typedef Shared<V, G> Sh;
  __syncwarp();
  float of[V];
#pragma unroll
  for (int v = 0; v < V; ++v) of[v] = Decays<LOGITS>::of(A[v]);
  st_f32(&sh.A[seg][li * V], of);
  st_f32(&sh.B[seg][li * V], B);
  if (li == 0) sh.start[seg] = start ? 1.f : 0.f;
  const bool any = __syncthreads_or(start);
  if (threadIdx.x < Sh::C) {
    const int ch = threadIdx.x;
    // u after a segment: one that a sequence begins in forgets what came before
    auto after = [&](int w, float v) {
      return any && sh.start[w] != 0.f ? sh.B[w][ch] : Decays<LOGITS>::apply(sh.A[w][ch], v, sh.B[w][ch]);
    };
    float v = carry;
    if (S > 1) {
      float ta = 1.f, tb = 0.f;
      bool ts = false;
#pragma unroll
      for (int w = 0; w < Sh::SEGS; ++w) {
        tb = after(w, tb);
        ta = Decays<LOGITS>::both(ta, sh.A[w][ch]);
        ts = ts || (any && sh.start[w] != 0.f);
      }
      const int par = round & 1;
      const uint32_t bar = smem_u32(&sh.bar[par]);
      if (threadIdx.x == 0 && sends) expect_maps(sh, round, S);
      typename Sh::Cta &to = sh.cta[par][r];
      const uint32_t here = smem_u32(&to.A[ch]);
      for (uint32_t k = 0; k < sends; ++k) {
        const uint32_t there = cluster_map(bar, k), dst = cluster_map(here, k);
        st_async(dst, ta, there);
        st_async(dst + 4 * Sh::C, tb, there);
        if (threadIdx.x == 0) st_async(dst + 8 * Sh::C, ts ? 1.f : 0.f, there);
      }
      const AbortFlag ab{&sh.abort, waits.err_word, ERRBIT_SCAN_TIMEOUT, waits.limit_ns};
      if (sends && !mbar_wait(bar, parity_of(round), ab)) {
        if (threadIdx.x == 0) sh.gave_up = round;
        sends = 0;
      }
      float mine = 0.f;
#pragma unroll
      for (uint32_t k = 0; k < kMaxCluster; ++k) {
        if (k >= S) break;
        const typename Sh::Cta &m = sh.cta[par][k];
        if (k == r) mine = v;
        v = m.start != 0.f ? m.B[ch] : Decays<LOGITS>::apply(m.A[ch], v, m.B[ch]);
      }
      carry = v;
      v = mine;
    }
#pragma unroll
    for (int w = 0; w < Sh::SEGS; ++w) {
      const float u_w = v;
      v = after(w, v);
      sh.A[w][ch] = u_w;
    }
    if (S == 1) carry = v;
  }
  __syncthreads();
  to_f32(ld_raw<float, V>(&sh.A[seg][li * V]), u);
}

// Group g's value of a variable of the whole warp's groups (G = 1: the warp's).
template <int G>
__device__ __forceinline__ int of_group(int v, int g) {
  return G == 1 ? v : __shfl_sync(0xffffffffu, v, g * (32 / G));
}
template <int G>
__device__ __forceinline__ bool all_of(bool b) {
  return G == 1 ? b : __all_sync(0xffffffffu, b);
}

// V channels of a state (4-byte aligned)
template <int V>
__device__ __forceinline__ Raw<float, V> ld_state(const float *p) {
  Raw<float, V> r;
#pragma unroll
  for (int v = 0; v < V; ++v) r.f[v] = p[v];
  return r;
}

// Sequences without a token keep their state: to[n] = from[n] (or 0), spread over the warps
// that own the channels.
template <int V>
__device__ __forceinline__ void copy_empty(const int32_t *__restrict__ cu, int n_seqs, int worker,
                                           int workers, int c, bool live, int C, const float *from, float *to) {
  for (int n = worker; n < n_seqs; n += workers) {
    if (__ldg(cu + n) != __ldg(cu + n + 1) || !live) continue;
#pragma unroll
    for (int v = 0; v < V; ++v)
      to[(int64_t)n * C + c + v] = from ? from[(int64_t)n * C + c + v] : 0.f;
  }
}

template <typename TX, typename TG, bool LOGITS, int V, int LS, int G>
__global__ void __launch_bounds__(kW * 32, 2) recurrence_kernel(RecurrenceLaunch p, Parts parts) {
  using RX = Ring<TX, V, LS>;
  using RG = Ring<TG, V, LS>;
  constexpr int STAGES = stages_of(RX::BYTES + RG::BYTES);
  extern __shared__ __align__(16) uint8_t smem[];
  RX rx(smem);
  RG rg(smem + STAGES * RX::BYTES);
  Shared<V, G> &sh = *reinterpret_cast<Shared<V, G> *>(smem + STAGES * (RX::BYTES + RG::BYTES));
  // (from lane 0: the compiler then keeps token indices and row pointers in uniform registers)
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t S = cluster_size(), r = cluster_rank();
  constexpr int LPG = 32 / G, SEGS = kW * G;
  const int grp = G == 1 ? 0 : lane / LPG, li = lane % LPG, seg = warp * G + grp;
  const int c = ((int)(blockIdx.x / S) * LPG + li) * V;
  const bool live = c < p.C;
  const int tb = parts.lo[blockIdx.y], te = parts.hi[blockIdx.y];
  const int chunk = (int)S * SEGS * LS;
  pdl_trigger();
  uint32_t sends = p.waits.hold_back && r + 1 == S ? 0 : S;   // CTAs that this thread sends its maps to
  begin(sh, S, sends == 0);
  pdl_wait();
  // lanes past the last channel load the last ones and store nothing
  const int cl = live ? c : p.C - V;
  const bool put_y = live && p.y;
  int t0 = tb + ((int)r * SEGS + seg) * LS;
  const TX *px = reinterpret_cast<const TX *>(p.x) + (int64_t)t0 * p.x_stride + cl;
  const TG *pg = reinterpret_cast<const TG *>(p.gate) + (int64_t)t0 * p.gate_stride + cl;
  TX *py = reinterpret_cast<TX *>(p.y) + (int64_t)t0 * p.y_stride + cl;
  int ahead = te - t0;   // tokens from the next segment to fetch to the run's end
  auto fetch = [&](int stage) {
    rx.issue(stage, px, p.x_stride, ahead);
    rg.issue(stage, pg, p.gate_stride, ahead);
    cp_commit();
    px += chunk * p.x_stride;
    pg += chunk * p.gate_stride;
    ahead -= chunk;
  };
  float carry = 0.f;
  int round = 0, stage = 0;
  int seq = parts.seq_lo[blockIdx.y], from = te, to = 0;   // the sequence looked up last: its tokens
#pragma unroll 1
  for (int i = 0; i < STAGES - 1; ++i) fetch(i);
  if (parts.some_empty)
    copy_empty<V>(p.cu, p.n_seqs, (int)((blockIdx.y * S + r) * SEGS) + seg, (int)(gridDim.y * S * SEGS), c,
                  live, p.C, p.h0, p.h_final);
#pragma unroll 1
  for (int tr0 = tb; tr0 < te; tr0 += chunk, t0 += chunk, py += chunk * p.y_stride, ++round) {
    const int lim = te - t0 < LS ? te - t0 : LS;    // tokens of the segment (may be <= 0)
    uint32_t mask = 0;
    const bool look = lim > 0 && (t0 <= from || t0 + LS >= to);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (!of_group<G>(look, g)) continue;
      int sq = of_group<G>(seq, g), f, t;
      const uint32_t m = lookup_up(p.cu, p.n_seqs, of_group<G>(t0, g), LS, sq, f, t);
      if (grp == g) {
        mask = m;
        seq = sq;
        from = f;
        to = t;
      }
    }
    // the state that the segment's first sequence start begins from, read in front of the wait
    // for the segment's own data (the other starts' are read where they are needed)
    const uint32_t inside = mask & ((1u << (lim > 0 ? lim : 0)) - 1u);
    const int first = inside ? __ffs(inside) - 1 : lim;   // tokens of the sequence before
    auto seq_of = [&](int t) {   // the sequence that holds token t >= t0
      int n = seq;
      while (n + 1 < p.n_seqs && __ldg(p.cu + n + 1) <= t) ++n;
      return n;
    };
    int n1 = 0;
    float hb[V] = {};
    if (inside) {
      n1 = seq_of(t0 + first);
      if (p.h0 && live) to_f32(ld_state<V>(p.h0 + (int64_t)n1 * p.C + c), hb);
    }
    fetch(stage == 0 ? STAGES - 1 : stage - 1);   // into the slots of the round before
    cp_wait<STAGES - 1>();
    float a[LS][V], x[LS][V], A[V], B[V], u[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      A[v] = LOGITS ? 1.f : 0.f;
      B[v] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < LS; ++i) {   // (tokens that do not exist have gates 0)
      float g[V];
      to_f32(rg.get(stage, i), g);
      to_f32(rx.get(stage, i), x[i]);
      decay<LOGITS>(g, a[i], A);
    }
    const bool whole = lim == LS && (mask & ~(1u << LS)) == 0;   // of one sequence, begun before
    auto put = [&](int i, const float (&h)[V]) {
      if (put_y) st_f32(py + i * p.y_stride, h);
    };
    auto put_final = [&](int n, const float (&h)[V]) {
      if (!live) return;
#pragma unroll
      for (int v = 0; v < V; ++v) p.h_final[(int64_t)n * p.C + c + v] = h[v];
    };
    if (all_of<G>(whole)) {
#pragma unroll
      for (int i = 0; i < LS; ++i) {
        vfma(B, a[i], B, x[i]);
        if (LOGITS) vmul(A, A, a[i]);
      }
      join<LOGITS>(sh, round, S, r, sends, p.waits, seg, li, A, B, false, carry, u);
#pragma unroll
      for (int i = 0; i < LS; ++i) {
        vfma(u, a[i], u, x[i]);
        put(i, u);
      }
      if (mask >> LS) put_final(seq, u);
    } else {
      // from the first sequence start on, the states do not depend on what lies before the
      // segment: they are final here
      int n = n1;
#pragma unroll
      for (int i = 0; i < LS; ++i) {
        if (i >= lim) continue;
        if (mask >> i & 1u) {
          if (i != first) {
            n = seq_of(t0 + i);
            if (p.h0 && live) to_f32(ld_state<V>(p.h0 + (int64_t)n * p.C + c), hb);
          }
#pragma unroll
          for (int v = 0; v < V; ++v) B[v] = p.h0 ? fmaf(a[i][v], hb[v], x[i][v]) : x[i][v];
        } else {
          vfma(B, a[i], B, x[i]);
          if (LOGITS) vmul(A, A, a[i]);
        }
        if (i >= first) {
          put(i, B);
          if (mask >> (i + 1) & 1u) put_final(n, B);
        }
      }
      join<LOGITS>(sh, round, S, r, sends, p.waits, seg, li, A, B, inside != 0, carry, u);
#pragma unroll
      for (int i = 0; i < LS; ++i) {
        if (i >= first) continue;
        vfma(u, a[i], u, x[i]);
        put(i, u);
        if (mask >> (i + 1) & 1u) put_final(seq, u);
      }
    }
    stage = stage == STAGES - 1 ? 0 : stage + 1;
  }
  leave(sh, S);
}

// Sequences of at most one token (decoding): h_final = a h0 + x, a thread per V channels.
template <typename TX, typename TG, bool LOGITS, int V>
__global__ void __launch_bounds__(256) recurrence_step_kernel(RecurrenceLaunch p) {
  const int per = (p.C + 256 * V - 1) / (256 * V);   // blocks per sequence
  pdl_trigger();
  pdl_wait();
  for (int64_t b = blockIdx.x; b < (int64_t)p.n_seqs * per; b += gridDim.x) {
    const int n = (int)(b / per);
    const int c = ((int)(b - (int64_t)n * per) * 256 + (int)threadIdx.x) * V;
    if (c >= p.C) continue;
    const int t = __ldg(p.cu + n);
    const bool some = __ldg(p.cu + n + 1) > t && t >= 0 && t < p.T;
    const int64_t hc = (int64_t)n * p.C + c;
    float h[V] = {};
    if (p.h0) to_f32(ld_raw<float, V>(p.h0 + hc), h);
    if (some) {
      float x[V], g[V];
      to_f32(ld_raw<TX, V>(reinterpret_cast<const TX *>(p.x) + t * p.x_stride + c), x);
      to_f32(ld_raw<TG, V>(reinterpret_cast<const TG *>(p.gate) + t * p.gate_stride + c), g);
      float none[V] = {};
      decay<LOGITS>(g, g, none);
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = p.h0 ? fmaf(g[v], h[v], x[v]) : x[v];
      if (p.y) st_f32(reinterpret_cast<TX *>(p.y) + t * p.y_stride + c, h);
    }
    st_f32(p.h_final + hc, h);
  }
}

// The same scan from the last token to the first: segment position i is token t1 - i, and a
// sequence "begins" at its last token.
template <typename TX, typename TG, bool LOGITS, int V, int LS, int G>
__global__ void __launch_bounds__(kW * 32, 2) recurrence_grad_kernel(RecurrenceGradLaunch p, Parts parts) {
  using RX = Ring<TX, V, LS>;
  using RG = Ring<TG, V, LS>;
  constexpr int STAGES = stages_of(2 * RX::BYTES + RG::BYTES);
  extern __shared__ __align__(16) uint8_t smem[];
  RX rd(smem), rh(smem + STAGES * RX::BYTES);
  RG rg(smem + 2 * STAGES * RX::BYTES);
  Shared<V, G> &sh = *reinterpret_cast<Shared<V, G> *>(smem + STAGES * (2 * RX::BYTES + RG::BYTES));
  // (from lane 0: the compiler then keeps token indices and row pointers in uniform registers)
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t S = cluster_size(), r = cluster_rank();
  constexpr int LPG = 32 / G, SEGS = kW * G;
  const int grp = G == 1 ? 0 : lane / LPG, li = lane % LPG, seg = warp * G + grp;
  const int c = ((int)(blockIdx.x / S) * LPG + li) * V;
  const bool live = c < p.C;
  const int tb = parts.lo[blockIdx.y], te = parts.hi[blockIdx.y];
  const int chunk = (int)S * SEGS * LS;
  pdl_trigger();
  uint32_t sends = p.waits.hold_back && r + 1 == S ? 0 : S;   // CTAs that this thread sends its maps to
  begin(sh, S, sends == 0);
  pdl_wait();
  const int cl = live ? c : p.C - V;
  int t1 = te - 1 - ((int)r * SEGS + seg) * LS;
  const TX *pd = reinterpret_cast<const TX *>(p.dy) + (int64_t)t1 * p.dy_stride + cl;
  const TG *pg = reinterpret_cast<const TG *>(p.gate) + (int64_t)t1 * p.gate_stride + cl;
  const TX *ph = reinterpret_cast<const TX *>(p.y) + (int64_t)(t1 - 1) * p.y_stride + cl;   // h_{t-1}
  TX *ox = reinterpret_cast<TX *>(p.dx) + (int64_t)t1 * p.dx_stride + cl;
  TG *og = reinterpret_cast<TG *>(p.dgate) + (int64_t)t1 * p.dgate_stride + cl;
  int ahead = t1 - tb + 1;   // tokens from the run's begin to the next segment to fetch
  auto fetch = [&](int stage) {
    rd.issue(stage, pd, -p.dy_stride, ahead);
    rh.issue(stage, ph, -p.y_stride, ahead - 1);
    rg.issue(stage, pg, -p.gate_stride, ahead);
    cp_commit();
    pd -= chunk * p.dy_stride;
    ph -= chunk * p.y_stride;
    pg -= chunk * p.gate_stride;
    ahead -= chunk;
  };
  float carry = 0.f;
  int round = 0, stage = 0;
  const int low = parts.seq_lo[blockIdx.y];
  int seq = parts.seq_hi[blockIdx.y] - 1, from = te, to = 0;   // the sequence looked up last
#pragma unroll 1
  for (int i = 0; i < STAGES - 1; ++i) fetch(i);
  if (parts.some_empty && p.dh0)
    copy_empty<V>(p.cu, p.n_seqs, (int)((blockIdx.y * S + r) * SEGS) + seg, (int)(gridDim.y * S * SEGS),
                  c, live, p.C, p.dh_final, p.dh0);
#pragma unroll 1
  for (int tr1 = te - 1; tr1 >= tb;
       tr1 -= chunk, t1 -= chunk, ox -= chunk * p.dx_stride, og -= chunk * p.dgate_stride, ++round) {
    const int lim = t1 - tb + 1 < LS ? t1 - tb + 1 : LS;
    // starts of the tokens [t0, t1 + 1]: token t ends its sequence when t + 1 starts one
    const int t0 = t1 - lim + 1;
    uint32_t mask = 0;
    const bool look = lim > 0 && (t0 <= from || t1 + 1 >= to);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (!of_group<G>(look, g)) continue;
      int sq, f, t;
      const uint32_t m = lookup_down(p.cu, low, of_group<G>(seq, g) + 1, of_group<G>(t0, g),
                                     of_group<G>(lim, g), sq, f, t);
      if (grp == g) {
        mask = m;
        seq = sq;
        from = f;
        to = t;
      }
    }
    // the sequence that holds token t (t0 <= t <= t1): the last one that begins at or before it
    auto seq_of = [&](int t) {
      int n = seq;
      while (n + 1 < p.n_seqs && __ldg(p.cu + n + 1) <= t) ++n;
      return n;
    };
    // bit i: token t1 - i ends (begins) a sequence
    const uint32_t rev = lim > 0 ? __brev(mask) >> (31 - lim) : 0u;  // bit j: t0 + lim - j starts
    const uint32_t ends = rev & ((1u << (lim > 0 ? lim : 0)) - 1u);
    const uint32_t begins = rev >> 1;
    // The states of the first of each (h0 and dh_final are read in front of the wait for the
    // segment's own data; a segment that holds more of them reads the others where it needs them).
    const int b1 = begins ? __ffs(begins) - 1 : -1, e1 = ends ? __ffs(ends) - 1 : -1;
    float hb[V], he[V];
#pragma unroll
    for (int v = 0; v < V; ++v) hb[v] = he[v] = 0.f;
    auto state = [&](const float *from, int i, float (&h)[V]) {   // of token t1 - i's sequence
      const int64_t at = (int64_t)seq_of(t1 - i) * p.C + c;
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = from && live ? from[at + v] : 0.f;
    };
    if (b1 >= 0 && p.h0) state(p.h0, b1, hb);
    if (e1 >= 0 && p.dh_final) state(p.dh_final, e1, he);
    fetch(stage == 0 ? STAGES - 1 : stage - 1);   // into the slots of the round before
    cp_wait<STAGES - 1>();
    float A[V], B[V], u[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      A[v] = LOGITS ? 1.f : 0.f;
      B[v] = 0.f;
    }
    float a[LS][V], d[LS][V], q[LS][V];   // q = h_{t-1} d(log a)/d(gate)
#pragma unroll
    for (int i = 0; i < LS; ++i) {
      float g[V], h[V];
      to_f32(rd.get(stage, i), d[i]);
      to_f32(rh.get(stage, i), h);
      to_f32(rg.get(stage, i), g);
      if (begins >> i & 1u) {
        if (i != b1) state(p.h0, i, hb);
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = hb[v];
      }
      decay<LOGITS, true>(g, a[i], h, q[i], A);
    }
    // the token's gradients; on entry u is what reaches h_t from behind, on exit u_t
    auto emit = [&](int i, float (&uu)[V]) {
      float G[V], dg[V];
      vadd(G, d[i], uu);
      vmul(uu, a[i], G);
      vmul(dg, uu, q[i]);
      if (live) {
        st_f32(ox - i * p.dx_stride, G);
        st_f32(og - i * p.dgate_stride, dg);
      }
    };
    auto put_first = [&](int i, const float (&uu)[V]) {
      if (!(begins >> i & 1u) || !live || !p.dh0) return;
      const int n = seq_of(t1 - i);
#pragma unroll
      for (int v = 0; v < V; ++v) p.dh0[(int64_t)n * p.C + c + v] = uu[v];
    };
    if (all_of<G>(lim == LS && mask == 0)) {
#pragma unroll
      for (int i = 0; i < LS; ++i) {
        vadd(B, d[i], B);
        vmul(B, a[i], B);
        if (LOGITS) vmul(A, A, a[i]);
      }
      join<LOGITS>(sh, round, S, r, sends, p.waits, seg, li, A, B, false, carry, u);
#pragma unroll
      for (int i = 0; i < LS; ++i) emit(i, u);
    } else {
      const int first = ends ? __ffs(ends) - 1 : lim;
#pragma unroll
      for (int i = 0; i < LS; ++i) {
        if (i >= lim) continue;
        if (i < first) {
          vadd(B, d[i], B);
          vmul(B, a[i], B);
          if (LOGITS) vmul(A, A, a[i]);
          continue;
        }
        if (ends >> i & 1u) {
          if (i != e1) state(p.dh_final, i, he);
#pragma unroll
          for (int v = 0; v < V; ++v) B[v] = he[v];
        }
        emit(i, B);
        put_first(i, B);
      }
      join<LOGITS>(sh, round, S, r, sends, p.waits, seg, li, A, B, ends != 0, carry, u);
#pragma unroll
      for (int i = 0; i < LS; ++i)
        if (i < first) {
          emit(i, u);
          put_first(i, u);
        }
    }
    stage = stage == STAGES - 1 ? 0 : stage + 1;
  }
  leave(sh, S);
}

// How a call is spread: runs of whole sequences (grid.y) times S CTAs of a cluster that share a
// run's tokens, for `tiles` channel tiles, with `chunk1` tokens of a CTA in a round.  Two CTAs run
// on an SM at a time (`want` a tile).  Runs come first (they exchange nothing): up to eight times
// as many as run at once where each still has eight rounds, the longest first, so that the GPU's
// own scheduling balances them.  A cluster takes up what is left: a run longer than its fair
// share of the tokens, or CTAs that would not run at all.
struct Spread {
  int P, S;
  Parts parts;
  int64_t ctas(int tiles) const { return (int64_t)tiles * P * S; }
};
Spread spread(const int32_t *cu, int n_seqs, int64_t T, int tiles, int chunk1) {
  Spread sp{};
  const int64_t slots = 2 * device_sm_count(), want = std::max<int64_t>(1, slots / std::max(1, tiles));
  const int64_t goal = std::max<int64_t>({T / (8 * want), std::min<int64_t>(T / want + 1, 8 * chunk1),
                                          T / (kMaxParts - 1) + 1});
  struct Run {
    int32_t lo, hi, seq_lo, seq_hi;
  } runs[kMaxParts];
  int P = 0, first = 0;
  for (int n = 1; n <= n_seqs; ++n) {
    sp.parts.some_empty |= cu[n] == cu[n - 1];
    if (cu[n] - cu[first] < goal && n < n_seqs) continue;
    if (cu[n] > cu[first]) runs[P++] = {cu[first], cu[n], first, n};
    first = n;
  }
  if (P == 0) runs[P++] = {0, 0, 0, 0};
  std::sort(runs, runs + P, [](const Run &a, const Run &b) {
    return a.hi - a.lo != b.hi - b.lo ? a.hi - a.lo > b.hi - b.lo : a.lo < b.lo;
  });
  for (int i = 0; i < P; ++i) {
    sp.parts.lo[i] = runs[i].lo;
    sp.parts.hi[i] = runs[i].hi;
    sp.parts.seq_lo[i] = runs[i].seq_lo;
    sp.parts.seq_hi[i] = runs[i].seq_hi;
  }
  sp.P = P;
  const int64_t most = runs[0].hi - runs[0].lo, fair = T / want + 1;
  for (sp.S = 1; sp.S < kMaxCluster; sp.S *= 2) {
    const int64_t rounds = (most + sp.S * chunk1 - 1) / (sp.S * chunk1);
    const bool fits = 2 * sp.ctas(tiles) <= slots;
    if (!(fits && rounds > 4) && !(4 * most > 5 * sp.S * fair && rounds > 8)) break;
  }
  return sp;
}

// `stage`: bytes of a round's operands in a CTA
template <int V, int G, typename Launch>
cudaError_t launch_spread(void (*kern)(Launch, Parts), const Launch &p, const Spread &sp, int tiles, int stage,
                          cudaStream_t s, bool pdl) {
  // The limit is the kernel's and the process's, not the call's: it is always set to the most that
  // a launch of `kern` takes, so that another host thread's call never lowers it before this launch.
  const size_t rings = (size_t)stages_of(stage) * stage, smem = rings + shared_bytes<V, G>(sp.S);
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)(rings + shared_bytes<V, G>(kMaxCluster)));
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)sp.S;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * sp.S), (unsigned)sp.P);
  cfg.blockDim = dim3(kW * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p, sp.parts);
}

// Launches `kern` (V channels a lane, segments of LS tokens, G groups of lanes a warp; `tok` bytes
// of operands per token and channel) if that makes a CTA for every SM, and needs no cluster where
// there are runs enough to fill the GPU (narrower tiles balance those better: 16384 x 2048 in 20
// sequences, fp32, 76 us against 87) or where `alone` is asked for; or if it is the last choice.
template <int V, int LS, int G, typename Launch>
bool choose(void (*kern)(Launch, Parts), const Launch &p, int tok, bool alone, bool last, cudaStream_t s, bool pdl,
            cudaError_t *e) {
  const int tiles = (p.C + 32 / G * V - 1) / (32 / G * V);
  const Spread sp = spread(p.cu_host, p.n_seqs, p.T, tiles, kW * G * LS);
  const bool runs = (int64_t)tiles * sp.P >= 2 * device_sm_count();
  if (!last && (sp.ctas(tiles) < device_sm_count() || ((alone || runs) && sp.S > 1))) return false;
  *e = launch_spread<V, G>(kern, p, sp, tiles, kW * 32 * V * LS * tok, s, pdl);
  return true;
}

bool vec_ok(const void *p, int64_t stride, int elem, int V) {
  return (reinterpret_cast<uintptr_t>(p) % (uintptr_t)(V * elem)) == 0 && stride % V == 0;
}

template <typename TX, typename TG, bool LOGITS>
cudaError_t go(const RecurrenceLaunch &p, cudaStream_t s, bool pdl) {
  auto fits = [&](int V) {
    return p.C % V == 0 && vec_ok(p.x, p.x_stride, sizeof(TX), V) && vec_ok(p.gate, p.gate_stride, sizeof(TG), V) &&
           vec_ok(p.y, p.y_stride, sizeof(TX), V);
  };
  int longest = 0;
  for (int n = 0; n < p.n_seqs; ++n) longest = std::max(longest, p.cu_host[n + 1] - p.cu_host[n]);
  if (longest <= 1) {
    const bool four = fits(4) && vec_ok(p.h0, 0, 4, 4) && vec_ok(p.h_final, 0, 4, 4);
    const int64_t blocks = (int64_t)p.n_seqs * ((p.C + (four ? 1023 : 255)) / (four ? 1024 : 256));
    const dim3 grid((unsigned)std::min<int64_t>(blocks, 1 << 20));
    return four ? launch_kernel(recurrence_step_kernel<TX, TG, LOGITS, 4>, grid, dim3(256), 0, s, pdl, p)
                : launch_kernel(recurrence_step_kernel<TX, TG, LOGITS, 1>, grid, dim3(256), 0, s, pdl, p);
  }
  // segments of 32 elements a thread where both operands have two bytes, else of 16
  constexpr int kTok = sizeof(TX) + sizeof(TG), kElems = kTok == 4 ? 32 : 16;
  // Four channels a lane take the fewest instructions, in tiles of 128 (16384 x 4096, 40 sequences,
  // bf16 and fp32 gates: 87 us; two in tiles of 64: 103); narrower tiles where those would be too
  // few or would need a cluster (16384 x 4096 in one sequence, fp32: 178 us, 147 with two channels
  // a lane; 65536 x 1024 in one sequence, bf16: 229 us in tiles of 64, 153 in tiles of 32).
  constexpr int LS4 = kElems / 4, LS2 = kElems / 2;
  cudaError_t e = cudaSuccess;
  if (fits(4) &&
      choose<4, LS4, 1>(recurrence_kernel<TX, TG, LOGITS, 4, LS4, 1>, p, kTok, true, false, s, pdl, &e))
    return e;
  if (!fits(2))
    choose<1, 16, 1>(recurrence_kernel<TX, TG, LOGITS, 1, 16, 1>, p, kTok, false, true, s, pdl, &e);
  else if (!choose<2, LS2, 1>(recurrence_kernel<TX, TG, LOGITS, 2, LS2, 1>, p, kTok, false, false, s, pdl, &e))
    choose<2, LS2, 2>(recurrence_kernel<TX, TG, LOGITS, 2, LS2, 2>, p, kTok, false, true, s, pdl, &e);
  return e;
}

template <typename TX, typename TG, bool LOGITS>
cudaError_t go(const RecurrenceGradLaunch &p, cudaStream_t s, bool pdl) {
  auto fits = [&](int V) {
    return p.C % V == 0 && vec_ok(p.dy, p.dy_stride, sizeof(TX), V) && vec_ok(p.gate, p.gate_stride, sizeof(TG), V) &&
           vec_ok(p.y, p.y_stride, sizeof(TX), V) && vec_ok(p.dx, p.dx_stride, sizeof(TX), V) &&
           vec_ok(p.dgate, p.dgate_stride, sizeof(TG), V);
  };
  // (at 10 or 12 bytes a token shorter segments: rings of 64 KB; 13130 x 2022, fp32: 105 us, 219
  // with segments of 8)
  constexpr int kTok = 2 * sizeof(TX) + sizeof(TG), LS2 = kTok >= 10 ? 4 : 8;
  // As above, in tiles of 64 (16384 x 4096, 40 sequences, fp32: 209 us; 246 in tiles of 128, 269
  // with two channels a lane) or 32 (20000 x 256 in three sequences: 59 us, 92 in tiles of 64).
  cudaError_t e = cudaSuccess;
  if (fits(4) &&
      choose<4, 4, 2>(recurrence_grad_kernel<TX, TG, LOGITS, 4, 4, 2>, p, kTok, false, false, s, pdl, &e))
    return e;
  if (!fits(2))
    choose<1, 8, 1>(recurrence_grad_kernel<TX, TG, LOGITS, 1, 8, 1>, p, kTok, false, true, s, pdl, &e);
  else if (!choose<2, LS2, 1>(recurrence_grad_kernel<TX, TG, LOGITS, 2, LS2, 1>, p, kTok, false, false, s, pdl, &e))
    choose<2, LS2, 2>(recurrence_grad_kernel<TX, TG, LOGITS, 2, LS2, 2>, p, kTok, false, true, s, pdl, &e);
  return e;
}

template <typename Launch>
cudaError_t by_type(const Launch &p, cudaStream_t s, bool pdl) {
  typedef __nv_bfloat16 H;
  if (p.n_seqs <= 0) return cudaSuccess;
  if (p.x_bf16)
    return p.gate_bf16 ? (p.logits ? go<H, H, true>(p, s, pdl) : go<H, H, false>(p, s, pdl))
                       : (p.logits ? go<H, float, true>(p, s, pdl) : go<H, float, false>(p, s, pdl));
  return p.gate_bf16 ? (p.logits ? go<float, H, true>(p, s, pdl) : go<float, H, false>(p, s, pdl))
                     : (p.logits ? go<float, float, true>(p, s, pdl) : go<float, float, false>(p, s, pdl));
}

}  // namespace

cudaError_t launch_recurrence(const RecurrenceLaunch &p, cudaStream_t s, bool pdl) { return by_type(p, s, pdl); }
cudaError_t launch_recurrence_grad(const RecurrenceGradLaunch &p, cudaStream_t s, bool pdl) {
  return by_type(p, s, pdl);
}

}  // namespace tr

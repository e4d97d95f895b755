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
// in a round each warp holds a segment of consecutive tokens of its lanes' channels in
// registers (the next round's loads already in flight), reduces it to one map (A, B) per
// channel, and the segments are joined in time order: the warps of a CTA through shared
// memory, the CTAs of the cluster through each other's shared memory, one cluster barrier a
// round.  Every warp then knows the state in front of its segment and replays the segment
// from registers.  Nothing is read twice, nothing passes through global memory, and the order
// of every sum is fixed, so results are bitwise reproducible.
//
// The packed tokens are scanned as one long sequence that starts over where a sequence
// begins.  That is a selection, not a product with a = 0, so infinities or NaN of one
// sequence never reach the next.  All states, products and sums are fp32; outputs are rounded
// once.
#include <cuda_bf16.h>

#include <algorithm>

#include "fp8_ptx.cuh"
#include "layer_ops.h"
#include "tr_internal.h"

namespace tr {
namespace {

constexpr int kW = 8;             // warps of a CTA: segments of a round
constexpr int kMaxParts = 64;     // independent runs of whole sequences (grid.y)
constexpr int kMaxCluster = 8;

struct Parts {
  int32_t at[kMaxParts + 1];      // token bounds of the runs, each at a sequence start
};

// V channels of one token as loaded
template <typename T, int V> struct Raw;
template <> struct Raw<__nv_bfloat16, 1> { unsigned short u; };
template <> struct Raw<__nv_bfloat16, 2> { uint32_t u; };
template <> struct Raw<float, 1> { float f; };
template <> struct Raw<float, 2> { float2 f; };

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> ld_raw(const void *p, int64_t off, bool in) {
  Raw<T, V> r{};
  if (in) r = *reinterpret_cast<const Raw<T, V> *>(reinterpret_cast<const T *>(p) + off);
  return r;
}
__device__ __forceinline__ void to_f32(const Raw<__nv_bfloat16, 1> &r, float (&f)[1]) {
  f[0] = __uint_as_float((uint32_t)r.u << 16);
}
__device__ __forceinline__ void to_f32(const Raw<__nv_bfloat16, 2> &r, float (&f)[2]) {
  f[0] = __uint_as_float(r.u << 16);
  f[1] = __uint_as_float(r.u & 0xffff0000u);
}
__device__ __forceinline__ void to_f32(const Raw<float, 1> &r, float (&f)[1]) { f[0] = r.f; }
__device__ __forceinline__ void to_f32(const Raw<float, 2> &r, float (&f)[2]) {
  f[0] = r.f.x;
  f[1] = r.f.y;
}
__device__ __forceinline__ void st_f32(__nv_bfloat16 *p, const float (&f)[1]) { *p = __float2bfloat16_rn(f[0]); }
__device__ __forceinline__ void st_f32(__nv_bfloat16 *p, const float (&f)[2]) {
  *reinterpret_cast<uint32_t *>(p) = pack_bf16x2(f[0], f[1]);
}
__device__ __forceinline__ void st_f32(float *p, const float (&f)[1]) { *p = f[0]; }
__device__ __forceinline__ void st_f32(float *p, const float (&f)[2]) {
  *reinterpret_cast<float2 *>(p) = make_float2(f[0], f[1]);
}

// a, and for the backward pass 1 - a where the gate is a logit.  Above 80 e^gate is held at
// e^80 (a < 2e-35); the comparison keeps a NaN.
template <bool LOGITS>
__device__ __forceinline__ float decay(float g, float &rest) {
  if (!LOGITS) return exp_ftz(g);
  const float e = exp_ftz(g > 80.f ? 80.f : g);
  const float a = __fdividef(1.f, 1.f + e);
  rest = e * a;
  return a;
}

// The maps of a round: per warp of this CTA, and per CTA of the cluster (two sets, used in
// turn: the barrier of a round is passed only when every reader of the round before is done).
template <int V>
struct Maps {
  float A[V][32], B[V][32];
  float start;                     // 1: a sequence begins inside, so A does not count
};
template <int V>
struct Shared {
  Maps<V> warp[2][kW];
  Maps<V> cta[2][kMaxCluster];
};

// Where sequences begin in tokens [t0, t0 + n], n <= 31: bit i for a cu entry equal to t0 + i
// (cu[N] = T among them); first = the last sequence with cu <= t0.  `hint` is a sequence known
// to begin at or before t0.  The whole warp calls it with the same arguments.
__device__ __forceinline__ uint32_t starts_mask(const int32_t *__restrict__ cu, int n_seqs, int t0,
                                                int n, int hint, int &first) {
  const int lane = threadIdx.x & 31;
  // the last index in [lo, n_seqs] with cu <= t0, 32 probes a step
  int lo = hint, hi = n_seqs + 1;             // cu[lo] <= t0, cu[hi] > t0 (hi: past the end)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + (lane + 1) * step;    // lane 31 is at or past hi
    const bool le = at < hi && __ldg(cu + at) <= t0;
    const int k = __popc(__ballot_sync(0xffffffffu, le));   // probes that hold are a prefix
    const int nlo = lo + k * step;
    hi = nlo + step < hi ? nlo + step : hi;
    lo = nlo;
  }
  first = lo;
  uint32_t m = __ldg(cu + lo) == t0 ? 1u : 0u;
  for (int i = lo + 1 + lane;; i += 32) {
    const bool past = i > n_seqs || __ldg(cu + i) - t0 > n;
    if (!past) m |= 1u << (__ldg(cu + i) - t0);
    if (__ballot_sync(0xffffffffu, past)) break;
  }
  return __reduce_or_sync(0xffffffffu, m);
}

// u after the map (A, B), or after a segment in which a sequence begins
__device__ __forceinline__ float apply(float A, float B, float start, float u) {
  return start != 0.f ? B : fmaf(A, u, B);
}

// Joins the warps' maps of a round.  In: this warp's map.  Out: the value in front of this
// warp's segment; `carry` (the value in front of the round) moves to the next round.
template <int V>
__device__ __forceinline__ void join(Shared<V> &sh, int par, uint32_t S, uint32_t r, const float (&A)[V],
                                     const float (&B)[V], bool start, float (&carry)[V], float (&u)[V]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Maps<V> &mine = sh.warp[par][warp];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    mine.A[v][lane] = A[v];
    mine.B[v][lane] = B[v];
  }
  if (lane == 0) mine.start = start ? 1.f : 0.f;
  __syncthreads();
  if (S > 1) {
    if (warp == 0) {
      float a[V], b[V], st = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        a[v] = 1.f;
        b[v] = 0.f;
      }
#pragma unroll
      for (int w = 0; w < kW; ++w) {
        const Maps<V> &m = sh.warp[par][w];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          b[v] = apply(m.A[v][lane], m.B[v][lane], m.start, b[v]);
          a[v] *= m.A[v][lane];
        }
        st = m.start != 0.f ? 1.f : st;
      }
      Maps<V> &to = sh.cta[par][r];
      for (uint32_t k = 0; k < S; ++k) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          st_cluster(smem_u32(&to.A[v][lane]), k, a[v]);
          st_cluster(smem_u32(&to.B[v][lane]), k, b[v]);
        }
        if (lane == 0) st_cluster(smem_u32(&to.start), k, st);
      }
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    for (uint32_t k = 0; k < S; ++k) {
      const Maps<V> &m = sh.cta[par][k];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (k == r) u[v] = carry[v];
        carry[v] = apply(m.A[v][lane], m.B[v][lane], m.start, carry[v]);
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) u[v] = carry[v];
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      const Maps<V> &m = sh.warp[par][w];
#pragma unroll
      for (int v = 0; v < V; ++v)
        carry[v] = apply(m.A[v][lane], m.B[v][lane], m.start, carry[v]);
    }
  }
  for (int w = 0; w < warp; ++w) {
    const Maps<V> &m = sh.warp[par][w];
#pragma unroll
    for (int v = 0; v < V; ++v) u[v] = apply(m.A[v][lane], m.B[v][lane], m.start, u[v]);
  }
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

template <typename TX, typename TG, bool LOGITS, int V, int LS>
__global__ void __launch_bounds__(kW * 32, 2) recurrence_kernel(RecurrenceLaunch p, Parts parts) {
  __shared__ Shared<V> sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t S = cluster_size(), r = cluster_rank();
  const int c = (int)(blockIdx.x / S) * 32 * V + lane * V;
  const bool live = c < p.C;
  const int tb = parts.at[blockIdx.y], te = parts.at[blockIdx.y + 1];
  const int chunk = (int)S * kW * LS;
  pdl_trigger();
  if (S > 1) {   // every CTA of the cluster has started before any writes to it
    cluster_arrive();
    cluster_wait();
  }
  pdl_wait();
  copy_empty<V>(p.cu, p.n_seqs, (int)((blockIdx.y * S + r) * kW) + warp, (int)(gridDim.y * S * kW), c,
                live, p.C, p.h0, p.h_final);
  Raw<TX, V> nx[LS];
  Raw<TG, V> ng[LS];
  const int seg0 = (int)r * kW * LS + warp * LS;
  auto fetch = [&](int t0) {
#pragma unroll
    for (int i = 0; i < LS; ++i) {
      const bool in = live && t0 + i < te;
      nx[i] = ld_raw<TX, V>(p.x, (int64_t)(t0 + i) * p.x_stride + c, in);
      ng[i] = ld_raw<TG, V>(p.gate, (int64_t)(t0 + i) * p.gate_stride + c, in);
    }
  };
  float carry[V] = {};
  int hint = 0, par = 0;
  fetch(tb + seg0);
  for (int tr0 = tb; tr0 < te; tr0 += chunk, par ^= 1) {
    const int t0 = tr0 + seg0;
    const int lim = te - t0 < LS ? te - t0 : LS;    // tokens of the segment (may be <= 0)
    float a[LS][V], x[LS][V];
#pragma unroll
    for (int i = 0; i < LS; ++i) {
      float g[V], rest;
      to_f32(nx[i], x[i]);
      to_f32(ng[i], g);
#pragma unroll
      for (int v = 0; v < V; ++v) a[i][v] = decay<LOGITS>(g[v], rest);
    }
    if (te - tr0 > chunk) fetch(t0 + chunk);
    int seq = 0;
    const uint32_t mask = lim > 0 ? starts_mask(p.cu, p.n_seqs, t0, LS, hint, seq) : 0u;
    hint = lim > 0 ? seq : hint;
    const uint32_t inside = mask & ((1u << (lim > 0 ? lim : 0)) - 1u);
    const int first = inside ? __ffs(inside) - 1 : lim;   // tokens of the sequence before
    float A[V], B[V], u[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      A[v] = 1.f;
      B[v] = 0.f;
    }
    auto put = [&](int t, const float (&h)[V]) {
      if (p.y && live) st_f32(reinterpret_cast<TX *>(p.y) + (int64_t)t * p.y_stride + c, h);
    };
    auto put_final = [&](int n, const float (&h)[V]) {
      if (!live) return;
#pragma unroll
      for (int v = 0; v < V; ++v) p.h_final[(int64_t)n * p.C + c + v] = h[v];
    };
    if (first == LS) {
#pragma unroll
      for (int i = 0; i < LS; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          B[v] = fmaf(a[i][v], B[v], x[i][v]);
          A[v] *= a[i][v];
        }
    } else {
      // from the first sequence start on, the states do not depend on what lies before the
      // segment: they are final here
      int n = seq;
#pragma unroll
      for (int i = 0; i < LS; ++i) {
        if (i >= lim) continue;
        if (mask >> i & 1u) {
          while (__ldg(p.cu + n + 1) <= t0 + i) ++n;
#pragma unroll
          for (int v = 0; v < V; ++v)
            B[v] = p.h0 && live ? fmaf(a[i][v], p.h0[(int64_t)n * p.C + c + v], x[i][v]) : x[i][v];
        } else {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            B[v] = fmaf(a[i][v], B[v], x[i][v]);
            A[v] *= a[i][v];
          }
        }
        if (i >= first) {
          put(t0 + i, B);
          if (mask >> (i + 1) & 1u) put_final(n, B);
        }
      }
    }
    join<V>(sh, par, S, r, A, B, inside != 0, carry, u);
    if (first == LS) {
#pragma unroll
      for (int i = 0; i < LS; ++i) {
#pragma unroll
        for (int v = 0; v < V; ++v) u[v] = fmaf(a[i][v], u[v], x[i][v]);
        put(t0 + i, u);
      }
      if (mask >> LS & 1u) put_final(seq, u);
    } else {
#pragma unroll
      for (int i = 0; i < LS; ++i) {
        if (i >= first) continue;
#pragma unroll
        for (int v = 0; v < V; ++v) u[v] = fmaf(a[i][v], u[v], x[i][v]);
        put(t0 + i, u);
        if (mask >> (i + 1) & 1u) put_final(seq, u);
      }
    }
  }
}

// The same scan from the last token to the first: segment position i is token t1 - i, and a
// sequence "begins" at its last token.
template <typename TX, typename TG, bool LOGITS, int V, int LS>
__global__ void __launch_bounds__(kW * 32, 2) recurrence_grad_kernel(RecurrenceGradLaunch p, Parts parts) {
  __shared__ Shared<V> sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t S = cluster_size(), r = cluster_rank();
  const int c = (int)(blockIdx.x / S) * 32 * V + lane * V;
  const bool live = c < p.C;
  const int tb = parts.at[blockIdx.y], te = parts.at[blockIdx.y + 1];
  const int chunk = (int)S * kW * LS;
  pdl_trigger();
  if (S > 1) {
    cluster_arrive();
    cluster_wait();
  }
  pdl_wait();
  if (p.dh0)
    copy_empty<V>(p.cu, p.n_seqs, (int)((blockIdx.y * S + r) * kW) + warp, (int)(gridDim.y * S * kW),
                  c, live, p.C, p.dh_final, p.dh0);
  Raw<TX, V> nd[LS], ny[LS];
  Raw<TG, V> ng[LS];
  const int seg0 = (int)r * kW * LS + warp * LS;
  auto fetch = [&](int t1) {
#pragma unroll
    for (int i = 0; i < LS; ++i) {
      const int t = t1 - i;
      const bool in = live && t >= tb;
      nd[i] = ld_raw<TX, V>(p.dy, (int64_t)t * p.dy_stride + c, in);
      ng[i] = ld_raw<TG, V>(p.gate, (int64_t)t * p.gate_stride + c, in);
      ny[i] = ld_raw<TX, V>(p.y, (int64_t)(t - 1) * p.y_stride + c, in && t > tb);
    }
  };
  float carry[V] = {};
  int par = 0;
  fetch(te - 1 - seg0);
  for (int tr1 = te - 1; tr1 >= tb; tr1 -= chunk, par ^= 1) {
    const int t1 = tr1 - seg0;
    const int lim = t1 - tb + 1 < LS ? t1 - tb + 1 : LS;
    float a[LS][V], w[LS][V], d[LS][V], hp[LS][V];   // w = d(log a)/d(gate)
#pragma unroll
    for (int i = 0; i < LS; ++i) {
      float g[V];
      to_f32(nd[i], d[i]);
      to_f32(ny[i], hp[i]);
      to_f32(ng[i], g);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        a[i][v] = decay<LOGITS>(g[v], w[i][v]);
        if (LOGITS) w[i][v] = -w[i][v];
      }
    }
    if (tr1 - tb >= chunk) fetch(t1 - chunk);
    // starts of the tokens [t0, t1 + 1]: token t ends its sequence when t + 1 starts one
    const int t0 = t1 - lim + 1;
    int seq = 0;
    const uint32_t mask = lim > 0 ? starts_mask(p.cu, p.n_seqs, t0, lim, 0, seq) : 0u;
    // bit i: token t1 - i ends (begins) a sequence
    const uint32_t rev = lim > 0 ? __brev(mask) >> (31 - lim) : 0u;  // bit j: t0 + lim - j starts
    const uint32_t ends = rev & ((1u << (lim > 0 ? lim : 0)) - 1u);
    const uint32_t begins = rev >> 1;
    const int first = ends ? __ffs(ends) - 1 : lim;
    float A[V], B[V], u[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      A[v] = 1.f;
      B[v] = 0.f;
    }
    // the token's gradients; on entry u is what reaches h_t from behind, on exit u_t
    auto emit = [&](int i, float (&uu)[V], int n) {
      const int t = t1 - i;
      float G[V], dg[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        G[v] = d[i][v] + uu[v];
        uu[v] = a[i][v] * G[v];
      }
      const bool begin = begins >> i & 1u;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float h = hp[i][v];
        if (begin) h = p.h0 && live ? p.h0[(int64_t)n * p.C + c + v] : 0.f;
        dg[v] = uu[v] * h;
        if (LOGITS) dg[v] *= w[i][v];
      }
      if (live) {
        st_f32(reinterpret_cast<TX *>(p.dx) + (int64_t)t * p.dx_stride + c, G);
        st_f32(reinterpret_cast<TG *>(p.dgate) + (int64_t)t * p.dgate_stride + c, dg);
        if (begin && p.dh0) {
#pragma unroll
          for (int v = 0; v < V; ++v) p.dh0[(int64_t)n * p.C + c + v] = uu[v];
        }
      }
    };
    // the sequence that holds token t (t0 <= t <= t1): the last one that begins at or before it
    auto seq_of = [&](int t) {
      int n = seq;
      while (n + 1 < p.n_seqs && __ldg(p.cu + n + 1) <= t) ++n;
      return n;
    };
    if (first == LS) {
#pragma unroll
      for (int i = 0; i < LS; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          B[v] = a[i][v] * (d[i][v] + B[v]);
          A[v] *= a[i][v];
        }
    } else {
      int n = 0;
#pragma unroll
      for (int i = 0; i < LS; ++i) {
        if (i >= lim) continue;
        if (i < first) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            B[v] = a[i][v] * (d[i][v] + B[v]);
            A[v] *= a[i][v];
          }
          continue;
        }
        if (ends >> i & 1u) {
          n = seq_of(t1 - i);
#pragma unroll
          for (int v = 0; v < V; ++v)
            B[v] = p.dh_final && live ? p.dh_final[(int64_t)n * p.C + c + v] : 0.f;
        }
        emit(i, B, n);
      }
    }
    join<V>(sh, par, S, r, A, B, ends != 0, carry, u);
    if (first > 0) {
      const int n = begins ? seq_of(t1) : 0;
#pragma unroll
      for (int i = 0; i < LS; ++i)
        if (i < first) emit(i, u, n);
    }
  }
}

// How a call is spread: P runs of whole sequences (grid.y) times S CTAs of a cluster that share
// a run's tokens, for `tiles` channel tiles.  Enough CTAs to fill the GPU twice over where the
// tokens allow it; runs come first (they exchange nothing), as far as whole sequences can be
// balanced, then the cluster.
struct Spread {
  int P, S;
  Parts parts;
};
Spread spread(const int32_t *cu, int n_seqs, int64_t T, int tiles, int chunk1) {
  Spread sp{};
  const int64_t want = std::max<int64_t>(1, 2 * device_sm_count() / std::max(1, tiles));
  int longest = 1;
  for (int n = 0; n < n_seqs; ++n) longest = std::max(longest, cu[n + 1] - cu[n]);
  const int64_t pmax = std::min<int64_t>({want, T / longest, T / chunk1, kMaxParts});
  sp.P = (int)std::max<int64_t>(1, pmax);
  sp.parts.at[0] = 0;
  int64_t most = 0;
  for (int i = 1; i <= sp.P; ++i) {
    if (i == sp.P) {
      sp.parts.at[i] = (int32_t)T;
    } else {
      const int64_t goal = T * i / sp.P;
      const int32_t *hi = std::lower_bound(cu, cu + n_seqs + 1, (int32_t)goal);
      int32_t at = *hi;
      if (hi != cu && goal - hi[-1] < *hi - goal) at = hi[-1];
      sp.parts.at[i] = std::max(at, sp.parts.at[i - 1]);
    }
    most = std::max<int64_t>(most, sp.parts.at[i] - sp.parts.at[i - 1]);
  }
  sp.S = 1;
  while (sp.S < kMaxCluster && sp.P * sp.S * 2 <= want && most > (int64_t)sp.S * chunk1) sp.S *= 2;
  return sp;
}

template <typename Launch>
cudaError_t launch_spread(void (*kern)(Launch, Parts), const Launch &p, const Spread &sp, int tiles,
                          cudaStream_t s, bool pdl) {
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
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p, sp.parts);
}

bool vec_ok(const void *p, int64_t stride, int elem) {
  return (reinterpret_cast<uintptr_t>(p) % (2 * elem)) == 0 && stride % 2 == 0;
}

template <typename TX, typename TG, bool LOGITS>
cudaError_t go(const RecurrenceLaunch &p, cudaStream_t s, bool pdl) {
  // two channels a lane where pairs are aligned; segments of as many tokens as keep the loads
  // in flight at 16 registers an operand
  const bool two = p.C % 2 == 0 && vec_ok(p.x, p.x_stride, sizeof(TX)) &&
                   vec_ok(p.gate, p.gate_stride, sizeof(TG)) && vec_ok(p.y, p.y_stride, sizeof(TX));
  constexpr int LS2 = sizeof(TX) + sizeof(TG) == 4 ? 16 : 8;
  const int tiles = (p.C + (two ? 63 : 31)) / (two ? 64 : 32);
  const Spread sp = spread(p.cu_host, p.n_seqs, p.T, tiles, kW * (two ? LS2 : 16));
  return two ? launch_spread<RecurrenceLaunch>(recurrence_kernel<TX, TG, LOGITS, 2, LS2>, p, sp, tiles, s, pdl)
             : launch_spread<RecurrenceLaunch>(recurrence_kernel<TX, TG, LOGITS, 1, 16>, p, sp, tiles, s, pdl);
}

template <typename TX, typename TG, bool LOGITS>
cudaError_t go(const RecurrenceGradLaunch &p, cudaStream_t s, bool pdl) {
  const bool two = p.C % 2 == 0 && vec_ok(p.dy, p.dy_stride, sizeof(TX)) &&
                   vec_ok(p.gate, p.gate_stride, sizeof(TG)) && vec_ok(p.y, p.y_stride, sizeof(TX)) &&
                   vec_ok(p.dx, p.dx_stride, sizeof(TX)) && vec_ok(p.dgate, p.dgate_stride, sizeof(TG));
  constexpr int LS2 = 8;
  const int tiles = (p.C + (two ? 63 : 31)) / (two ? 64 : 32);
  const Spread sp = spread(p.cu_host, p.n_seqs, p.T, tiles, kW * 8);
  return two ? launch_spread<RecurrenceGradLaunch>(recurrence_grad_kernel<TX, TG, LOGITS, 2, LS2>, p, sp, tiles, s, pdl)
             : launch_spread<RecurrenceGradLaunch>(recurrence_grad_kernel<TX, TG, LOGITS, 1, 8>, p, sp, tiles, s, pdl);
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

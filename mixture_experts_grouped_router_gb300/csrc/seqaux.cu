// The load-balancing loss of every sequence of a ragged batch, the router's z
// loss, and their logit gradient.
//
// For sequence b with n_b live tokens, counts c_be of their choices and
// probabilities p_te (softmax, or sigmoid scores over their sum):
//     f_be = E c_be / (k n_b),   P_be = mean of p_te,
//     L = coeff / S sum_b sum_e f_be P_be  +  z_coeff / N sum_t lse_t^2
// (S sequences that have live tokens, N live tokens, lse the logarithm of the sum of the
// exponentials), and with the counts held fixed
//     dl_te = coeff / (S n_b) J_te (f_be - sum_j f_bj p_tj) + z_coeff 2 lse_t softmax_te / N,
// J = p (softmax) or s (1 - s) / sum s (sigmoid).  The gradient takes the counts alone of
// the whole sequence, so that they are counted first (4 k bytes a token) and one pass over
// the logits gives both the sums P and the gradient.
//
// The balance loss needs no P: sum_e f_be P_be is the mean over the sequence's tokens of
// sum_e f_be p_te, which the gradient takes anyway.
//
// Deterministic: atomics add integers alone, sums of floats are taken in a fixed order.  A
// block's tokens may lie in several sequences; its part of sequence b's P is slot (block +
// b) of the workspace: both grow along the tokens, one at least from part to part, so that
// no two parts share a slot.
//
// What bounds it: a step's instructions and their chain.  65521 tokens of 256 experts, sigmoid: 21 us
// for the loss's pass, 24 for the gradient's, calls following one another (each by itself with cold
// caches 23.5 and 26.2), some 175 warp instructions a token at 16 warps a SM, 40% of the issue slots; small
// batches the latency of the launches (count, logits, finish; 7 to 10 us in a graph).
#include <math.h>

#include <algorithm>

#include "internal.h"
#include "lowbit.cuh"
#include "seqaux_layout.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxE = 256;
constexpr int kMaxBlocks = 1280;  // of the pass over the logits

MOE_DEVINL int clampi(int v, int lo, int hi) { return min(max(v, lo), hi); }

MOE_DEVINL int warp_sum_i(int v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Counts by sequence.  A histogram has 8 columns, by lane, so that a warp's choices of one
// expert seldom meet.
constexpr int kCols = 8;
constexpr int kCountThreads = 1024;  // at most

struct Histogram {
  int *h;  // [E][kCols]
  int E;
  MOE_DEVINL void clear() {
    for (int i = threadIdx.x; i < E * kCols; i += blockDim.x) h[i] = 0;
  }
  MOE_DEVINL void add(int e) {
    if ((uint32_t)e < (uint32_t)E) atomicAdd(&h[e * kCols + (threadIdx.x & (kCols - 1))], 1);
  }
  // Expert e's count (the columns in an order that keeps a warp's reads apart).
  MOE_DEVINL int total(int e) const {
    int n = 0;
#pragma unroll
    for (int i = 0; i < kCols; ++i) n += h[e * kCols + ((i + (e >> 2)) & (kCols - 1))];
    return n;
  }
  // Choices of the live tokens of [lo, hi) by the block's threads; returns the thread's live tokens.
  MOE_DEVINL int count(const SeqAuxArgs &a, int lo, int hi) {
    const int step = blockDim.x;
    if (a.mask == nullptr) {
      const int64_t end = (int64_t)hi * a.k;
      int64_t i = (int64_t)lo * a.k + threadIdx.x;
      for (; i + 15 * step < end; i += 16 * step) {
        int e[16];
#pragma unroll
        for (int u = 0; u < 16; ++u) e[u] = ld_i32(a.idx + i + u * step);
#pragma unroll
        for (int u = 0; u < 16; ++u) add(e[u]);
      }
      for (; i < end; i += 4 * step) {
        int e[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) e[u] = i + u * step < end ? ld_i32(a.idx + i + u * step) : -1;
#pragma unroll
        for (int u = 0; u < 4; ++u) add(e[u]);
      }
      return threadIdx.x == 0 ? hi - lo : 0;
    }
    // choice i is slot r of token t; both move on by additions
    const int dt = step / a.k, dr = step - dt * a.k;
    int t = lo + threadIdx.x / a.k, r = threadIdx.x % a.k, n = 0;
    while (t < hi) {
      int e[8];
      bool live[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        e[u] = -1;
        live[u] = false;
        if (t < hi) {
          live[u] = ld_u8(a.mask + t) != 0;
          e[u] = ld_i32(a.idx + (int64_t)t * a.k + r);
          if (r == 0) n += live[u];
        }
        t += dt;
        r += dr;
        if (r >= a.k) {
          r -= a.k;
          ++t;
        }
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) add(live[u] ? e[u] : -1);
    }
    return n;
  }
};

// A block a sequence.
__global__ void __launch_bounds__(kCountThreads)
seq_count_kernel(const SeqAuxArgs a) {
  __shared__ int hist[kMaxE * kCols];
  __shared__ int s_n;
  const int lane = threadIdx.x & 31, b = blockIdx.x;
  Histogram h = {hist, a.E};
  h.clear();
  if (threadIdx.x == 0) s_n = 0;
  __syncthreads();
  grid_dependency_begin();
  const int lo = clampi(ld_i32(a.offsets + b), 0, a.T);
  const int hi = clampi(ld_i32(a.offsets + b + 1), lo, a.T);
  const int n = warp_sum_i(h.count(a, lo, hi));
  if (lane == 0 && n > 0) atomicAdd(&s_n, n);
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) a.counts[(int64_t)b * a.E + e] = h.total(e);
  if (threadIdx.x == 0) a.tokens[b] = s_n;
}

__global__ void __launch_bounds__(kThreads)
seq_zero_kernel(const SeqAuxArgs a) {
  grid_dependency_begin();
  const int64_t n = (int64_t)a.B * a.E;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n + a.B; i += (int64_t)gridDim.x * kThreads)
    (i < n ? a.counts + i : a.tokens + (i - n))[0] = 0;
}

// The last j in [-1, n) with v[j] <= t (v ascending, v[-1] = -inf), by 32 probes a step.
MOE_DEVINL int last_at_most(const int32_t *v, int n, int t, int lane) {
  int lo = -1, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo - 1 + 31) / 32;
    const int p = lo + 1 + lane * step;
    const uint32_t m = __ballot_sync(0xffffffffu, p < hi && ld_i32(v + min(p, n - 1)) <= t);
    const int c = m == 0xffffffffu ? 32 : __ffs(~m) - 1;  // probes that are, from the first on
    const int above = lo + 1 + c * step;
    if (c > 0) lo = lo + 1 + (c - 1) * step;
    if (c < 32 && above < hi) hi = above;
  }
  return lo;
}

// The last j in [lo, hi) with v[j] <= t, by each lane for itself (v[lo] <= t, or lo is -1).
MOE_DEVINL int last_between(const int32_t *v, int lo, int hi, int t) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (ld_i32(v + mid) <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// A block a chunk of tokens, where a sequence may be counted by many.  A chunk of one sequence is a
// histogram; those of several look for each choice's sequence, and count in shared memory as long as
// that has a cell for each sequence and expert.
constexpr int kCells = kMaxE * kCols;
constexpr int kDeep = 4;  // choices of a thread at a time
__global__ void __launch_bounds__(kThreads)
seq_count_chunks_kernel(const SeqAuxArgs a, int chunk) {
  __shared__ int hist[kCells];
  __shared__ int s_n, s_b[2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t0 = blockIdx.x * chunk, t1 = min(a.T, t0 + chunk);
  for (int i = threadIdx.x; i < kCells; i += kThreads) hist[i] = 0;
  if (threadIdx.x == 0) s_n = 0;
  // (offsets, choices and mask are older than the kernel before this one, which clears counts)
  const int choices = (t1 - t0) * a.k;
  int e[kDeep], t[kDeep];
  bool live[kDeep];
  auto load = [&](int i0) {
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const int i = i0 + u * kThreads;
      t[u] = t0 + i / a.k;
      live[u] = i < choices && (a.mask == nullptr || ld_u8(a.mask + t[u]) != 0);
      e[u] = i < choices ? ld_i32(a.idx + (int64_t)t0 * a.k + i) : -1;
    }
  };
  load(threadIdx.x);
  if (warp < 2) {
    const int at = last_at_most(a.offsets, a.B + 1, warp == 0 ? t0 : t1 - 1, lane);
    if (lane == 0) s_b[warp] = at;
  }
  __syncthreads();
  const int b = s_b[0], last = s_b[1];
  if (last <= b) {
    if (b >= 0 && b < a.B) {
      Histogram h = {hist, a.E};
      int n = 0;
      for (int i0 = threadIdx.x; i0 < choices; i0 += kDeep * kThreads) {
        if (i0 >= kDeep * kThreads) load(i0);
#pragma unroll
        for (int u = 0; u < kDeep; ++u) {
          if (!live[u]) continue;
          h.add(e[u]);
          n += i0 + u * kThreads == (t[u] - t0) * a.k;
        }
      }
      n = warp_sum_i(n);
      if (lane == 0 && n > 0) atomicAdd(&s_n, n);
      __syncthreads();
      grid_dependency_wait();
      for (int e = threadIdx.x; e < a.E; e += kThreads) {
        const int c = h.total(e);
        if (c > 0) atomicAdd(a.counts + (int64_t)b * a.E + e, c);
      }
      if (threadIdx.x == 0 && s_n > 0) atomicAdd(a.tokens + b, s_n);
    }
    grid_dependency_begin();
    return;
  }
  const int cell_of = a.E + 1;  // a sequence's counts, and its tokens
  const bool shared = (int64_t)(last - b + 1) * cell_of <= kCells;
  if (!shared) grid_dependency_wait();
  for (int i0 = threadIdx.x; i0 < choices; i0 += kDeep * kThreads) {
    if (i0 >= kDeep * kThreads) load(i0);
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      if (!live[u]) continue;
      const int c = last_between(a.offsets, b, last + 1, t[u]);
      if (c < 0 || c >= a.B) continue;
      const bool counts = (uint32_t)e[u] < (uint32_t)a.E, first = i0 + u * kThreads == (t[u] - t0) * a.k;
      if (shared) {
        int *cell = hist + (c - b) * cell_of;
        if (counts) atomicAdd(cell + e[u], 1);
        if (first) atomicAdd(cell + a.E, 1);
      } else {
        if (counts) atomicAdd(a.counts + (int64_t)c * a.E + e[u], 1);
        if (first) atomicAdd(a.tokens + c, 1);
      }
    }
  }
  if (shared) {
    __syncthreads();
    grid_dependency_wait();
    for (int i = threadIdx.x; i < (last - b + 1) * cell_of; i += kThreads) {
      const int c = i / cell_of, e = i - c * cell_of, n = hist[i];
      if (n > 0) atomicAdd(e < a.E ? a.counts + (int64_t)(b + c) * a.E + e : a.tokens + b + c, n);
    }
  }
  grid_dependency_begin();
}

// (sequences with live tokens, live tokens) of the batch, in every thread.
MOE_DEVINL int2 batch_size(const int32_t *tokens, int B, int (*s)[kWarps]) {
  int S = 0, N = 0;
  for (int b = threadIdx.x; b < B; b += 4 * kThreads) {
    int n[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) n[u] = b + u * kThreads < B ? ld_i32(tokens + b + u * kThreads) : 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      S += n[u] > 0;
      N += n[u];
    }
  }
  S = warp_sum_i(S);
  N = warp_sum_i(N);
  const int lane = threadIdx.x & 31;
  if (lane == 0) {
    s[0][threadIdx.x >> 5] = S;
    s[1][threadIdx.x >> 5] = N;
  }
  __syncthreads();
  S = warp_sum_i(lane < kWarps ? s[0][lane] : 0);
  N = warp_sum_i(lane < kWarps ? s[1][lane] : 0);
  __syncthreads();
  return make_int2(S, N);
}

// 1 / v to within a bit
MOE_DEVINL float rcp_f(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

template <int LPT>
MOE_DEVINL float token_sum(float v) {
#pragma unroll
  for (int o = LPT / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int LPT>
MOE_DEVINL float token_max(float v) {
#pragma unroll
  for (int o = LPT / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// e^x of pairs, within |x| 2^-24 + 2^-22 of it (the product's rounding, and the power's); 0 from
// -88 on and of -inf, no number of NaN.  The product's error can be added back (three more
// instructions a pair: 65521 tokens of 256 experts 54.5 us, without 52), but is no larger than the
// power's own where logits lie within 4 of 0.
MOE_DEVINL uint64_t exp_near(uint64_t x) {
  float t0, t1, e0, e1;
  unpack2(mul2(x, pack2(1.44269502f, 1.44269502f)), t0, t1);
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(t0));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(t1));
  return pack2(e0, e1);
}

MOE_DEVINL float both(uint64_t v) {
  float lo, hi;
  unpack2(v, lo, hi);
  return lo + hi;
}

// A token's numbers, V experts a lane: u = e^(x - shift), s the score before it is normalised
// and j its derivative (softmax: u itself); their sums over the token's experts, and that of
// f s.
template <int V>
struct Token {
  uint64_t u[V / 2], s[V / 2], j[V / 2];
  float sum, size, fs, shift;
};

// Of logits x (-200: no expert, or a token that is not live).  No shift where the sum of e^x
// says that the largest logit is no further than 17 from 0 (tame_sum; one of +inf or NaN makes
// the sum so too, -inf adds 0): no maximum over the experts, and one exponential for the softmax
// and the sigmoid e^x / (1 + e^x).
MOE_DEVINL bool tame_sum(float sum) { return sum >= 1e-5f && sum <= 1e7f; }

template <int LPT, int V, bool SIGMOID>
MOE_DEVINL void token_scores(const float *x, const uint64_t *f, Token<V> &k) {
  uint64_t sum = 0, size = 0, fs = 0;
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    k.u[i] = exp_near(pack2(x[2 * i], x[2 * i + 1]));
    sum = add2(sum, k.u[i]);
    if (SIGMOID) {
      float a, b;
      unpack2(add2(k.u[i], pack2(1.0f, 1.0f)), a, b);
      const uint64_t r = pack2(rcp_f(a), rcp_f(b));
      k.s[i] = mul2(k.u[i], r);
      k.j[i] = mul2(k.s[i], r);
      size = add2(size, k.s[i]);
    } else {
      k.s[i] = k.j[i] = k.u[i];
    }
    fs = fma2(f[i], k.s[i], fs);
  }
  k.sum = token_sum<LPT>(both(sum));
  k.size = SIGMOID ? token_sum<LPT>(both(size)) : k.sum;
  k.fs = token_sum<LPT>(both(fs));
  k.shift = 0.0f;
}

// The same with the largest logit as the shift, for any logits.  (65521 tokens of 256 experts, all of
// them so: 101 us in all, where others take 52; with an exponential and a quotient each for u, s and
// 1 - s 219.)
template <int LPT, int V, bool SIGMOID>
MOE_DEVINL void token_scores_any(const float *x, const uint64_t *f, Token<V> &k) {
  float v[V], s[V], j[V], m = -INFINITY, sum = 0.0f, size = 0.0f, fs = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    v[i] = x[i] != x[i] ? -INFINITY : x[i];
    m = fmaxf(m, v[i]);
  }
  m = token_max<LPT>(m);
  k.shift = m > -INFINITY ? m : 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float u = expf(v[i] - k.shift);
    sum += u;
    s[i] = j[i] = u;
    if (SIGMOID) {
      // s and r = 1 - s; where every logit is under 0, s times e^-shift, which their quotients lose
      // again (so that logits whose sigmoids all vanish in fp32 keep their proportions)
      const float e = expf(-fabsf(v[i])), q = 1.0f / (1.0f + e), eq = e * q;
      const float r = v[i] < 0.0f ? q : eq;
      s[i] = k.shift < 0.0f ? u * q : v[i] < 0.0f ? eq : q;
      j[i] = s[i] * r;
      size += s[i];
    }
    float f0, f1;
    unpack2(f[i >> 1], f0, f1);
    fs = fmaf(i & 1 ? f1 : f0, s[i], fs);
    v[i] = u;
  }
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    k.u[i] = pack2(v[2 * i], v[2 * i + 1]);
    k.s[i] = pack2(s[2 * i], s[2 * i + 1]);
    k.j[i] = pack2(j[2 * i], j[2 * i + 1]);
  }
  k.sum = token_sum<LPT>(sum);
  k.size = SIGMOID ? token_sum<LPT>(size) : k.sum;
  k.fs = token_sum<LPT>(fs);
}

// A row's experts of a lane: columns 4 and 4 consecutive (VEC) or LPT apart.
template <int LPT, int V, bool VEC>
struct Columns {
  int l, E;
  MOE_DEVINL int at(int i) const { return VEC ? ((i >> 2) * LPT + l) * 4 + (i & 3) : i * LPT + l; }
  // the row into the thread's place of a stage, and back from there
  MOE_DEVINL void copy(float *place, const float *row) const {
    if (VEC) {
#pragma unroll
      for (int h = 0; h < V / 4; ++h)
        if (at(4 * h) < E)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                           (uint32_t)__cvta_generic_to_shared(place + h * (4 * kThreads) + 4 * threadIdx.x)),
                       "l"(row + at(4 * h))
                       : "memory");
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (at(i) < E)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                           (uint32_t)__cvta_generic_to_shared(place + i * kThreads + threadIdx.x)),
                       "l"(row + at(i))
                       : "memory");
    }
  }
  MOE_DEVINL void take(const float *place, float *x, bool on, float fill) const {
    if (VEC) {
#pragma unroll
      for (int h = 0; h < V / 4; ++h) {
        const float4 w = *reinterpret_cast<const float4 *>(place + h * (4 * kThreads) + 4 * threadIdx.x);
        const bool in = on && at(4 * h) < E;
        x[4 * h] = in ? w.x : fill;
        x[4 * h + 1] = in ? w.y : fill;
        x[4 * h + 2] = in ? w.z : fill;
        x[4 * h + 3] = in ? w.w : fill;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = on && at(i) < E ? place[i * kThreads + threadIdx.x] : fill;
    }
  }
  MOE_DEVINL void store(float *row, const float *x) const {
    if (VEC) {
#pragma unroll
      for (int h = 0; h < V / 4; ++h)
        if (at(4 * h) < E)
          st_v4(row + at(4 * h), make_uint4(__float_as_uint(x[4 * h]), __float_as_uint(x[4 * h + 1]),
                                            __float_as_uint(x[4 * h + 2]), __float_as_uint(x[4 * h + 3])));
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (at(i) < E) row[at(i)] = x[i];
    }
  }
};

// The loss of S sequences and N tokens.
MOE_DEVINL void write_loss(const SeqAuxArgs &a, float bal, float z, int S, int N) {
  a.loss[0] = a.coeff * bal / (float)max(S, 1);
  // (without a z loss the squares may have passed fp32's range)
  a.loss[1] = a.z_coeff != 0.0f ? a.z_coeff * z / (float)max(N, 1) : 0.0f;
}

// A small batch's counts and tokens, and zeros for P of sequences without live tokens, by one
// block; cell: kSmallCells words of its shared memory.
constexpr int kSmallCells = kWarps * kMaxE;
MOE_DEVINL void count_small(const SeqAuxArgs &a, int *cell) {
  const int cells = a.B * (a.E + 1);  // counts, then tokens
  int *tokens = cell + a.B * a.E;
  for (int i = threadIdx.x; i < cells; i += kThreads) cell[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * a.k; i += kThreads) {
    const int t = i / a.k, e = ld_i32(a.idx + i);
    if (a.mask != nullptr && ld_u8(a.mask + t) == 0) continue;
    const int b = last_between(a.offsets, -1, a.B + 1, t);
    if (b < 0 || b >= a.B) continue;
    if ((uint32_t)e < (uint32_t)a.E) atomicAdd(&cell[b * a.E + e], 1);
    if (i == t * a.k) atomicAdd(&tokens[b], 1);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < cells; i += kThreads) {
    if (i >= a.B * a.E) {
      a.tokens[i - a.B * a.E] = cell[i];
    } else {
      a.counts[i] = cell[i];
      if (tokens[i / a.E] == 0) a.probs[i] = 0.0f;
    }
  }
  __syncthreads();
}

// One pass over the logits: a token is LPT lanes of V experts each, a block takes `chunk`
// consecutive tokens in steps of kWarps * 32 / LPT.  A step's logits (and the gradients that
// are added to) come by asynchronous copies kAhead steps ahead, each lane's to a place of its
// own: a step's chain of sums and exponentials is 0.5 us long, a load's way as long again.
// A step that holds the end of a sequence is taken by both.  How the tokens are dealt out: a chunk
// a block, all to one block, or a sequence a block (and what lies before the first and behind
// the last sequence to two more).
enum { kChunks = 0, kOneBlock = 1, kSequences = 2 };
constexpr int kMaskTokens = 2048;  // of a block, kept in shared memory
constexpr int kManyEnds = 3;
constexpr int ahead_of(int v) { return v > 8 ? 2 : 4; }
template <int LPT, int V, bool VEC, bool SIGMOID>
__global__ void __launch_bounds__(kThreads, V > 8 ? 2 : 3)
seq_aux_kernel(const SeqAuxArgs a, int chunk, int mode, float *__restrict__ part,
               float2 *__restrict__ terms) {
  constexpr int kTok = 32 / LPT;  // tokens of a warp at a time
  constexpr int kStep = kWarps * kTok, kStage = V * kThreads, kAhead = ahead_of(V);
  extern __shared__ __align__(16) float ring[];  // logits [kAhead][kStage], then gradients
  __shared__ float s_p[V * kThreads];  // [kWarps][kMaxE] of sums, or [kStep][V * LPT] of probabilities
  __shared__ int s_seq[kStep];
  __shared__ float s_t[2][kWarps];
  __shared__ int s_n[2][kWarps];
  __shared__ uint8_t s_mask[kMaskTokens];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, grp = lane / LPT;
  const Columns<LPT, V, VEC> col = {lane % LPT, a.E};
  const bool sums = a.probs != nullptr, grad = a.d_logits != nullptr;
  const bool with_z = a.z_coeff != 0.0f, add = grad && a.accumulate;
  // Logits, offsets, mask and what is added to are older than the kernel before this one
  // where that is one of this call (it waited for them); the counts are not.
  if (!sums || mode == kOneBlock) grid_dependency_begin();
  int t0 = blockIdx.x * chunk, t1 = min(a.T, t0 + chunk);
  if (mode == kSequences) {
    const int q = blockIdx.x;
    t0 = q == a.B ? 0 : clampi(ld_i32(a.offsets + min(q, a.B)), 0, a.T);
    t1 = q > a.B ? a.T : clampi(ld_i32(a.offsets + (q == a.B ? 0 : q + 1)), t0, a.T);
  }
  const int mine = warp * kTok + grp;  // the lane's token of a step
  int ahead = 0;                       // the step that is copied next
  auto fetch = [&]() {
    const int u = t0 + ahead * kStep + mine;
    if (u < t1) {
      float *place = ring + (ahead % kAhead) * kStage;
      col.copy(place, a.logits + (int64_t)u * a.ld);
      if (add) col.copy(place + kAhead * kStage, a.d_logits + (int64_t)u * a.ld_d);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ++ahead;
  };
#pragma unroll
  for (int k = 0; k < kAhead; ++k) fetch();
  const bool masked = a.mask != nullptr, near_mask = t1 - t0 <= kMaskTokens;
  if (masked && near_mask)
    for (int i = threadIdx.x; i < t1 - t0; i += kThreads) s_mask[i] = (uint8_t)ld_u8(a.mask + t0 + i);
  if (mode == kOneBlock) count_small(a, reinterpret_cast<int *>(s_p));
  int b, next;
  if (mode == kSequences) {
    b = (int)blockIdx.x == a.B ? -1 : min((int)blockIdx.x, a.B);
    next = t1;
  } else {
    b = last_at_most(a.offsets, a.B + 1, t0, lane);
    next = b < a.B ? ld_i32(a.offsets + b + 1) : a.T;
  }
  if (sums && mode != kOneBlock) grid_dependency_begin();
  int2 sn = make_int2(0, 0);
  float per_seq = 0.0f, gz = 0.0f;
  if (grad || mode == kOneBlock) {
    sn = batch_size(a.tokens, a.B, s_n);
    per_seq = a.d_loss * a.coeff / (float)max(sn.x, 1);
    gz = a.d_loss * 2.0f * a.z_coeff / (float)max(sn.y, 1);
  }
  __syncthreads();
  if (mode == kSequences && sums && b >= 0 && b < a.B && ld_i32(a.tokens + b) <= 0)
    for (int e = threadIdx.x; e < a.E; e += kThreads) a.probs[(int64_t)b * a.E + e] = 0.0f;
  float z = 0.0f, bal = 0.0f;
  int step = 0;
  // what a token adds to the sums, and its gradient
  auto finish_token = [&](const uint64_t *f, uint64_t *acc2, float by_n, float g0, const Token<V> &k, int u,
                          bool valid, bool on, const float *place) {
    // (a token that is not live, or has no logit above -inf: p = 0 and no z)
    const bool some = k.sum > 0.0f;
    const float inv = k.size > 0.0f ? rcp_f(k.size) : 0.0f, c = k.fs * inv;
    const float lse = with_z && some ? k.shift + logf(k.sum) : 0.0f;
    if (sums) {
      const uint64_t inv2 = pack2(inv, inv);
#pragma unroll
      for (int i = 0; i < V / 2; ++i) acc2[i] = fma2(k.s[i], inv2, acc2[i]);
      if (col.l == 0) {
        z = fmaf(lse, lse, z);
        bal = fmaf(c, by_n, bal);
      }
    }
    if (grad && valid && (on || !add)) {
      // d = k1 j (f - c) + k2 u
      const float k1 = g0 * inv, k2 = some ? gz * lse * rcp_f(k.sum) : 0.0f;
      const float k0 = SIGMOID ? -c * k1 : fmaf(-c, k1, k2);
      const uint64_t k12 = pack2(k1, k1), k22 = pack2(k2, k2), k02 = pack2(k0, k0);
      float g[V];
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        uint64_t d = mul2(fma2(f[i], k12, k02), k.j[i]);
        if (SIGMOID) d = fma2(k.u[i], k22, d);
        unpack2(d, g[2 * i], g[2 * i + 1]);
      }
      if (add) {
        float old[V];
        col.take(place + kAhead * kStage, old, true, 0.0f);
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] += old[i];
      }
      col.store(a.d_logits + (int64_t)u * a.ld_d, g);
    }
  };
  for (int t = t0; t < t1;) {
    // Where a step holds the ends of several sequences they are taken at once, each token with the
    // numbers of its own: an end by itself costs a block 0.6 us (65521 tokens of 256 experts, 36
    // sequences of one token and a long one: 226 us, now 71)
    if (mode != kSequences && next <= t0 + (step + 1) * kStep && b + 1 < a.B &&
        ld_i32(a.offsets + b + 2) <= t0 + (step + 1) * kStep) {
      const int step_end = min(t1, t0 + (step + 1) * kStep), u = t0 + step * kStep + mine;
      const int last = last_at_most(a.offsets, a.B + 1, step_end, lane);
      const int end = last >= 0 ? min(ld_i32(a.offsets + last), step_end) : 0;
      if (last - b >= kManyEnds && end > t) {
        const int c = last_between(a.offsets, b, last + 1, u);
        const bool valid = u >= t && u < end;
        const int n = c >= 0 && c < a.B ? ld_i32(a.tokens + c) : 0;
        const float by_n = n > 0 ? 1.0f / (float)n : 0.0f;
        const float fs = (float)a.E / (float)a.k * by_n;
        if (col.l == 0) s_seq[mine] = valid && n > 0 ? c : -1;
        uint64_t f[V / 2], p2[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          float v[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int e = col.at(2 * i + h);
            v[h] = n > 0 && e < a.E ? fs * (float)ld_i32(a.counts + (int64_t)c * a.E + e) : 0.0f;
          }
          f[i] = pack2(v[0], v[1]);
          p2[i] = 0;
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
        const bool on = valid && n > 0 && (!masked || (near_mask ? s_mask[u - t0] : ld_u8(a.mask + u)) != 0);
        const float *place = ring + (step % kAhead) * kStage;
        float x[V];
        col.take(place, x, on, -200.0f);
        Token<V> k;
        token_scores<LPT, V, SIGMOID>(x, f, k);
        if (__any_sync(0xffffffffu, on && !tame_sum(k.sum))) {
          col.take(place, x, on, -INFINITY);
          token_scores_any<LPT, V, SIGMOID>(x, f, k);
        }
        finish_token(f, p2, by_n, per_seq * by_n, k, u, valid, on, place);
        if (sums) {
#pragma unroll
          for (int i = 0; i < V / 2; ++i) {
            float p0, p1;
            unpack2(p2[i], p0, p1);
            s_p[mine * (V * LPT) + col.at(2 * i)] = p0;
            s_p[mine * (V * LPT) + col.at(2 * i + 1)] = p1;
          }
          __syncthreads();
          // a sequence's sum by the thread that finds its first token
          for (int i = threadIdx.x; i < kStep * a.E; i += kThreads) {
            const int v = i / a.E, e = i - v * a.E, q = s_seq[v];
            if (q < 0 || (v > 0 && s_seq[v - 1] == q)) continue;
            float p = 0.0f;
            for (int w = v; w < kStep && s_seq[w] == q; ++w) p += s_p[w * (V * LPT) + e];
            if (mode != kChunks) a.probs[(int64_t)q * a.E + e] = p / (float)ld_i32(a.tokens + q);
            else part[((int64_t)blockIdx.x + q) * a.E + e] = p;
          }
          __syncthreads();
        }
        if (end == t0 + (step + 1) * kStep) {
          fetch();
          ++step;
        }
        t = end;
        b = last;
        next = b < a.B ? ld_i32(a.offsets + b + 1) : a.T;
        continue;
      }
    }
    const bool of_one = b >= 0 && b < a.B;
    const int n = of_one ? ld_i32(a.tokens + b) : 0;
    uint64_t f[V / 2], acc2[V / 2];
    int count[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
      count[i] = of_one && col.at(i) < a.E ? ld_i32(a.counts + (int64_t)b * a.E + col.at(i)) : 0;
    // where the next sequence ends, wanted after this one
    const int after = b + 1 < a.B ? ld_i32(a.offsets + b + 2) : a.T;
    const int end = min(t1, max(next, t + 1));
    const float by_n = n > 0 ? 1.0f / (float)n : 0.0f;
    const float g0 = per_seq * by_n, fs = (float)a.E / (float)a.k * by_n;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      f[i] = pack2(fs * (float)count[2 * i], fs * (float)count[2 * i + 1]);
      acc2[i] = 0;
    }
    auto finish = [&](const Token<V> &k, int u, bool valid, bool on, const float *place) {
      finish_token(f, acc2, by_n, g0, k, u, valid, on, place);
    };
    // the logits of the lane's token of this step, `fill` where it is not live or not of this sequence
    auto take = [&](float *x, float fill, int &u, bool &valid, const float *&place) -> bool {
      u = t0 + step * kStep + mine;
      valid = u >= t && u < end;
      bool on = valid && n > 0;
      if (masked && on) on = (near_mask ? s_mask[u - t0] : ld_u8(a.mask + u)) != 0;
      place = ring + (step % kAhead) * kStage;
      col.take(place, x, on, fill);
      return on;
    };
    // on to the next step, if this one ends before the sequence does
    auto onward = [&]() -> bool {
      if (t0 + (step + 1) * kStep > end && end < t1) return false;
      fetch();
      ++step;
      return t0 + step * kStep < end;
    };
    for (bool more = true; more;) {
      float x[V];
      int u;
      bool valid;
      const float *place;
      bool odd = false;
      while (more) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
        const bool on = take(x, -200.0f, u, valid, place);
        Token<V> k;
        token_scores<LPT, V, SIGMOID>(x, f, k);
        odd = __any_sync(0xffffffffu, on && !tame_sum(k.sum));
        if (odd) break;
        finish(k, u, valid, on, place);
        more = onward();
      }
      if (odd) {  // a step with such logits
        const bool on = take(x, -INFINITY, u, valid, place);
        Token<V> k;
        token_scores_any<LPT, V, SIGMOID>(x, f, k);
        finish(k, u, valid, on, place);
        more = onward();
      }
    }
    float acc[V];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) unpack2(acc2[i], acc[2 * i], acc[2 * i + 1]);
    if (sums && n > 0) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int o = LPT; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
        if (grp == 0 && col.at(i) < a.E) s_p[warp * kMaxE + col.at(i)] = acc[i];
      }
      __syncthreads();
      for (int e = threadIdx.x; e < a.E; e += kThreads) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += s_p[w * kMaxE + e];
        if (mode != kChunks) a.probs[(int64_t)b * a.E + e] = v * by_n;
        else part[((int64_t)blockIdx.x + b) * a.E + e] = v;
      }
      __syncthreads();
    }
    t = end;
    if (t < t1) {  // most often the next sequence
      if (t == next && after > t && b + 1 < a.B) {
        ++b;
        next = after;
      } else {
        b = last_at_most(a.offsets, a.B + 1, t, lane);
        next = b < a.B ? ld_i32(a.offsets + b + 1) : a.T;
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (!sums) return;
  z = warp_sum(z);
  bal = warp_sum(bal);
  if (lane == 0) {
    s_t[0][warp] = bal;
    s_t[1][warp] = z;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    bal = z = 0.0f;
    for (int w = 0; w < kWarps; ++w) {
      bal += s_t[0][w];
      z += s_t[1][w];
    }
    if (mode == kOneBlock) write_loss(a, bal, z, sn.x, sn.y);
    else terms[blockIdx.x] = make_float2(bal, z);
  }
}

// P of 32 experts of a sequence from its slots (block (b - first, group of 32)); the first block
// past the sequences adds up the loss.
constexpr int kFinishThreads = 512;  // at most
__global__ void __launch_bounds__(kFinishThreads)
seq_aux_finish_kernel(const SeqAuxArgs a, int first, int chunk, int blocks, const float *__restrict__ part,
                      const float2 *__restrict__ terms) {
  __shared__ float s[kFinishThreads / 32][33];
  __shared__ int s_n[2][kFinishThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, kW = blockDim.x >> 5;
  const int b = first + blockIdx.x, e = blockIdx.y * 32 + lane;
  grid_dependency_begin();
  if (b == a.B) {
    if (blockIdx.y > 0) return;
    float bal = 0.0f, z = 0.0f;
    int S = 0, N = 0;
    for (int i = threadIdx.x; i < blocks; i += blockDim.x) {
      bal += ld_f32(&terms[i].x);
      z += ld_f32(&terms[i].y);
    }
    for (int i = threadIdx.x; i < a.B; i += blockDim.x) {
      const int n = ld_i32(a.tokens + i);
      S += n > 0;
      N += n;
    }
    bal = warp_sum(bal);
    z = warp_sum(z);
    S = warp_sum_i(S);
    N = warp_sum_i(N);
    if (lane == 0) {
      s[warp][0] = bal;
      s[warp][1] = z;
      s_n[0][warp] = S;
      s_n[1][warp] = N;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      bal = z = 0.0f;
      S = N = 0;
      for (int w = 0; w < kW; ++w) {
        bal += s[w][0];
        z += s[w][1];
        S += s_n[0][w];
        N += s_n[1][w];
      }
      write_loss(a, bal, z, S, N);
    }
    return;
  }
  const int lo = clampi(ld_i32(a.offsets + b), 0, a.T);
  const int hi = clampi(ld_i32(a.offsets + b + 1), lo, a.T);
  const int n = ld_i32(a.tokens + b);
  float v = 0.0f;
  if (n > 0 && hi > lo && e < a.E) {
    const int i1 = min((hi - 1) / chunk, blocks - 1);
#pragma unroll 8
    for (int i = lo / chunk + warp; i <= i1; i += kW) v += ld_f32(part + ((int64_t)i + b) * a.E + e);
  }
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && e < a.E) {
    v = 0.0f;
    for (int w = 0; w < kW; ++w) v += s[w][lane];
    a.probs[(int64_t)b * a.E + e] = n > 0 ? v / (float)n : 0.0f;
  }
}

// Experts a lane, and lanes a token.  16 past 128 experts (half of a token's sums across lanes and
// of its scalars: 60000 tokens of 160 28.3 us in all, with eight 30.9); fewer experts gain nothing
// (64: 9.3 and 9.5) or lose (500 sequences of 262 tokens 27.9 and 25.5: longer steps, more of them cut).
int experts_per_lane(int E) { return E > 128 ? 16 : 8; }

int lanes_per_token(int E) {
  int l = 1;
  while (experts_per_lane(E) * l < E) l *= 2;
  return l;
}

int tokens_per_step(int E) { return kWarps * (32 / lanes_per_token(E)); }

// Blocks of the pass over the logits (one wave), and the tokens of each.
void split(int T, int E, int per_sm, int *blocks, int *chunk) {
  const int step = tokens_per_step(E);
  const int most = std::min(kMaxBlocks, per_sm * num_sms());
  const int64_t steps = ((int64_t)T + step - 1) / step;
  const int64_t each = std::max<int64_t>(1, (steps + most - 1) / most);
  *chunk = (int)(each * step);
  *blocks = (int)((steps + each - 1) / each);
}

// The workspace of a call (of the bytes that it is asked for, whatever its address).
struct Workspace : SeqAuxLayout {
  float *part;
  float2 *terms;
  Workspace(void *p, int T, int E, int B)
      : SeqAuxLayout(p, std::min<int64_t>(kMaxBlocks, ((int64_t)T + tokens_per_step(E) - 1) / tokens_per_step(E)),
                     E, B),
        part(static_cast<float *>(part_at)),
        terms(static_cast<float2 *>(terms_at)) {}
};

// Sequences of which a block each is worth its reading of every sequence's tokens; a shorter finish
// pays it back where there are many experts.  us in a graph, by sequences / by chunks, 145 tokens:
//   sequences              1024           4096          65536
//   8 experts, loss     11.2 / 12.4    25.5 / 21.6
//     gradient           7.1 / 5.9     21.1 / 6.6     1329 / 13
//     both at once      12.4 / 13.2    30.5 / 22.2    1236 / 199
//   256 experts, loss   13.3 / 21.9    32.5 / 51.9
//     gradient           7.6 / 5.6     21.0 / 6.7     1348 / 13
//     both at once      14.6 / 22.6    38.6 / 52.9    1598 / 645
// One limit for all three calls, so that the gradient by itself takes the loss's steps: a step with far
// logits is taken another way, which differs in the last bits.
int most_by_sequence(int E) { return std::max(1024, 16 * E); }

// How the tokens are dealt out.  One block takes the whole call where there are few logits, whose
// counts fit its shared memory (256 tokens of 8 experts 4.1 us in a graph, in three kernels 6.6;
// but 1000 of 16 11.4 and 7.7).  A block a sequence where these are shorter than half a step, none
// can be longer than 64 steps, and they are not too many (145 tokens of 16 experts in 273 sequences
// 8.2 us, by chunks 11.2).
int mode_of(const SeqAuxArgs &a) {
  const int step = tokens_per_step(a.E);
  if (a.loss != nullptr && a.T > 0 && (int64_t)a.T * a.E <= 8192 && a.T * a.k <= 4096 && a.B <= 8 &&
      a.B * (a.E + 1) <= kSmallCells)
    return kOneBlock;
  const bool short_ones = 2ll * a.T < (int64_t)a.B * step && a.T <= 64 * step;
  return short_ones && a.B <= most_by_sequence(a.E) ? kSequences : kChunks;
}

// The pass over the logits; its blocks and their tokens are left for the finish.
template <int LPT, int V, bool VEC, bool SIGMOID>
cudaError_t launch_pass(const SeqAuxArgs &a, const Workspace &w, int *blocks, int *chunk, cudaStream_t s) {
  constexpr auto kernel = seq_aux_kernel<LPT, V, VEC, SIGMOID>;
  constexpr size_t ring = sizeof(float) * ahead_of(V) * V * kThreads;
  struct Set {
    cudaError_t status;
    int per_sm[2];  // resident blocks, without and with gradients to add to
  };
  static PerDevice<Set> known;
  const Set set = known.get(current_device(), [] {
    Set v = {cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(2 * ring)), {1, 1}};
    for (int k = 0; k < 2 && v.status == cudaSuccess; ++k)
      v.status = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&v.per_sm[k], kernel, kThreads, (k + 1) * ring);
    return v;
  });
  if (set.status != cudaSuccess) return set.status;
  const int add = a.d_logits != nullptr && a.accumulate ? 1 : 0;
  const int mode = mode_of(a);
  split(a.T, a.E, std::max(1, set.per_sm[add]), blocks, chunk);
  if (mode == kOneBlock) {
    *blocks = 1;
    *chunk = a.T;
  } else if (mode == kSequences) {
    *blocks = a.B + 2;
  }
  return launch_dependent(kernel, *blocks, kThreads, (1 + add) * ring, s, a, *chunk, mode, w.part, w.terms);
}

template <int LPT, int V>
cudaError_t launch_pass(const SeqAuxArgs &a, const Workspace &w, int *blocks, int *chunk, cudaStream_t s) {
  auto whole = [](const float *p, int64_t ld) {
    return p == nullptr || ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 4 == 0);
  };
  const bool sigmoid = a.score_fn == MOE_SCORE_SIGMOID;
  if (a.E % 4 == 0 && whole(a.logits, a.ld) && whole(a.d_logits, a.ld_d))
    return sigmoid ? launch_pass<LPT, V, true, true>(a, w, blocks, chunk, s)
                   : launch_pass<LPT, V, true, false>(a, w, blocks, chunk, s);
  return sigmoid ? launch_pass<LPT, V, false, true>(a, w, blocks, chunk, s)
                 : launch_pass<LPT, V, false, false>(a, w, blocks, chunk, s);
}

cudaError_t launch_count(const SeqAuxArgs &a, cudaStream_t s) {
  const int64_t choices = (int64_t)a.T * a.k;
  // A block a sequence up to 2^15 choices: a launch and the atomics less, 1.3 to 2.4 us (8192 tokens of 4
  // choices, 64 even sequences 7.3 us in all, by chunks 9.0; all but a token each in one of them 21.4 and
  // 17.2).  The host does not see lengths, and what one long sequence of many choices would cost the
  // block that counts it grows with them (131072 tokens, 500 even sequences 18.6 and 21.3, one with most
  // of them 85 and 63; 128 sequences 16.2 and 18.1, 60 and 37): past that chunks, whose counts meet in
  // atomics, and for two or three sequences of some thousand tokens (8192 of 8 choices in 2 11.7 by chunks).
  const int64_t each = choices / a.B;
  if (choices <= (1 << 13) || (choices <= (1 << 15) && each <= (1 << 13)))
    return launch_dependent(seq_count_kernel, (unsigned)a.B, each <= 1024 ? 256 : kCountThreads, 0, s, a);
  const int64_t cells = (int64_t)a.B * (a.E + 1);
  const unsigned zero = (unsigned)std::min<int64_t>((cells + kThreads - 1) / kThreads, num_sms());
  const cudaError_t e = launch_dependent(seq_zero_kernel, zero, kThreads, 0, s, a);
  if (e != cudaSuccess) return e;
  // tokens of a block: 512 choices (2048: 55.5 us of 65521 tokens of 8, not 52.6), more where that is over four blocks a SM
  const int64_t most = 4ll * num_sms(), least = (512 + a.k - 1) / a.k;
  const int64_t chunk = std::max(least, (a.T + most - 1) / most);
  return launch_dependent(seq_count_chunks_kernel, (unsigned)((a.T + chunk - 1) / chunk), kThreads, 0, s,
                          a, (int)chunk);
}

}  // namespace

size_t seq_aux_workspace_bytes(int T, int E, int B) { return Workspace(nullptr, T, E, B).bytes; }

cudaError_t launch_seq_aux(const SeqAuxArgs &a, void *ws, cudaStream_t s) {
  const Workspace w(ws, a.T, a.E, a.B);
  cudaError_t e = cudaSuccess;
  const int mode = mode_of(a);
  if (a.loss != nullptr && mode != kOneBlock) e = launch_count(a, s);
  if (e != cudaSuccess) return e;
  int blocks = 0, chunk = 1;
  if (a.T > 0 && experts_per_lane(a.E) == 16) {
    e = launch_pass<16, 16>(a, w, &blocks, &chunk, s);
  } else if (a.T > 0) {
    switch (lanes_per_token(a.E)) {
      case 1: e = launch_pass<1, 8>(a, w, &blocks, &chunk, s); break;
      case 2: e = launch_pass<2, 8>(a, w, &blocks, &chunk, s); break;
      case 4: e = launch_pass<4, 8>(a, w, &blocks, &chunk, s); break;
      case 8: e = launch_pass<8, 8>(a, w, &blocks, &chunk, s); break;
      default: e = launch_pass<16, 8>(a, w, &blocks, &chunk, s); break;
    }
  }
  if (e != cudaSuccess || a.loss == nullptr || mode == kOneBlock) return e;
  if (mode == kSequences && a.T > 0)  // P is there
    return launch_dependent(seq_aux_finish_kernel, 1, kFinishThreads, 0, s, a, a.B, chunk, blocks, w.part, w.terms);
  // a sequence has blocks / B + 1 slots on average (but one may have nearly all: with 128 threads
  // 131072 tokens of which one of 500 sequences has most took 50 us, 36 with 256)
  const int threads = blocks / a.B < 4 ? 256 : kFinishThreads;
  return launch_dependent(seq_aux_finish_kernel, dim3((unsigned)a.B + 1, (unsigned)((a.E + 31) / 32)),
                          threads, 0, s, a, 0, chunk, blocks, w.part, w.terms);
}

}  // namespace moe

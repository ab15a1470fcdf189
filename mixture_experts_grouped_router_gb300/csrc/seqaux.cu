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
// Deterministic: integers are counted by atomics in shared memory, sums of floats are
// taken in a fixed order.  A block's tokens may lie in several sequences; its part of
// sequence b is slot (block + b) of the workspace: both grow along the tokens, one at
// least from part to part, so that no two parts share a slot.
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

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

MOE_DEVINL uint32_t cluster_size() {
  uint32_t v;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(v));
  return v;
}

MOE_DEVINL void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

MOE_DEVINL int ld_cluster(const int *p, uint32_t rank) {
  uint32_t a = (uint32_t)__cvta_generic_to_shared(p);
  int v;
  asm volatile("{\n\t.reg .b32 t;\n\tmapa.shared::cluster.u32 t, %1, %2;\n\t"
               "ld.shared::cluster.s32 %0, [t];\n\t}"
               : "=r"(v)
               : "r"(a), "r"(rank)
               : "memory");
  return v;
}

// counts[b, e] and tokens[b]: a cluster of blocks a sequence.  The histogram has a column a
// lane, so that a warp's choices of one expert do not meet in a bank.
__global__ void __launch_bounds__(kThreads)
seq_count_kernel(const SeqAuxArgs a, int32_t *__restrict__ done) {
  __shared__ int hist[kMaxE * 32];
  __shared__ int total[kMaxE + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cl = (int)cluster_size(), rank = (int)blockIdx.x % cl, b = (int)blockIdx.x / cl;
  for (int i = threadIdx.x; i < a.E * 32; i += kThreads) hist[i] = 0;
  if (threadIdx.x <= a.E) total[threadIdx.x] = 0;
  if (threadIdx.x == 0) total[a.E] = 0;
  __syncthreads();
  grid_dependency_begin();
  if (blockIdx.x == 0 && threadIdx.x == 0) *done = 0;
  const int lo = clampi(ld_i32(a.offsets + b), 0, a.T);
  const int hi = clampi(ld_i32(a.offsets + b + 1), lo, a.T);
  if (a.mask == nullptr) {
    const int64_t end = (int64_t)hi * a.k;
#pragma unroll 4
    for (int64_t i = (int64_t)lo * a.k + rank * kThreads + threadIdx.x; i < end; i += cl * kThreads) {
      const int e = ld_i32(a.idx + i);
      if ((uint32_t)e < (uint32_t)a.E) atomicAdd(&hist[e * 32 + lane], 1);
    }
    if (rank == 0 && threadIdx.x == 0) total[a.E] = hi - lo;
  } else {
    int n = 0;
    for (int t = lo + rank * kThreads + threadIdx.x; t < hi; t += cl * kThreads) {
      if (ld_u8(a.mask + t) == 0) continue;
      ++n;
      for (int j = 0; j < a.k; ++j) {
        const int e = ld_i32(a.idx + (int64_t)t * a.k + j);
        if ((uint32_t)e < (uint32_t)a.E) atomicAdd(&hist[e * 32 + lane], 1);
      }
    }
    n = warp_sum_i(n);
    if (lane == 0) atomicAdd(&total[a.E], n);
  }
  __syncthreads();
  for (int e = warp; e < a.E; e += kWarps) {
    const int n = warp_sum_i(hist[e * 32 + lane]);
    if (lane == 0) total[e] = n;
  }
  if (cl > 1) cluster_sync();
  else __syncthreads();
  if (rank == 0) {
    for (int e = threadIdx.x; e <= a.E; e += kThreads) {
      int n = total[e];
      for (int r = 1; r < cl; ++r) n += ld_cluster(&total[e], r);
      if (e < a.E) a.counts[(int64_t)b * a.E + e] = n;
      else a.tokens[b] = n;
    }
  }
  if (cl > 1) cluster_sync();  // the others' totals are read until here
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

// (sequences with live tokens, live tokens) of the batch, in every thread.
MOE_DEVINL int2 batch_size(const int32_t *tokens, int B, int (*s)[kWarps]) {
  int S = 0, N = 0;
  for (int b = threadIdx.x; b < B; b += kThreads) {
    const int n = ld_i32(tokens + b);
    S += n > 0;
    N += n;
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

// One pass over the logits: a token is LPT lanes of 8 experts each (4 + 4 consecutive ones
// where rows are 16-byte aligned), a block takes `chunk` consecutive tokens.
template <int LPT, bool VEC, bool SIGMOID>
__global__ void __launch_bounds__(kThreads)
seq_aux_kernel(const SeqAuxArgs a, int chunk, float *__restrict__ part, float *__restrict__ zpart) {
  constexpr int kTok = 32 / LPT;  // tokens of a warp at a time
  __shared__ float s_p[kWarps][kMaxE];
  __shared__ float s_z[kWarps];
  __shared__ int s_n[2][kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane % LPT, grp = lane / LPT;
  auto column = [&](int i) { return VEC ? ((i >> 2) * LPT + l) * 4 + (i & 3) : i * LPT + l; };
  const bool sums = a.probs != nullptr, grad = a.d_logits != nullptr;
  const bool with_soft = !SIGMOID || a.z_coeff != 0.0f;
  grid_dependency_begin();
  float per_seq = 0.0f, gz = 0.0f;
  if (grad) {
    const int2 sn = batch_size(a.tokens, a.B, s_n);
    per_seq = a.d_loss * a.coeff / (float)max(sn.x, 1);
    gz = a.d_loss * 2.0f * a.z_coeff / (float)max(sn.y, 1);
  }
  const int t0 = blockIdx.x * chunk, t1 = min(a.T, t0 + chunk);
  float z = 0.0f;
  for (int t = t0; t < t1;) {
    const int b = last_at_most(a.offsets, a.B + 1, t, lane);
    const int next = b < a.B ? ld_i32(a.offsets + b + 1) : a.T;
    const int end = min(t1, max(next, t + 1));
    const int n = b >= 0 && b < a.B ? ld_i32(a.tokens + b) : 0;
    float f[8], acc[8];
    float g0 = 0.0f;
    if (n > 0) g0 = per_seq / (float)n;
    const float fs = n > 0 ? (float)a.E / ((float)a.k * (float)n) : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = column(i);
      f[i] = n > 0 && grad && e < a.E ? fs * (float)ld_i32(a.counts + (int64_t)b * a.E + e) : 0.0f;
      acc[i] = 0.0f;
    }
    for (int u0 = t + warp * kTok; u0 < end; u0 += kWarps * kTok) {
      const int u = u0 + grp;
      const bool valid = u < end;
      const bool live = valid && n > 0 && (a.mask == nullptr || ld_u8(a.mask + u) != 0);
      const float *row = a.logits + (int64_t)u * a.ld;
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = -INFINITY;
      if (live) {
        if (VEC) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (column(4 * h) < a.E) {
              const uint4 w = ld_stream_v4(row + column(4 * h));
              x[4 * h] = __uint_as_float(w.x);
              x[4 * h + 1] = __uint_as_float(w.y);
              x[4 * h + 2] = __uint_as_float(w.z);
              x[4 * h + 3] = __uint_as_float(w.w);
            }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (column(i) < a.E) x[i] = ld_f32(row + column(i));
        }
      }
      float p[8], soft[8], jac[8], lse = 0.0f;
      if (with_soft) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (x[i] != x[i]) x[i] = -INFINITY;  // NaN ranks below every number
          m = fmaxf(m, x[i]);
        }
        m = token_max<LPT>(m);
        // a token without a logit above -inf (or not live) has p = 0 and no z
        const bool some = m > -INFINITY;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          soft[i] = some ? expf(x[i] - m) : 0.0f;
          sum += soft[i];
        }
        sum = token_sum<LPT>(sum);
        const float inv = some ? 1.0f / sum : 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) soft[i] *= inv;
        if (some) lse = m + logf(sum);
      }
      if (SIGMOID) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          p[i] = x[i] == x[i] ? 1.0f / (1.0f + expf(-x[i])) : 0.0f;
          sum += p[i];
        }
        sum = token_sum<LPT>(sum);
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          jac[i] = p[i] * (1.0f - p[i]) * inv;
          p[i] *= inv;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = jac[i] = soft[i];
      }
      if (sums) {
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += p[i];
        if (l == 0) z = fmaf(lse, lse, z);
      }
      if (grad) {
        float c = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) c = fmaf(f[i], p[i], c);
        c = token_sum<LPT>(c);
        const float zl = gz * lse;
        float g[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          g[i] = g0 * jac[i] * (f[i] - c);
          if (with_soft) g[i] = fmaf(zl, soft[i], g[i]);
          if (!live) g[i] = 0.0f;
        }
        if (valid && !(a.accumulate && !live)) {
          float *out = a.d_logits + (int64_t)u * a.ld_d;
          if (VEC) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (column(4 * h) < a.E) {
                float *o = out + column(4 * h);
                if (a.accumulate) {
                  const uint4 w = ld_stream_v4(o);
                  g[4 * h] += __uint_as_float(w.x);
                  g[4 * h + 1] += __uint_as_float(w.y);
                  g[4 * h + 2] += __uint_as_float(w.z);
                  g[4 * h + 3] += __uint_as_float(w.w);
                }
                st_v4(o, make_uint4(__float_as_uint(g[4 * h]), __float_as_uint(g[4 * h + 1]),
                                    __float_as_uint(g[4 * h + 2]), __float_as_uint(g[4 * h + 3])));
              }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (column(i) < a.E) out[column(i)] = a.accumulate ? out[column(i)] + g[i] : g[i];
          }
        }
      }
    }
    if (sums && n > 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int o = LPT; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
        if (grp == 0 && column(i) < a.E) s_p[warp][column(i)] = acc[i];
      }
      __syncthreads();
      for (int e = threadIdx.x; e < a.E; e += kThreads) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += s_p[w][e];
        part[((int64_t)blockIdx.x + b) * a.E + e] = v;
      }
      __syncthreads();
    }
    t = end;
  }
  if (!sums) return;
  z = warp_sum(z);
  if (lane == 0) s_z[warp] = z;
  __syncthreads();
  if (threadIdx.x == 0) {
    float v = 0.0f;
    for (int w = 0; w < kWarps; ++w) v += s_z[w];
    zpart[blockIdx.x] = v;
  }
}

// P of 32 experts of a sequence from its slots, and its part of the loss; the last block
// of the grid adds the parts up.
__global__ void __launch_bounds__(kThreads)
seq_aux_finish_kernel(const SeqAuxArgs a, int chunk, int blocks, const float *__restrict__ part,
                      const float *__restrict__ zpart, float *__restrict__ terms,
                      int32_t *__restrict__ done) {
  __shared__ float s[kWarps][33];
  __shared__ int s_n[2][kWarps];
  __shared__ int s_last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.x, e = blockIdx.y * 32 + lane;
  grid_dependency_begin();
  const int lo = clampi(ld_i32(a.offsets + b), 0, a.T);
  const int hi = clampi(ld_i32(a.offsets + b + 1), lo, a.T);
  const int n = ld_i32(a.tokens + b);
  float v = 0.0f;
  if (n > 0 && hi > lo && e < a.E) {
    const int i1 = min((hi - 1) / chunk, blocks - 1);
#pragma unroll 4
    for (int i = lo / chunk + warp; i <= i1; i += kWarps)
      v += ld_f32(part + ((int64_t)i + b) * a.E + e);
  }
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0) {
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += s[w][lane];
    const float P = n > 0 ? v / (float)n : 0.0f;
    float term = 0.0f;
    if (e < a.E) {
      a.probs[(int64_t)b * a.E + e] = P;
      if (n > 0)
        term = (float)a.E * (float)ld_i32(a.counts + (int64_t)b * a.E + e) /
               ((float)a.k * (float)n) * P;
    }
    term = warp_sum(term);
    if (lane == 0) {
      terms[(int64_t)b * gridDim.y + blockIdx.y] = term;
      __threadfence();
      s_last = atomicAdd(done, 1) == (int)(gridDim.x * gridDim.y) - 1;
    }
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  const int2 sn = batch_size(a.tokens, a.B, s_n);
  const int64_t n_terms = (int64_t)gridDim.x * gridDim.y;
  float bal = 0.0f, z = 0.0f;
  for (int64_t i = threadIdx.x; i < n_terms; i += kThreads) bal += ld_f32(terms + i);
  for (int i = threadIdx.x; i < blocks; i += kThreads) z += ld_f32(zpart + i);
  bal = warp_sum(bal);
  z = warp_sum(z);
  if (lane == 0) {
    s[0][warp] = bal;
    s[1][warp] = z;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    bal = z = 0.0f;
    for (int w = 0; w < kWarps; ++w) {
      bal += s[0][w];
      z += s[1][w];
    }
    a.loss[0] = a.coeff * bal / (float)max(sn.x, 1);
    // (without a z loss the squares may have passed fp32's range)
    a.loss[1] = a.z_coeff != 0.0f ? a.z_coeff * z / (float)max(sn.y, 1) : 0.0f;
  }
}

int lanes_per_token(int E) {
  int l = 1;
  while (8 * l < E) l *= 2;
  return l;
}

// Blocks of the pass over the logits (one wave), and the tokens of each.
void split(int T, int E, int *blocks, int *chunk) {
  const int step = kWarps * (32 / lanes_per_token(E));
  const int most = std::min(kMaxBlocks, 4 * num_sms());
  const int64_t steps = ((int64_t)T + step - 1) / step;
  const int64_t each = std::max<int64_t>(1, (steps + most - 1) / most);
  *chunk = (int)(each * step);
  *blocks = (int)((steps + each - 1) / each);
}

struct Workspace {
  float *part, *zpart, *terms;
  int32_t *done;
  size_t bytes;
  Workspace(void *p, int T, int E, int B) {
    const int step = kWarps * (32 / lanes_per_token(E));
    const size_t blocks = (size_t)std::min<int64_t>(kMaxBlocks, ((int64_t)T + step - 1) / step);
    done = static_cast<int32_t *>(p);
    zpart = reinterpret_cast<float *>(done + 4);
    terms = zpart + blocks;
    part = terms + (size_t)B * ((E + 31) / 32);
    bytes = 16 + 4 * (blocks + (size_t)B * ((E + 31) / 32) + (blocks + (size_t)B) * (size_t)E);
  }
};

template <int LPT, bool VEC>
cudaError_t launch_pass(const SeqAuxArgs &a, int blocks, int chunk, float *part, float *zpart,
                        cudaStream_t s) {
  return a.score_fn == MOE_SCORE_SIGMOID
             ? launch_dependent(seq_aux_kernel<LPT, VEC, true>, blocks, kThreads, 0, s, a, chunk, part, zpart)
             : launch_dependent(seq_aux_kernel<LPT, VEC, false>, blocks, kThreads, 0, s, a, chunk, part, zpart);
}

template <int LPT>
cudaError_t launch_pass(const SeqAuxArgs &a, int blocks, int chunk, float *part, float *zpart,
                        cudaStream_t s) {
  auto whole = [](const float *p, int64_t ld) {
    return p == nullptr || ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 4 == 0);
  };
  const bool vec = a.E % 4 == 0 && whole(a.logits, a.ld) && whole(a.d_logits, a.ld_d);
  return vec ? launch_pass<LPT, true>(a, blocks, chunk, part, zpart, s)
             : launch_pass<LPT, false>(a, blocks, chunk, part, zpart, s);
}

cudaError_t launch_count(const SeqAuxArgs &a, int32_t *done, cudaStream_t s) {
  // A sequence's choices are counted by one block, by eight where it has (or, the batch
  // being large, one of them may have) many.
  const int64_t choices = (int64_t)a.T * a.k;
  const unsigned cl = choices / a.B >= 4096 || choices >= (1 << 18) ? 8 : 1;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cl;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cl * (unsigned)a.B);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, seq_count_kernel, a, done);
}

}  // namespace

size_t seq_aux_workspace_bytes(int T, int E, int B) { return Workspace(nullptr, T, E, B).bytes; }

cudaError_t launch_seq_aux(const SeqAuxArgs &a, void *ws, cudaStream_t s) {
  const Workspace w(ws, a.T, a.E, a.B);
  cudaError_t e = cudaSuccess;
  if (a.idx != nullptr || a.loss != nullptr) e = launch_count(a, w.done, s);
  if (e != cudaSuccess) return e;
  int blocks, chunk;
  split(a.T, a.E, &blocks, &chunk);
  if (blocks > 0 && (a.probs != nullptr || a.d_logits != nullptr)) {
    switch (lanes_per_token(a.E)) {
      case 1: e = launch_pass<1>(a, blocks, chunk, w.part, w.zpart, s); break;
      case 2: e = launch_pass<2>(a, blocks, chunk, w.part, w.zpart, s); break;
      case 4: e = launch_pass<4>(a, blocks, chunk, w.part, w.zpart, s); break;
      case 8: e = launch_pass<8>(a, blocks, chunk, w.part, w.zpart, s); break;
      case 16: e = launch_pass<16>(a, blocks, chunk, w.part, w.zpart, s); break;
      default: e = launch_pass<32>(a, blocks, chunk, w.part, w.zpart, s); break;
    }
    if (e != cudaSuccess) return e;
  }
  if (a.loss == nullptr) return cudaSuccess;
  return launch_dependent(seq_aux_finish_kernel, dim3((unsigned)a.B, (unsigned)((a.E + 31) / 32)),
                          kThreads, 0, s, a, chunk, blocks, w.part, w.zpart, w.terms, w.done);
}

}  // namespace moe

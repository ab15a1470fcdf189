// The norm of all gradients together, and their clipping.
//
//     norm = scale sqrt(sum over tensors and elements of g^2)
//     out  = g scale min(1, max_norm / (norm + 1e-6))     (in place where out is g)
// A plan of chunks (pieces of tensors of a few thousand elements, made once by the host)
// tells the warps what to read: tensors of any number, size, type and alignment are one
// launch.  The first kernel writes a sum a block, the second adds these up again in every
// block (the same order, so the same number) and scales.  It walks the chunks from the last
// one back: what the first one read last is still in L2.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

MOE_DEVINL ClipChunk load_chunk(const ClipChunk *p) {
  ClipChunk c;
  asm volatile("ld.global.v2.u64 {%0, %1}, [%2];" : "=l"(c.g), "=l"(c.out) : "l"(p) : "memory");
  asm volatile("ld.global.v2.s32 {%0, %1}, [%2];" : "=r"(c.n), "=r"(c.kind) : "l"(&p->n) : "memory");
  return c;
}

// A type's 8 consecutive elements, in one access (32 bytes of fp32).
struct Bf16x8 {
  using Elem = uint16_t;
  static constexpr int kU = 8;  // vectors in flight: 128 bytes a lane
  uint4 a;
  MOE_DEVINL void zero() { a = make_uint4(0, 0, 0, 0); }
  MOE_DEVINL void load(const uint16_t *p) { a = ld_stream_v4(p); }
  MOE_DEVINL void get(float *v) const { bf16x8_to_f32(a, v); }
  MOE_DEVINL static float one(const uint16_t *p) { return __uint_as_float(ld_u16(p) << 16); }
  MOE_DEVINL static void store(uint16_t *p, const float *v) { st_v4(p, f32_to_bf16x8(v)); }
  MOE_DEVINL static void store_one(uint16_t *p, float v) {
    *reinterpret_cast<bf16_t *>(p) = __float2bfloat16_rn(v);
  }
};

struct F32x8 {
  using Elem = float;
  static constexpr int kU = 4;
  float f[8];
  MOE_DEVINL void zero() {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 0.0f;
  }
  MOE_DEVINL void load(const float *p) { ld_stream_f32x8(p, f); }
  MOE_DEVINL void get(float *v) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = f[i];
  }
  MOE_DEVINL static float one(const float *p) { return ld_f32(p); }
  MOE_DEVINL static void store(float *p, const float *v) { st_f32x8(p, v); }
  MOE_DEVINL static void store_one(float *p, float v) { *p = v; }
};

// Values whose squares leave fp32's range are squared in 64 bits.  That is looked at for
// 32 or 64 values at a time, by their fp32 sum: one that is neither 0 nor in the range's
// middle, where squares that vanish are nothing beside it.  (64-bit additions are slow on
// GB300: one for every 8 values took 0.3 ms of 1.4 G values.)
MOE_DEVINL bool in_range(float s) { return s >= 1e-28f && s <= 1e37f; }

template <typename V>
MOE_DEVINL double square_sum_64(const V *raw) {
  double s = 0.0;
  for (int u = 0; u < V::kU; ++u) {
    float v[8];
    raw[u].get(v);
    for (int i = 0; i < 8; ++i) s += (double)v[i] * (double)v[i];
  }
  return s;
}

// The warp's lanes' sums of squares of a chunk, added to acc.
template <typename V>
MOE_DEVINL void chunk_squares(const ClipChunk &c, int lane, double &acc) {
  const typename V::Elem *g = static_cast<const typename V::Elem *>(c.g);
  int i = 0;
  if (!(c.kind & 4)) {
    for (; i + 8 <= c.n; i += 256 * V::kU) {
      V raw[V::kU];
#pragma unroll
      for (int u = 0; u < V::kU; ++u) {
        const int j = i + 256 * u + 8 * lane;
        raw[u].zero();
        if (j + 8 <= c.n) raw[u].load(g + j);
      }
      float s[2] = {0.0f, 0.0f}, any = 0.0f;
#pragma unroll
      for (int u = 0; u < V::kU; ++u) {
        float v[8];
        raw[u].get(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e & 1] = fmaf(v[e], v[e], s[e & 1]);
      }
      const float sum = s[0] + s[1];
      if (in_range(sum)) {
        acc += (double)sum;
      } else {
#pragma unroll
        for (int u = 0; u < V::kU; ++u) {
          float v[8];
          raw[u].get(v);
#pragma unroll
          for (int e = 0; e < 8; ++e) any = v[e] != 0.0f ? 1.0f : any;
        }
        if (any != 0.0f) acc += square_sum_64(raw);
      }
    }
    i = c.n & ~7;
  }
  for (i += lane; i < c.n; i += 32) {
    const double v = (double)V::one(g + i);
    acc += v * v;
  }
}

// Sum over the block's threads, in thread 0's warp (64-bit additions being slow, by few).
MOE_DEVINL double block_sum(double v, double *s) {
  s[threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.x >= 32) return 0.0;
  v = 0.0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) v += s[w * 32 + threadIdx.x];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__global__ void __launch_bounds__(kThreads, 4)
grad_square_kernel(const ClipChunk *__restrict__ plan, int64_t chunks, double *__restrict__ part) {
  __shared__ double s[kThreads];
  const int lane = threadIdx.x & 31;
  const int64_t step = (int64_t)gridDim.x * kWarps;
  int64_t at = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  double acc = 0.0;
  grid_dependency_begin();
  ClipChunk c = {};
  if (at < chunks) c = load_chunk(plan + at);
  while (at < chunks) {
    at += step;
    ClipChunk next = {};
    if (at < chunks) next = load_chunk(plan + at);  // on its way while this one is summed
    if (c.kind & 1) chunk_squares<F32x8>(c, lane, acc);
    else chunk_squares<Bf16x8>(c, lane, acc);
    c = next;
  }
  acc = block_sum(acc, s);
  if (threadIdx.x == 0) part[blockIdx.x] = acc;
}

// Sum of the blocks' parts, in thread 0.
MOE_DEVINL double total_of(const double *part, int parts, double *s) {
  double v = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) {
    double p;
    asm volatile("ld.global.f64 %0, [%1];" : "=d"(p) : "l"(part + i) : "memory");
    v += p;
  }
  return block_sum(v, s);
}

template <typename V, typename O>
MOE_DEVINL void chunk_scale(const ClipChunk &c, int lane, float f) {
  constexpr int kU = 4;
  const typename V::Elem *g = static_cast<const typename V::Elem *>(c.g);
  typename O::Elem *out = static_cast<typename O::Elem *>(c.out);
  int i = 0;
  if (!(c.kind & 4)) {
    for (; i + 8 <= c.n; i += 256 * kU) {
      V raw[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int j = i + 256 * u + 8 * lane;
        if (j + 8 <= c.n) raw[u].load(g + j);
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int j = i + 256 * u + 8 * lane;
        if (j + 8 > c.n) continue;
        float v[8];
        raw[u].get(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= f;
        O::store(out + j, v);
      }
    }
    i = c.n & ~7;
  }
  for (i += lane; i < c.n; i += 32) O::store_one(out + i, V::one(g + i) * f);
}

__global__ void __launch_bounds__(kThreads, 4)
grad_scale_kernel(const ClipChunk *__restrict__ plan, int64_t chunks, const double *__restrict__ part,
                  int parts, float scale, float max_norm, float *__restrict__ norm) {
  __shared__ double s[kThreads];
  __shared__ float s_f;
  const int lane = threadIdx.x & 31;
  const int64_t step = (int64_t)gridDim.x * kWarps;
  int64_t k = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  // the plan is older than the kernel before this one
  ClipChunk c = {};
  if (k < chunks) c = load_chunk(plan + (chunks - 1 - k));
  grid_dependency_begin();
  const double sum = total_of(part, parts, s);
  if (threadIdx.x == 0) {
    const double total = (double)scale * sqrt(sum);
    if (blockIdx.x == 0) *norm = (float)total;
    // a norm that is no number, or infinite, clips nothing
    const double q = (double)max_norm / (total + 1e-6);
    s_f = total <= 1.7e308 && q < 1.0 ? (float)((double)scale * q) : scale;
  }
  __syncthreads();
  const float f = s_f;
  while (k < chunks) {
    k += step;
    ClipChunk next = {};
    if (k < chunks) next = load_chunk(plan + (chunks - 1 - k));
    if (f != 1.0f || c.g != c.out) {
      switch (c.kind & 3) {
        case 0: chunk_scale<Bf16x8, Bf16x8>(c, lane, f); break;
        case 1: chunk_scale<F32x8, Bf16x8>(c, lane, f); break;
        case 2: chunk_scale<Bf16x8, F32x8>(c, lane, f); break;
        default: chunk_scale<F32x8, F32x8>(c, lane, f); break;
      }
    }
    c = next;
  }
}

__global__ void __launch_bounds__(kThreads)
grad_norm_kernel(const double *__restrict__ part, int parts, float scale, float *__restrict__ norm) {
  __shared__ double s[kThreads];
  grid_dependency_begin();
  const double sum = total_of(part, parts, s);
  if (threadIdx.x == 0) *norm = (float)((double)scale * sqrt(sum));
}

}  // namespace

cudaError_t launch_clip(const ClipChunk *plan, int64_t chunks, float scale, float max_norm, bool write,
                        float *norm, double *part, cudaStream_t st) {
  auto grid = [&](int per_sm) {
    const int64_t want = std::max<int64_t>(1, (chunks + kWarps - 1) / kWarps);
    return (int)std::min<int64_t>({want, (int64_t)num_sms() * per_sm, (int64_t)kClipMaxBlocks});
  };
  const int parts = grid(blocks_per_sm<grad_square_kernel>(kThreads));
  cudaError_t e = launch_dependent(grad_square_kernel, parts, kThreads, 0, st, plan, chunks, part);
  if (e != cudaSuccess) return e;
  if (!write) return launch_dependent(grad_norm_kernel, 1, kThreads, 0, st, part, parts, scale, norm);
  return launch_dependent(grad_scale_kernel, grid(blocks_per_sm<grad_scale_kernel>(kThreads)), kThreads,
                          0, st, plan, chunks, part, parts, scale, max_norm, norm);
}

}  // namespace moe

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

// Values whose squares leave fp32's range are squared in 64 bits; that is looked at
// for 32 values at a time (a sum that is neither 0 nor in the range's middle).
MOE_DEVINL bool in_range(float s) { return s >= 1e-28f && s <= 1e37f; }

MOE_DEVINL double square_sum(const float *v, int n) {
  double s = 0.0;
  for (int i = 0; i < n; ++i) s += (double)v[i] * (double)v[i];
  return s;
}

template <int N>
MOE_DEVINL void add_squares(const float *v, double &acc) {
  float a = 0.0f, b = 0.0f;
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    a = fmaf(v[i], v[i], a);
    b = fmaf(v[i + 1], v[i + 1], b);
  }
  const float s = a + b;
  if (in_range(s)) {
    acc += (double)s;
    return;
  }
  bool any = false;
#pragma unroll
  for (int i = 0; i < N; ++i) any |= v[i] != 0.0f;
  if (any) acc += square_sum(v, N);
}

MOE_DEVINL float load_one(const ClipChunk &c, int i) {
  return c.kind & 1 ? ld_f32(static_cast<const float *>(c.g) + i)
                    : __uint_as_float(ld_u16(static_cast<const uint16_t *>(c.g) + i) << 16);
}

// 8 elements from i on.
MOE_DEVINL void load_raw(const ClipChunk &c, int i, uint4 &a, uint4 &b) {
  if (c.kind & 1) {
    a = ld_stream_v4(static_cast<const float *>(c.g) + i);
    b = ld_stream_v4(static_cast<const float *>(c.g) + i + 4);
  } else {
    a = ld_stream_v4(static_cast<const uint16_t *>(c.g) + i);
  }
}

MOE_DEVINL void values8(int kind, const uint4 &a, const uint4 &b, float *v) {
  if (kind & 1) {
    const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(u[i]);
  } else {
    bf16x8_to_f32(a, v);
  }
}

constexpr int kU = 4;  // vectors of 8 in flight

__global__ void __launch_bounds__(kThreads)
grad_square_kernel(const ClipChunk *__restrict__ plan, int64_t chunks, double *__restrict__ part) {
  __shared__ double s[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  double acc = 0.0;
  grid_dependency_begin();
  for (int64_t at = (int64_t)blockIdx.x * kWarps + warp; at < chunks; at += (int64_t)gridDim.x * kWarps) {
    const ClipChunk c = load_chunk(plan + at);
    int i = 0;
    if (!(c.kind & 4)) {
      for (; i + 8 <= c.n; i += 256 * kU) {
        uint4 a[kU], b[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int j = i + 256 * u + 8 * lane;
          a[u] = b[u] = make_uint4(0, 0, 0, 0);
          if (j + 8 <= c.n) load_raw(c, j, a[u], b[u]);
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          float v[8];
          values8(c.kind, a[u], b[u], v);
          add_squares<8>(v, acc);
        }
      }
      i = c.n & ~7;
    }
    for (i += lane; i < c.n; i += 32) {
      const double v = (double)load_one(c, i);
      acc += v * v;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if (lane == 0) s[warp] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    acc = 0.0;
    for (int w = 0; w < kWarps; ++w) acc += s[w];
    part[blockIdx.x] = acc;
  }
}

// Sum of the blocks' parts, the same in every thread.
MOE_DEVINL double total_of(const double *part, int parts, double *s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  double v = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) {
    double p;
    asm volatile("ld.global.f64 %0, [%1];" : "=d"(p) : "l"(part + i) : "memory");
    v += p;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0) s[warp] = v;
  __syncthreads();
  v = 0.0;
  for (int w = 0; w < kWarps; ++w) v += s[w];
  return v;
}

__global__ void __launch_bounds__(kThreads)
grad_scale_kernel(const ClipChunk *__restrict__ plan, int64_t chunks, const double *__restrict__ part,
                  int parts, float scale, float max_norm, float *__restrict__ norm) {
  __shared__ double s[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dependency_begin();
  const double total = (double)scale * sqrt(total_of(part, parts, s));
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)total;
  // a norm that is no number, or infinite, clips nothing
  const double q = (double)max_norm / (total + 1e-6);
  const float c = total <= 1.7e308 && q < 1.0 ? (float)((double)scale * q) : scale;
  for (int64_t k = (int64_t)blockIdx.x * kWarps + warp; k < chunks; k += (int64_t)gridDim.x * kWarps) {
    const ClipChunk ch = load_chunk(plan + (chunks - 1 - k));
    if (c == 1.0f && ch.g == ch.out) continue;
    int i = 0;
    if (!(ch.kind & 4)) {
      for (; i + 8 <= ch.n; i += 256 * kU) {
        uint4 a[kU], b[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int j = i + 256 * u + 8 * lane;
          if (j + 8 <= ch.n) load_raw(ch, j, a[u], b[u]);
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int j = i + 256 * u + 8 * lane;
          if (j + 8 > ch.n) continue;
          float v[8];
          values8(ch.kind, a[u], b[u], v);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] *= c;
          if (ch.kind & 2) {
            float *o = static_cast<float *>(ch.out) + j;
            st_v4(o, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                __float_as_uint(v[3])));
            st_v4(o + 4, make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]),
                                    __float_as_uint(v[6]), __float_as_uint(v[7])));
          } else {
            st_v4(static_cast<uint16_t *>(ch.out) + j, f32_to_bf16x8(v));
          }
        }
      }
      i = ch.n & ~7;
    }
    for (i += lane; i < ch.n; i += 32) {
      const float v = load_one(ch, i) * c;
      if (ch.kind & 2) static_cast<float *>(ch.out)[i] = v;
      else static_cast<bf16_t *>(ch.out)[i] = __float2bfloat16_rn(v);
    }
  }
}

__global__ void __launch_bounds__(kThreads)
grad_norm_kernel(const double *__restrict__ part, int parts, float scale, float *__restrict__ norm) {
  __shared__ double s[kWarps];
  grid_dependency_begin();
  const double total = (double)scale * sqrt(total_of(part, parts, s));
  if (threadIdx.x == 0) *norm = (float)total;
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

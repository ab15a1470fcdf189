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
  uint4 a;
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
  float f[8];
  MOE_DEVINL void load(const float *p) { ld_stream_f32x8(p, f); }
  MOE_DEVINL void get(float *v) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = f[i];
  }
  MOE_DEVINL static float one(const float *p) { return ld_f32(p); }
  MOE_DEVINL static void store(float *p, const float *v) { st_f32x8(p, v); }
  MOE_DEVINL static void store_one(float *p, float v) { *p = v; }
};

// Squares are summed from pieces of 16 bytes, kPieces a lane at a time, copied to shared
// memory kAhead times ahead (each lane reads what it copied: no barrier).
constexpr int kPieces = 8;
constexpr int kAhead = 3;
constexpr int kSquareSmem = kAhead * kPieces * 16 * kThreads;

// Values whose squares leave fp32's range are squared in 64 bits.  That is looked at for 32
// or 64 values at a time, by their fp32 sum: one that is neither 0 nor in the range's
// middle, where squares that vanish are nothing beside it.  (64-bit additions are slow on
// GB300: one for every 8 values took 0.1 ms of 1.4 G values.)
MOE_DEVINL bool in_range(float s) { return s >= 1e-28f && s <= 1e37f; }

MOE_DEVINL int values(const uint4 &w, bool f32, float *v) {
  if (!f32) {
    bf16x8_to_f32(w, v);
    return 8;
  }
  v[0] = __uint_as_float(w.x);
  v[1] = __uint_as_float(w.y);
  v[2] = __uint_as_float(w.z);
  v[3] = __uint_as_float(w.w);
  return 4;
}

template <bool F32>
MOE_DEVINL void add_squares(const uint8_t *mine, double &acc) {
  constexpr int kN = F32 ? 4 : 8;
  float s[2] = {0.0f, 0.0f};
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    float v[8];
    values(*reinterpret_cast<const uint4 *>(mine + u * (16 * kThreads)), F32, v);
#pragma unroll
    for (int e = 0; e < kN; ++e) s[e & 1] = fmaf(v[e], v[e], s[e & 1]);
  }
  const float sum = s[0] + s[1];
  if (in_range(sum)) {
    acc += (double)sum;
    return;
  }
  for (int u = 0; u < kPieces; ++u) {
    float v[8];
    values(*reinterpret_cast<const uint4 *>(mine + u * (16 * kThreads)), F32, v);
#pragma unroll
    for (int e = 0; e < kN; ++e)
      if (v[e] != 0.0f) acc += (double)v[e] * (double)v[e];
  }
}

// A warp's walk over its chunks, a step of kPieces * 32 pieces at a time.
struct Steps {
  const ClipChunk *plan;
  int64_t at, chunks, stride;
  ClipChunk c, next;
  int i, n;  // the chunk's first piece that is not taken, its pieces
  MOE_DEVINL void start() {
    i = 0;
    n = at < chunks && !(c.kind & 4) ? (c.kind & 1 ? c.n >> 2 : c.n >> 3) : 0;
  }
  MOE_DEVINL void fetch_next() {
    if (at + stride < chunks) next = load_chunk(plan + at + stride);
  }
  MOE_DEVINL Steps(const ClipChunk *p, int64_t first, int64_t count, int64_t by)
      : plan(p), at(first), chunks(count), stride(by), c{}, next{} {
    if (at < chunks) c = load_chunk(plan + at);
    fetch_next();
    start();
  }
  MOE_DEVINL bool done() const { return at >= chunks; }
  // whether the step that was taken was the chunk's last one
  MOE_DEVINL bool step() {
    i += 32 * kPieces;
    return i >= n;
  }
  MOE_DEVINL void advance() {
    at += stride;
    c = next;
    fetch_next();
    start();
  }
};

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

__global__ void __launch_bounds__(kThreads, 2)
grad_square_kernel(const ClipChunk *__restrict__ plan, int64_t chunks, double *__restrict__ part) {
  extern __shared__ __align__(16) uint8_t ring[];  // [kAhead][kPieces][threads][16]
  __shared__ double s[kThreads];
  constexpr int kStage = kPieces * 16 * kThreads;
  const int lane = threadIdx.x & 31;
  uint8_t *mine = ring + threadIdx.x * 16;
  double acc = 0.0;
  grid_dependency_begin();
  const int64_t first = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  Steps in(plan, first, chunks, (int64_t)gridDim.x * kWarps);  // what is copied
  Steps out = in;                                              // what is summed
  auto copy = [&](int stage) {
    if (!in.done()) {
      const uint8_t *g = static_cast<const uint8_t *>(in.c.g);
      uint8_t *to = mine + stage * kStage;
#pragma unroll
      for (int u = 0; u < kPieces; ++u) {
        const int j = in.i + 32 * u + lane;
        // (a copy of no bytes fills its 16 with zeros)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         (uint32_t)__cvta_generic_to_shared(to + u * (16 * kThreads))),
                     "l"(j < in.n ? g + 16ll * j : (const uint8_t *)plan), "r"(j < in.n ? 16 : 0)
                     : "memory");
      }
      if (in.step()) in.advance();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int k = 0; k < kAhead; ++k) copy(k);
  int stage = 0;
  while (!out.done()) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
    if (out.c.kind & 1) add_squares<true>(mine + stage * kStage, acc);
    else add_squares<false>(mine + stage * kStage, acc);
    if (out.step()) {  // the elements that fill no piece
      const bool f32 = out.c.kind & 1;
      for (int i = out.c.kind & 4 ? lane : (out.n << (f32 ? 2 : 3)) + lane; i < out.c.n; i += 32) {
        const double v = f32 ? F32x8::one(static_cast<const float *>(out.c.g) + i)
                             : Bf16x8::one(static_cast<const uint16_t *>(out.c.g) + i);
        acc += v * v;
      }
      out.advance();
    }
    copy(stage);
    if (++stage == kAhead) stage = 0;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
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

// The norm, and the factor that clips (a norm that is infinite or no number: none).  In fp32
// where everything is well inside its range: a 64-bit root and quotient take 2 us.
MOE_DEVINL float norm_of(double sum, float scale, float &factor, float max_norm) {
  if (sum >= 1e-30 && sum <= 1e30 && scale >= 1e-15f && scale <= 1e15f) {
    const float total = scale * sqrtf((float)sum), q = max_norm / (total + 1e-6f);
    factor = q < 1.0f ? scale * q : scale;
    return total;
  }
  const double total = (double)scale * sqrt(sum), q = (double)max_norm / (total + 1e-6);
  factor = total <= 1.7e308 && q < 1.0 ? (float)((double)scale * q) : scale;
  return (float)total;
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

__global__ void __launch_bounds__(kThreads, 3)
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
    const float total = norm_of(sum, scale, s_f, max_norm);
    if (blockIdx.x == 0) *norm = total;
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
  float factor;
  if (threadIdx.x == 0) *norm = norm_of(sum, scale, factor, 0.0f);
}

}  // namespace

cudaError_t launch_clip(const ClipChunk *plan, int64_t chunks, float scale, float max_norm, bool write,
                        float *norm, double *part, cudaStream_t st) {
  auto grid = [&](int per_sm) {
    const int64_t want = std::max<int64_t>(1, (chunks + kWarps - 1) / kWarps);
    return (int)std::min<int64_t>({want, (int64_t)num_sms() * per_sm, (int64_t)kClipMaxBlocks});
  };
  static PerDevice<cudaError_t> allowed;
  cudaError_t e = allowed.get(current_device(), [] {
    return cudaFuncSetAttribute(grad_square_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSquareSmem);
  });
  if (e != cudaSuccess) return e;
  const int parts = grid(2);
  e = launch_dependent(grad_square_kernel, parts, kThreads, kSquareSmem, st, plan, chunks, part);
  if (e != cudaSuccess) return e;
  if (!write) return launch_dependent(grad_norm_kernel, 1, kThreads, 0, st, part, parts, scale, norm);
  return launch_dependent(grad_scale_kernel, grid(blocks_per_sm<grad_scale_kernel>(kThreads)), kThreads,
                          0, st, plan, chunks, part, parts, scale, max_norm, norm);
}

}  // namespace moe

// The norm of all gradients together, and their clipping.
//
//     norm = scale sqrt(sum over tensors and elements of g^2)
//     out  = g scale min(1, max_norm / (norm + 1e-6))     (in place where out is g)
// A plan of chunks (pieces of tensors of a few thousand elements, made once by the host)
// tells the warps what to read: tensors of any number, size, type and alignment are one
// launch.  The first kernel writes a sum a block, the second adds these up again in every
// block (the same order, so the same number) and scales.  It walks the chunks from the last
// one back: what the first one read last is still in L2.
//
// HBM bounds both: 1.41 G bf16 gradients take 405 us (7.0 TB/s) to square and 885 us (6.4 TB/s of
// reads and writes) to scale, 1244 us at the measured copy's rate; loads that wait for the
// arithmetic of the ones before them took 668 and 887.
#include <float.h>
#include <math.h>

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

MOE_DEVINL float load_one(const ClipChunk &c, int i) {
  return c.kind & 1 ? ld_f32(static_cast<const float *>(c.g) + i)
                    : __uint_as_float(ld_u16(static_cast<const uint16_t *>(c.g) + i) << 16);
}

// Gradients come in pieces of 16 bytes, kPieces a lane at a time, copied to shared memory
// kAhead times ahead (each lane reads what it copied: no barrier).
constexpr int kPieces = 8;
constexpr int kAhead = 3;
constexpr int kStage = kPieces * 16 * kThreads;
constexpr int kRing = kAhead * kStage;

// Squares are added in fp32 for 32 or 64 values at a time, that sum in 64 bits (64-bit additions are
// slow on GB300: one for every 8 values took 0.1 ms of 1.4 G values).  A sum that is neither 0 nor in
// the middle of fp32's range, where squares that vanish are nothing beside it, is taken again of the
// values times a power of two, and where that leaves the range too (both ends at once, infinities),
// in 64 bits.  Lanes behind a tensor's end and experts without tokens have zeros only: the norm of
// 200 M bf16 zeros or values of 1e-18 took 773 us in 64 bits and takes 64 now, ordinary ones' 62.
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
  const bool large = sum > 1.0f;
  const float by = large ? 0x1p-72f : 0x1p72f;
  uint32_t some = 0;
  s[0] = s[1] = 0.0f;
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const uint4 w = *reinterpret_cast<const uint4 *>(mine + u * (16 * kThreads));
    some |= w.x | w.y | w.z | w.w;
    float v[8];
    values(w, F32, v);
#pragma unroll
    for (int e = 0; e < kN; ++e) s[e & 1] = fmaf(v[e] * by, v[e] * by, s[e & 1]);
  }
  if ((some & (F32 ? 0x7fffffffu : 0x7fff7fffu)) == 0) return;
  const float scaled = s[0] + s[1];
  if (in_range(scaled)) {
    acc += (double)scaled * (large ? 0x1p144 : 0x1p-144);
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

// A warp's walk over its chunks (from the plan's end back where REVERSE), a step of kPieces *
// 32 pieces at a time.
template <bool REVERSE>
struct Steps {
  const ClipChunk *plan;
  int64_t at, chunks, stride;
  ClipChunk c, next;
  int i, n;  // the chunk's first piece that is not taken, its pieces
  bool skip; // chunks in place are left as they are
  MOE_DEVINL ClipChunk chunk(int64_t k) const { return load_chunk(plan + (REVERSE ? chunks - 1 - k : k)); }
  MOE_DEVINL void start() {
    i = 0;
    n = at < chunks && (c.kind & 12) != 4 ? (c.kind & 1 ? c.n >> 2 : c.n >> 3) : 0;
    if (skip && c.g == c.out) n = c.n = 0;
  }
  MOE_DEVINL void fetch_next() {
    if (at + stride < chunks) next = chunk(at + stride);  // on its way while this one is worked on
  }
  MOE_DEVINL Steps(const ClipChunk *p, int64_t first, int64_t count, int64_t by, bool skip_in_place = false)
      : plan(p), at(first), chunks(count), stride(by), c{}, next{}, skip(skip_in_place) {
    if (at < chunks) c = chunk(at);
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
  // the step's pieces into `to`
  MOE_DEVINL void copy(uint8_t *to, int lane) {
    if (!done()) {
      const uint8_t *g = static_cast<const uint8_t *>(c.g);
#pragma unroll
      for (int u = 0; u < kPieces; ++u) {
        const int j = i + 32 * u + lane;
        // (a copy of no bytes fills its 16 with zeros)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         (uint32_t)__cvta_generic_to_shared(to + u * (16 * kThreads))),
                     "l"(j < n ? g + 16ll * j : (const uint8_t *)plan), "r"(j < n ? 16 : 0)
                     : "memory");
      }
      if (step()) advance();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // the first of the elements that fill no piece
  MOE_DEVINL int rest() const { return (c.kind & 12) == 4 ? 0 : n << (c.kind & 1 ? 2 : 3); }
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
  const int lane = threadIdx.x & 31;
  uint8_t *mine = ring + threadIdx.x * 16;
  double acc = 0.0;
  grid_dependency_begin();
  Steps<false> in(plan, (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5), chunks,
                  (int64_t)gridDim.x * kWarps);  // what is copied
  Steps<false> out = in;                         // what is summed
#pragma unroll
  for (int k = 0; k < kAhead; ++k) in.copy(mine + k * kStage, lane);
  int stage = 0;
  while (!out.done()) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
    if (out.c.kind & 1) add_squares<true>(mine + stage * kStage, acc);
    else add_squares<false>(mine + stage * kStage, acc);
    if (out.step()) {
      for (int i = out.rest() + lane; i < out.c.n; i += 32) {
        const double v = load_one(out.c, i);
        acc += v * v;
      }
      out.advance();
    }
    in.copy(mine + stage * kStage, lane);
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

// out = (g before) by.  A factor that fp32 holds with few bits or not at all (the norm of large
// gradients, a small max_norm) has a power of two taken out, which g is multiplied with first: that is
// exact but for elements whose output vanishes.
struct Factor {
  float by, before;
};

// The norm, and the factor that clips (a norm that is infinite in fp32, as the caller reads it, or no
// number: none).  In fp32 where everything is well inside its range: a 64-bit root and quotient
// take 2 us.
MOE_DEVINL float norm_of(double sum, float scale, float max_norm, Factor &f) {
  if (sum >= 1e-30 && sum <= 1e30 && scale >= 1e-15f && scale <= 1e15f) {
    const float total = scale * sqrtf((float)sum), q = max_norm / (total + 1e-6f);
    f = {q < 1.0f ? scale * q : scale, 1.0f};
    if (f.by >= 0x1p-64f) return total;
  }
  const double total = (double)scale * sqrt(sum), q = (double)max_norm / (total + 1e-6);
  const float norm = (float)total;
  const double by = norm <= FLT_MAX && q < 1.0 ? (double)scale * q : (double)scale;
  if (by >= 0x1p-100) f = {(float)by, 1.0f};
  else if (by >= 0x1p-160) f = {(float)(by * 0x1p64), 0x1p-64f};
  else f = {(float)(by * 0x1p126), 0x1p-126f};
  return norm;
}

// Piece j of a chunk, scaled, to its place.
MOE_DEVINL void scale_piece(const ClipChunk &c, int j, const uint4 &w, const Factor &f) {
  float v[8];
  values(w, c.kind & 1, v);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = v[e] * f.before * f.by;  // (fp32: the last four are no values)
  if (c.kind & 1) {
    if (c.kind & 2) {
      st_v4(static_cast<float *>(c.out) + 4 * j,
            make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                       __float_as_uint(v[3])));
    } else {
      const uint4 q = f32_to_bf16x8(v);
      *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(c.out) + 4 * j) = make_uint2(q.x, q.y);
    }
  } else if (c.kind & 2) {
    st_f32x8(static_cast<float *>(c.out) + 8 * j, v);
  } else {
    st_v4(static_cast<uint16_t *>(c.out) + 8 * j, f32_to_bf16x8(v));
  }
}

// A step's pieces, scaled, to a place that starts on no piece: the warp takes them from `row`, where its
// lanes copied them, element by element in order.  100 M bf16 clipped to bf16: 118 us, 99 where both
// start alike, 913 with elements that are read one by one.
template <typename G, typename O>
MOE_DEVINL void scale_in_order(const Steps<true> &at, const uint8_t *row, const Factor &f, int lane) {
  constexpr int kN = 16 / (int)sizeof(G);
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const int first = (at.i + 32 * u) * kN, left = at.n * kN - first;
    const G *from = reinterpret_cast<const G *>(row + u * (16 * kThreads));
    O *to = static_cast<O *>(at.c.out) + first;
#pragma unroll
    for (int e = 0; e < kN; ++e) {
      const int j = 32 * e + lane;
      if (j < left) {
        if constexpr (sizeof(O) == 4) to[j] = (float)from[j] * f.before * f.by;
        else to[j] = __float2bfloat16_rn((float)from[j] * f.before * f.by);
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads, 2)
grad_scale_kernel(const ClipChunk *__restrict__ plan, int64_t chunks, const double *__restrict__ part,
                  int parts, float scale, float max_norm, float *__restrict__ norm) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ double s[kThreads];
  __shared__ Factor s_f;
  const int lane = threadIdx.x & 31;
  uint8_t *mine = ring + threadIdx.x * 16;
  const int64_t first = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5), stride = (int64_t)gridDim.x * kWarps;
  // the plan and the gradients are older than the kernel before this one
  Steps<true> in(plan, first, chunks, stride), out = in;
#pragma unroll
  for (int k = 0; k < kAhead; ++k) in.copy(mine + k * kStage, lane);
  grid_dependency_begin();
  const double sum = total_of(part, parts, s);
  if (threadIdx.x == 0) {
    const float total = norm_of(sum, scale, max_norm, s_f);
    if (blockIdx.x == 0) *norm = total;
  }
  __syncthreads();
  const Factor f = s_f;
  if (f.by == 1.0f) {  // only what is not in place
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    in = out = Steps<true>(plan, first, chunks, stride, true);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) in.copy(mine + k * kStage, lane);
  }
  int stage = 0;
  while (!out.done()) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
    if (out.c.kind & 8) {
      __syncwarp();
      const uint8_t *row = mine + stage * kStage - 16 * lane;
      if (out.c.kind & 1) {
        if (out.c.kind & 2) scale_in_order<float, float>(out, row, f, lane);
        else scale_in_order<float, bf16_t>(out, row, f, lane);
      } else {
        if (out.c.kind & 2) scale_in_order<bf16_t, float>(out, row, f, lane);
        else scale_in_order<bf16_t, bf16_t>(out, row, f, lane);
      }
      __syncwarp();  // before the next copy there
    } else {
#pragma unroll
      for (int u = 0; u < kPieces; ++u) {
        const int j = out.i + 32 * u + lane;
        if (j < out.n)
          scale_piece(out.c, j, *reinterpret_cast<const uint4 *>(mine + stage * kStage + u * (16 * kThreads)), f);
      }
    }
    if (out.step()) {
      for (int i = out.rest() + lane; i < out.c.n; i += 32) {
        const float v = load_one(out.c, i) * f.before * f.by;
        if (out.c.kind & 2) static_cast<float *>(out.c.out)[i] = v;
        else static_cast<bf16_t *>(out.c.out)[i] = __float2bfloat16_rn(v);
      }
      out.advance();
    }
    in.copy(mine + stage * kStage, lane);
    if (++stage == kAhead) stage = 0;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

__global__ void __launch_bounds__(kThreads)
grad_norm_kernel(const double *__restrict__ part, int parts, float scale, float *__restrict__ norm) {
  __shared__ double s[kThreads];
  grid_dependency_begin();
  const double sum = total_of(part, parts, s);
  Factor none;
  if (threadIdx.x == 0) *norm = norm_of(sum, scale, INFINITY, none);
}

}  // namespace

cudaError_t launch_clip(const ClipChunk *plan, int64_t chunks, float scale, float max_norm, bool write,
                        float *norm, double *part, cudaStream_t st) {
  static PerDevice<cudaError_t> allowed;
  cudaError_t e = allowed.get(current_device(), [] {
    const cudaFuncAttribute at = cudaFuncAttributeMaxDynamicSharedMemorySize;
    const cudaError_t a = cudaFuncSetAttribute(grad_square_kernel, at, kRing);
    return a != cudaSuccess ? a : cudaFuncSetAttribute(grad_scale_kernel, at, kRing);
  });
  if (e != cudaSuccess) return e;
  // two blocks a SM, as their rings go
  const int blocks = (int)std::min<int64_t>({std::max<int64_t>(1, (chunks + kWarps - 1) / kWarps),
                                             2ll * num_sms(), (int64_t)kClipMaxBlocks});
  e = launch_dependent(grad_square_kernel, blocks, kThreads, kRing, st, plan, chunks, part);
  if (e != cudaSuccess) return e;
  if (!write) return launch_dependent(grad_norm_kernel, 1, kThreads, 0, st, part, blocks, scale, norm);
  return launch_dependent(grad_scale_kernel, blocks, kThreads, kRing, st, plan, chunks, part, blocks, scale,
                          max_norm, norm);
}

}  // namespace moe

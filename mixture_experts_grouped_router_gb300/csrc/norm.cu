// The RMS norm before the experts, with the residual's addition and 8-bit
// outputs, and its backward.
//
//     h = round(x + residual)                     (the residual stream's type)
//     r = (mean_j h_j^2 + eps)^(-1/2),   y_j = bf16(h_j r w_j)
// and, from dy and the gradient d_res that reaches h past the block,
//     g_j = dy_j w_j,   dh_j = r g_j - r^3 mean(g h) h_j + d_res_j,
//     dw_j = sum over rows of dy_j h_j r.
// The norm is of the h that is stored, so that the backward, which reads it back, is the
// derivative of what the forward computed.  The 8-bit codes are those of the bf16 y (what
// the block-scaled and the checkpoint quantisers make of it, bit for bit): a program that
// keeps both has codes of the tensor it computed with.  All sums and products are fp32.
#include <algorithm>

#include "internal.h"
#include "lowbit.cuh"

namespace moe {
namespace {

// 8 consecutive elements of the residual stream (bf16 or fp32) or of a weight.
template <typename S>
struct Vec8;

template <>
struct Vec8<uint16_t> {
  uint4 a;
  MOE_DEVINL void zero() { a = make_uint4(0, 0, 0, 0); }
  MOE_DEVINL void load(const uint16_t *p) { a = ld_stream_v4(p); }
  template <typename F>
  MOE_DEVINL void take(F piece) { a = piece(0); }  // from its pieces of 16 bytes
  MOE_DEVINL void get(float *v) const { bf16x8_to_f32(a, v); }
  MOE_DEVINL void set(const float *v) { a = f32_to_bf16x8(v); }
  MOE_DEVINL void store(uint16_t *p) const { st_v4(p, a); }
};

template <>
struct Vec8<float> {
  uint4 a, b;
  MOE_DEVINL void zero() { a = b = make_uint4(0, 0, 0, 0); }
  MOE_DEVINL void load(const float *p) {
    a = ld_stream_v4(p);
    b = ld_stream_v4(p + 4);
  }
  template <typename F>
  MOE_DEVINL void take(F piece) {
    a = piece(0);
    b = piece(1);
  }
  MOE_DEVINL void get(float *v) const {
    const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(u[i]);
  }
  MOE_DEVINL void set(const float *v) {
    a = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                   __float_as_uint(v[3]));
    b = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]),
                   __float_as_uint(v[7]));
  }
  MOE_DEVINL void store(float *p) const {
    st_v4(p, a);
    st_v4(p + 4, b);
  }
};

// The weights are read by every row: loads that may stay in L1, behind the wait for the
// kernel before (which may have written them).
MOE_DEVINL uint4 ld_v4(const void *p) {
  uint4 r;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

MOE_DEVINL void load_w(const void *w, int w_dtype, int col, float *v) {
  if (w_dtype == MOE_DTYPE_F32) {
    Vec8<float> t;
    t.a = ld_v4(static_cast<const float *>(w) + col);
    t.b = ld_v4(static_cast<const float *>(w) + col + 4);
    t.get(v);
  } else {
    bf16x8_to_f32(ld_v4(static_cast<const uint16_t *>(w) + col), v);
  }
}

// A row belongs to a team of W warps; a block holds several teams where W is small.
// Vector v of a lane is at column (32 (v W + warp) + lane) 8: 4 lanes hold a block of 32.
struct Team {
  int W, warp, lane, id;
  MOE_DEVINL explicit Team(int w)
      : W(w), warp((int)(threadIdx.x >> 5) % w), lane(threadIdx.x & 31),
        id((int)(threadIdx.x >> 5) / w) {}
  MOE_DEVINL int col(int v) const { return ((v * W + warp) * 32 + lane) * 8; }
  // Sum over the team's lanes, by way of red[warps of the block] (the same in every lane).
  MOE_DEVINL float sum(float v, float *red) const {
    v = warp_sum(v);
    if (W == 1) return v;
    if (lane == 0) red[id * W + warp] = v;
    sync();
    return warp_sum(lane < W ? red[id * W + lane] : 0.0f);
  }
  MOE_DEVINL void sync() const {
    asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(W * 32) : "memory");
  }
};

template <int VPL, typename S, int CODES>
__global__ void __launch_bounds__(VPL > 2 ? 512 : 1024)
rms_norm_kernel(const RmsNormArgs a, int W, int teams) {
  __shared__ float red[32];
  const Team t(W);
  grid_dependency_begin();
  const int64_t row = (int64_t)blockIdx.x * teams + t.id;
  if (row >= a.rows) return;
  const S *res = static_cast<const S *>(a.residual);
  S *h = static_cast<S *>(a.h);
  uint4 xv[VPL];
  Vec8<S> hv[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int c = t.col(v);
    xv[v] = make_uint4(0, 0, 0, 0);
    hv[v].zero();
    if (c < a.cols) {
      if (a.x != nullptr) xv[v] = ld_stream_v4(a.x + row * a.ldx + c);
      if (res != nullptr) hv[v].load(res + row * a.ld_res + c);
    }
  }
  // one vector a lane (few rows): the weights come along, not a latency later
  constexpr bool kEarly = VPL == 1;
  float we[8];
  if (kEarly && t.col(0) < a.cols) load_w(a.w, a.w_dtype, t.col(0), we);
  float ss = 0.0f;
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int c = t.col(v);
    float f[8], g[8];
    bf16x8_to_f32(xv[v], f);
    hv[v].get(g);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] += g[i];
    hv[v].set(f);
    if (h != nullptr && c < a.cols) hv[v].store(h + row * a.ldh + c);
    hv[v].get(f);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
  }
  const float r = rsqrtf(t.sum(ss, red) / (float)a.cols + a.eps);
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int c = t.col(v);
    const bool in = c < a.cols;
    float f[8], w[8];
    hv[v].get(f);
    if (!kEarly && in) load_w(a.w, a.w_dtype, c, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = in ? f[i] * r * (kEarly ? we[i] : w[i]) : 0.0f;
    const uint4 y = f32_to_bf16x8(f);
    if (a.y != nullptr && in) st_v4(a.y + row * a.ldy + c, y);
    if (CODES == MOE_CODES_MX) {
      uint32_t code;
      const uint2 q = mx_quantize8(y, code);
      // the four blocks of an atom's row lie side by side
      code <<= 8 * ((t.lane >> 2) & 3);
      code |= __shfl_xor_sync(0xffffffffu, code, 4);
      code |= __shfl_xor_sync(0xffffffffu, code, 8);
      if (in) {
        *reinterpret_cast<uint2 *>(a.q + row * a.ldq + c) = q;
        if ((t.lane & 15) == 0) {
          const int rw = (int)(row & 127);
          uint8_t *at = static_cast<uint8_t *>(a.scales) +
                        ((row >> 7) * (a.cols >> 7) + (c >> 7)) * 512 + (rw & 31) * 16 + (rw >> 5) * 4;
          *reinterpret_cast<uint32_t *>(at) = code;
        }
      }
    } else if (CODES == MOE_CODES_ACT8) {
      uint32_t sb;
      const uint2 q = act8_quantize8(y, sb);
      if (in) {
        *reinterpret_cast<uint2 *>(a.q + row * a.ldq + c) = q;
        if ((t.lane & 3) == 0)
          static_cast<uint16_t *>(a.scales)[row * a.lds + (c >> 5)] = (uint16_t)sb;
      }
    }
  }
}

// The weights of 8 columns, zeros past the last one.
MOE_DEVINL void weights(const RmsNormBwdArgs &a, int col, float *w) {
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 0.0f;
  if (col < a.cols) load_w(a.w, a.w_dtype, col, w);
}

// 16 bytes from global to shared memory, asynchronously.
MOE_DEVINL void copy_async(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src)
               : "memory");
}

// Backward: a block's teams walk over rows and keep their columns' sums of dy h r in
// registers; at the end the block's teams are added up in order and the block's row of
// `part` is written.  part == NULL: no gradient of w is wanted.
//
// Rows come in by asynchronous copies, `stages` rows ahead of the arithmetic: every thread
// copies what it will read itself (h, dy, d_residual: kChunks pieces of 16 bytes), so that
// no barrier is needed and loads stay under way while a row's sums are taken.
// kThreads: the most that a block has; w stays in registers where that is 512.
template <int VPL, typename S, int kThreads>
__global__ void __launch_bounds__(kThreads)
rms_norm_bwd_kernel(const RmsNormBwdArgs a, int W, int teams, int stages, float *__restrict__ part) {
  constexpr int kWide = sizeof(S) / 2;             // pieces of 8 elements of the stream
  constexpr int kPieces = VPL * (2 * kWide + 1);   // of a thread and row
  __shared__ float red[2][2][32];
  extern __shared__ __align__(16) uint8_t smem[];  // [stages][kPieces][threads][16]
  const Team t(W);
  constexpr bool kKeepW = kThreads <= 512;
  float dw[VPL][8], kept[kKeepW ? VPL : 1][8];
  const S *h = static_cast<const S *>(a.h);
  const S *res = static_cast<const S *>(a.d_residual);
  S *dh = static_cast<S *>(a.dh);
  const int64_t step = (int64_t)gridDim.x * teams;
  int64_t row = (int64_t)blockIdx.x * teams + t.id, ahead = row;
  const int piece = blockDim.x * 16, stage = kPieces * piece;
  uint8_t *mine = smem + threadIdx.x * 16;
  auto fetch = [&](int s) {
    if (ahead < a.rows) {
      uint8_t *to = mine + s * stage;
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        const int c = t.col(v);
        if (c < a.cols) {
#pragma unroll
          for (int k = 0; k < kWide; ++k) {
            copy_async(to + (v * kWide + k) * piece, h + ahead * a.ldh + c + 4 * k);
            if (res != nullptr)
              copy_async(to + ((VPL + v) * kWide + k) * piece, res + ahead * a.ld_dres + c + 4 * k);
          }
          copy_async(to + (2 * VPL * kWide + v) * piece, a.dy + ahead * a.ld_dy + c);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ahead += step;
  };
  auto piece_at = [&](int s, int k) {
    return *reinterpret_cast<const uint4 *>(mine + s * stage + k * piece);
  };
  grid_dependency_begin();
  for (int s = 0; s < stages; ++s) fetch(s);
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[v][i] = 0.0f;
    if (kKeepW) weights(a, t.col(v), kept[v]);
  }
  int turn = 0, s = 0;
  for (; row < a.rows; row += step, turn ^= 1) {
    // all but the rows ahead have landed
    if (stages == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (stages == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
    uint4 dy[VPL];
    Vec8<S> hv[VPL], rv[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      dy[v] = make_uint4(0, 0, 0, 0);
      hv[v].zero();
      rv[v].zero();
      if (t.col(v) < a.cols) {
        hv[v].take([&](int k) { return piece_at(s, v * kWide + k); });
        if (res != nullptr) rv[v].take([&](int k) { return piece_at(s, (VPL + v) * kWide + k); });
        dy[v] = piece_at(s, 2 * VPL * kWide + v);
      }
    }
    float ss = 0.0f, gh = 0.0f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      float f[8], g[8], w[8];
      hv[v].get(f);
      bf16x8_to_f32(dy[v], g);
      if (!kKeepW) weights(a, t.col(v), w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = fmaf(f[i], f[i], ss);
        gh = fmaf(g[i] * (kKeepW ? kept[v][i] : w[i]), f[i], gh);
      }
    }
    fetch(s);  // (what was there is in registers)
    if (++s == stages) s = 0;
    ss = warp_sum(ss);
    gh = warp_sum(gh);
    if (W > 1) {  // (two buffers in turn: the next row's sums need no second barrier)
      if (t.lane == 0) {
        red[turn][0][t.id * W + t.warp] = ss;
        red[turn][1][t.id * W + t.warp] = gh;
      }
      t.sync();
      ss = warp_sum(t.lane < W ? red[turn][0][t.id * W + t.lane] : 0.0f);
      gh = warp_sum(t.lane < W ? red[turn][1][t.id * W + t.lane] : 0.0f);
    }
    const float r = rsqrtf(ss / (float)a.cols + a.eps);
    const float s3 = r * r * r * (gh / (float)a.cols);
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int c = t.col(v);
      float f[8], g[8], d[8], w[8];
      hv[v].get(f);
      bf16x8_to_f32(dy[v], g);
      rv[v].get(d);
      if (!kKeepW) weights(a, c, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dw[v][i] = fmaf(g[i], f[i] * r, dw[v][i]);
        d[i] += fmaf(-s3, f[i], r * (g[i] * (kKeepW ? kept[v][i] : w[i])));
      }
      if (c < a.cols) {
        Vec8<S> o;
        o.set(d);
        o.store(dh + row * a.ld_dh + c);
        if (a.dx != nullptr) st_v4(a.dx + row * a.ld_dx + c, f32_to_bf16x8(d));
      }
    }
  }
  if (part == nullptr) return;
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  float *s_dw = reinterpret_cast<float *>(smem);  // [teams - 1][cols]
  if (t.id > 0) {
#pragma unroll
    for (int v = 0; v < VPL; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (t.col(v) < a.cols) s_dw[(t.id - 1) * a.cols + t.col(v) + i] = dw[v][i];
  }
  __syncthreads();
  if (t.id > 0) return;
  float *out = part + (int64_t)blockIdx.x * a.cols;
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int c = t.col(v);
    if (c >= a.cols) continue;
    for (int k = 0; k < teams - 1; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) dw[v][i] += s_dw[k * a.cols + c + i];
    Vec8<float> o;
    o.set(dw[v]);
    o.store(out + c);
  }
}

// dw[c] = (dw[c] +) sum over the blocks' rows of part, in a fixed order.
constexpr int kSumRows = 32;  // rows of part summed at a time by one block of 32 columns
__global__ void __launch_bounds__(32 * kSumRows)
dw_sum_kernel(const float *__restrict__ part, int parts, int cols, float *__restrict__ dw,
              int accumulate) {
  __shared__ float s[kSumRows][33];
  grid_dependency_begin();
  const int c = blockIdx.x * 32 + threadIdx.x, k = threadIdx.y;
  float v = 0.0f;
  if (c < cols)
    for (int p = k; p < parts; p += kSumRows) v += ld_f32(part + (int64_t)p * cols + c);
  s[k][threadIdx.x] = v;
  __syncthreads();
  // row k of the transposed sums: one warp a column
  v = warp_sum(s[threadIdx.x][k]);
  const int col = blockIdx.x * 32 + k;
  if (threadIdx.x == 0 && col < cols) dw[col] = accumulate ? dw[col] + v : v;
}

// Warps of a row's team with `vpl` vectors of 8 a lane.
int team_warps(int cols, int vpl) { return (cols + 256 * vpl - 1) / (256 * vpl); }

template <int VPL, typename S>
cudaError_t norm_launch(const RmsNormArgs &a, cudaStream_t st) {
  const int W = team_warps(a.cols, VPL), teams = std::max(1, 8 / W);
  const unsigned grid = (unsigned)((a.rows + teams - 1) / teams);
  const dim3 block(32 * W * teams);
  switch (a.codes) {
    case MOE_CODES_MX:
      return launch_dependent(rms_norm_kernel<VPL, S, MOE_CODES_MX>, grid, block, 0, st, a, W, teams);
    case MOE_CODES_ACT8:
      return launch_dependent(rms_norm_kernel<VPL, S, MOE_CODES_ACT8>, grid, block, 0, st, a, W, teams);
    default:
      return launch_dependent(rms_norm_kernel<VPL, S, MOE_CODES_NONE>, grid, block, 0, st, a, W, teams);
  }
}

template <typename S>
cudaError_t norm_by_size(const RmsNormArgs &a, cudaStream_t st) {
  // few rows: more warps a row, for the latency
  const bool few = a.rows < 2 * num_sms();
  if (few && a.cols <= 8192) return norm_launch<1, S>(a, st);
  if (few) return norm_launch<2, S>(a, st);
  return norm_launch<4, S>(a, st);
}

constexpr int kBwdVpl = 2;  // 16384 columns in 32 warps

// How the backward is laid out over a SM: blocks, rows ahead, bytes of a block.
struct BwdShape {
  int W, teams, threads, per_sm, stages;
  size_t smem;
  BwdShape(int cols, int elem) {
    W = team_warps(cols, kBwdVpl);
    teams = std::max(1, 8 / W);
    threads = 32 * W * teams;
    per_sm = std::max(1, kBwdResident / threads);
    const size_t stage = (size_t)threads * 16 * kBwdVpl * (elem + 1);
    const size_t each = kBwdSmem / per_sm;
    stages = (int)std::min<size_t>(3, each / stage);
    smem = std::max(stage * stages, (size_t)(teams - 1) * cols * sizeof(float));
  }
  static constexpr int kBwdResident = 512;   // threads of a SM (128 registers)
  static constexpr size_t kBwdSmem = 216 << 10;
};

// Blocks that the backward is launched with at most (its rows of `part`).
int64_t bwd_parts(int64_t rows, int cols) {
  const BwdShape b(cols, 2);
  return std::min<int64_t>((rows + b.teams - 1) / b.teams, 160 * b.per_sm);
}

template <auto Kernel>
cudaError_t allow_smem() {
  static PerDevice<cudaError_t> done;
  return done.get(current_device(), [] {
    return cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)BwdShape::kBwdSmem);
  });
}

template <typename S, int kThreads>
cudaError_t bwd_kernel(const RmsNormBwdArgs &a, const BwdShape &b, unsigned grid, float *part, cudaStream_t st) {
  const cudaError_t e = allow_smem<rms_norm_bwd_kernel<kBwdVpl, S, kThreads>>();
  if (e != cudaSuccess) return e;
  return launch_dependent(rms_norm_bwd_kernel<kBwdVpl, S, kThreads>, grid, b.threads, b.smem, st, a, b.W,
                          b.teams, b.stages, part);
}

template <typename S>
cudaError_t bwd_launch(const RmsNormBwdArgs &a, float *part, cudaStream_t st) {
  const BwdShape b(a.cols, (int)sizeof(S));
  const unsigned grid =
      (unsigned)std::min<int64_t>(bwd_parts(a.rows, a.cols), (int64_t)num_sms() * b.per_sm);
  const cudaError_t e = b.threads <= 512 ? bwd_kernel<S, 512>(a, b, grid, part, st)
                                         : bwd_kernel<S, 1024>(a, b, grid, part, st);
  if (e != cudaSuccess || part == nullptr) return e;
  return launch_dependent(dw_sum_kernel, (unsigned)((a.cols + 31) / 32), dim3(32, kSumRows), 0, st,
                          part, (int)grid, a.cols, a.dw, a.accumulate);
}

}  // namespace

cudaError_t launch_rms_norm(const RmsNormArgs &a, cudaStream_t st) {
  return a.stream_dtype == MOE_DTYPE_F32 ? norm_by_size<float>(a, st) : norm_by_size<uint16_t>(a, st);
}

size_t rms_norm_bwd_workspace_bytes(int64_t rows, int cols) {
  return (size_t)bwd_parts(rows, cols) * (size_t)cols * sizeof(float);
}

cudaError_t launch_rms_norm_bwd(const RmsNormBwdArgs &a, float *part, cudaStream_t st) {
  if (a.rows == 0) {  // sums over no rows
    if (a.dw == nullptr || a.accumulate) return cudaSuccess;
    return cudaMemsetAsync(a.dw, 0, (size_t)a.cols * sizeof(float), st);
  }
  return a.stream_dtype == MOE_DTYPE_F32 ? bwd_launch<float>(a, part, st)
                                         : bwd_launch<uint16_t>(a, part, st);
}

}  // namespace moe

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

// 8 consecutive elements in fp32, in pairs (one instruction for two).
struct Pairs {
  uint64_t p[4];
  MOE_DEVINL void zero() {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = 0;
  }
};

MOE_DEVINL Pairs from_bf16(const uint4 &w) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  Pairs r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r.p[i] = pack2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
  return r;
}

MOE_DEVINL uint4 to_bf16(const Pairs &v) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    unpack2(v.p[i], lo, hi);
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u[i]) : "f"(hi), "f"(lo));
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

MOE_DEVINL Pairs from_f32(const uint4 &a, const uint4 &b) {
  const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  Pairs r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r.p[i] = pack2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
  return r;
}

// The two sums of squares / products of pairs, as one number.
MOE_DEVINL float both(uint64_t v) {
  float lo, hi;
  unpack2(v, lo, hi);
  return lo + hi;
}

// Streamed loads and stores of 8 elements of the residual stream.  fp32: one access of 32 bytes
// where rows are aligned to that (FULL).
template <typename S, bool FULL>
struct Vec8;

template <bool FULL>
struct Vec8<uint16_t, FULL> {
  uint4 a;
  MOE_DEVINL void zero() { a = make_uint4(0, 0, 0, 0); }
  MOE_DEVINL void load(const uint16_t *p) { a = ld_stream_v4(p); }
  // + x, rounded once
  MOE_DEVINL void add(const uint4 &x) {
    __nv_bfloat162 *v = reinterpret_cast<__nv_bfloat162 *>(&a);
    const __nv_bfloat162 *u = reinterpret_cast<const __nv_bfloat162 *>(&x);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __hadd2(v[i], u[i]);
  }
  MOE_DEVINL Pairs get() const { return from_bf16(a); }
  MOE_DEVINL void set(const Pairs &v) { a = to_bf16(v); }
  MOE_DEVINL void store(uint16_t *p) const { st_v4(p, a); }
};

template <bool FULL>
struct Vec8<float, FULL> {
  Pairs v;
  MOE_DEVINL void zero() { v.zero(); }
  MOE_DEVINL void load(const float *p) {
    if (FULL) {
      float f[8];
      ld_stream_f32x8(p, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) v.p[i] = pack2(f[2 * i], f[2 * i + 1]);
    } else {
      v = from_f32(ld_stream_v4(p), ld_stream_v4(p + 4));
    }
  }
  MOE_DEVINL void add(const uint4 &x) {
    const Pairs u = from_bf16(x);
#pragma unroll
    for (int i = 0; i < 4; ++i) v.p[i] = add2(v.p[i], u.p[i]);
  }
  MOE_DEVINL Pairs get() const { return v; }
  MOE_DEVINL void set(const Pairs &u) { v = u; }
  MOE_DEVINL void store(float *p) const {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack2(v.p[i], f[2 * i], f[2 * i + 1]);
    if (FULL) {
      st_f32x8(p, f);
    } else {
      st_v4(p, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3])));
      st_v4(p + 4, make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]),
                              __float_as_uint(f[7])));
    }
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

MOE_DEVINL Pairs load_w(const void *w, int w_dtype, int col) {
  if (w_dtype == MOE_DTYPE_F32) {
    const float *p = static_cast<const float *>(w) + col;
    return from_f32(ld_v4(p), ld_v4(p + 4));
  }
  return from_bf16(ld_v4(static_cast<const uint16_t *>(w) + col));
}

// A row belongs to a team of W warps; a block holds several teams where W is small.  Warp w
// of a team has the columns from 256 VPL w on; vector v of a lane is at 256 v + 8 lane of
// these: 4 lanes hold a block of 32.
struct Team {
  int W, warp, lane, id;
  MOE_DEVINL explicit Team(int w)
      : W(w), warp((int)(threadIdx.x >> 5) % w), lane(threadIdx.x & 31),
        id((int)(threadIdx.x >> 5) / w) {}
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

// FULL: the team's lanes have cols columns exactly, and fp32 rows start on 32 bytes.  What
// bounds it: HBM for bf16 output (16384 x 4096: 79 us, 6800 GB/s); with codes the issue of
// instructions came first (290 for 8 values a lane before the arithmetic in pairs, 80 us).
template <int VPL, typename S, int CODES, bool FULL>
__global__ void __launch_bounds__(VPL > 2 ? 512 : 1024)
rms_norm_kernel(const RmsNormArgs a, int W, int teams) {
  __shared__ float red[32];
  const Team t(W);
  grid_dependency_begin();
  const int64_t row = (int64_t)blockIdx.x * teams + t.id;
  if (row >= a.rows) return;
  const int c0 = t.warp * (256 * VPL) + t.lane * 8;
  auto in = [&](int v) { return FULL || c0 + 256 * v < a.cols; };
  const S *res = static_cast<const S *>(a.residual) + row * a.ld_res + c0;
  const uint16_t *x = a.x + row * a.ldx + c0;
  uint4 xv[VPL];
  Vec8<S, FULL> hv[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    xv[v] = make_uint4(0, 0, 0, 0);
    hv[v].zero();
    if (in(v)) {
      if (a.x != nullptr) xv[v] = ld_stream_v4(x + 256 * v);
      if (a.residual != nullptr) hv[v].load(res + 256 * v);
    }
  }
  // one vector a lane (few rows): the weights come along, not a latency later
  constexpr bool kEarly = VPL == 1;
  Pairs early;
  early.zero();
  if (kEarly && in(0)) early = load_w(a.w, a.w_dtype, c0);
  uint64_t s2 = 0;
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    hv[v].add(xv[v]);
    if (a.h != nullptr && in(v)) hv[v].store(static_cast<S *>(a.h) + row * a.ldh + c0 + 256 * v);
    const Pairs f = hv[v].get();
#pragma unroll
    for (int i = 0; i < 4; ++i) s2 = fma2(f.p[i], f.p[i], s2);
  }
  const float r = rsqrtf(t.sum(both(s2), red) / (float)a.cols + a.eps);
  const uint64_t r2 = pack2(r, r);
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int c = c0 + 256 * v;
    // (past the last column h is 0, and any weight will do)
    const Pairs w = kEarly ? early : load_w(a.w, a.w_dtype, FULL ? c : min(c, a.cols - 8));
    Pairs f = hv[v].get();
#pragma unroll
    for (int i = 0; i < 4; ++i) f.p[i] = mul2(mul2(f.p[i], r2), w.p[i]);
    const uint4 y = to_bf16(f);
    if (a.y != nullptr && in(v)) st_v4(a.y + row * a.ldy + c, y);
    if (CODES == MOE_CODES_MX) {
      uint32_t code;
      const uint2 q = mx_quantize8(y, code);
      // the four blocks of an atom's row lie side by side
      code <<= 8 * ((t.lane >> 2) & 3);
      code |= __shfl_xor_sync(0xffffffffu, code, 4);
      code |= __shfl_xor_sync(0xffffffffu, code, 8);
      if (in(v)) {
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
      if (in(v)) {
        *reinterpret_cast<uint2 *>(a.q + row * a.ldq + c) = q;
        if ((t.lane & 3) == 0)
          static_cast<uint16_t *>(a.scales)[row * a.lds + (c >> 5)] = (uint16_t)sb;
      }
    }
  }
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
// Rows come in by asynchronous copies, `stages` rows ahead of the arithmetic: a warp copies
// what its own lanes will read (h, dy, d_residual), so that a warp's barrier is enough and
// loads stay under way while a row's sums are taken (16384 x 4096 bf16: 82 us, 6550 GB/s;
// without: 106 us).  kThreads: the most that a block has; w stays in registers where that is
// 512.
template <int VPL, typename S, int kThreads>
__global__ void __launch_bounds__(kThreads)
rms_norm_bwd_kernel(const RmsNormBwdArgs a, int W, int teams, int stages, float *__restrict__ part) {
  constexpr int kWide = sizeof(S) / 2;             // copies of a warp for 8 elements a lane
  constexpr int kCopies = VPL * (2 * kWide + 1);   // of a warp and row, 512 bytes each
  __shared__ float red[2][2][32];
  extern __shared__ __align__(16) uint8_t smem[];  // [stages][warps][kCopies][512]
  const Team t(W);
  constexpr bool kKeepW = kThreads <= 512;
  const int c0 = t.warp * (256 * VPL) + t.lane * 8;
  auto in = [&](int v) { return c0 + 256 * v < a.cols; };
  Pairs dw[VPL], kept[kKeepW ? VPL : 1];
  const S *h = static_cast<const S *>(a.h);
  const S *res = static_cast<const S *>(a.d_residual);
  S *dh = static_cast<S *>(a.dh);
  const int64_t step = (int64_t)gridDim.x * teams;
  int64_t row = (int64_t)blockIdx.x * teams + t.id, ahead = row;
  const int stage = (int)(blockDim.x >> 5) * kCopies * 512;
  uint8_t *mine = smem + (threadIdx.x >> 5) * (kCopies * 512);
  // the warp's next row into stage s: 256 columns of each operand at a time, lane by lane
  auto fetch = [&](int s) {
    if (ahead < a.rows) {
      uint8_t *to = mine + s * stage + t.lane * 16;
      const int w0 = t.warp * (256 * VPL);
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
#pragma unroll
        for (int k = 0; k < kWide; ++k) {
          const int c = w0 + 256 * v + (256 / kWide) * k + t.lane * (8 / kWide);
          if (c < a.cols) {
            copy_async(to + (v * kWide + k) * 512, h + ahead * a.ldh + c);
            if (res != nullptr)
              copy_async(to + ((VPL + v) * kWide + k) * 512, res + ahead * a.ld_dres + c);
          }
        }
        if (in(v)) copy_async(to + (2 * VPL * kWide + v) * 512, a.dy + ahead * a.ld_dy + c0 + 256 * v);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ahead += step;
  };
  // the lane's 8 elements of the stream's operand number n
  auto take = [&](int s, int n) {
    const uint4 *p = reinterpret_cast<const uint4 *>(mine + s * stage + n * (kWide * 512)) + t.lane * kWide;
    return kWide == 1 ? from_bf16(p[0]) : from_f32(p[0], p[kWide - 1]);
  };
  grid_dependency_begin();
  for (int s = 0; s < stages; ++s) fetch(s);
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    dw[v].zero();
    if (kKeepW) {
      kept[v].zero();
      if (in(v)) kept[v] = load_w(a.w, a.w_dtype, c0 + 256 * v);
    }
  }
  int turn = 0, s = 0;
  for (; row < a.rows; row += step, turn ^= 1) {
    // all but the rows ahead have landed
    if (stages == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (stages == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
    Pairs hv[VPL], gv[VPL], rv[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      hv[v].zero();
      gv[v].zero();
      rv[v].zero();
      if (in(v)) {
        hv[v] = take(s, v);
        if (res != nullptr) rv[v] = take(s, VPL + v);
        gv[v] = from_bf16(reinterpret_cast<const uint4 *>(mine + s * stage + (2 * VPL * kWide + v) * 512)[t.lane]);
      }
    }
    __syncwarp();
    fetch(s);  // (what was there is in registers)
    if (++s == stages) s = 0;
    uint64_t ss2 = 0, gh2 = 0;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      Pairs w;
      if (!kKeepW && in(v)) w = load_w(a.w, a.w_dtype, c0 + 256 * v);
      else if (!kKeepW) w.zero();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ss2 = fma2(hv[v].p[i], hv[v].p[i], ss2);
        gh2 = fma2(mul2(gv[v].p[i], kKeepW ? kept[v].p[i] : w.p[i]), hv[v].p[i], gh2);
      }
    }
    float ss = warp_sum(both(ss2)), gh = warp_sum(both(gh2));
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
    const float s3 = -(r * r * r * (gh / (float)a.cols));
    const uint64_t r2 = pack2(r, r), s2 = pack2(s3, s3);
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int c = c0 + 256 * v;
      Pairs w;
      if (!kKeepW && in(v)) w = load_w(a.w, a.w_dtype, c);
      else if (!kKeepW) w.zero();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        dw[v].p[i] = fma2(gv[v].p[i], mul2(hv[v].p[i], r2), dw[v].p[i]);
        const uint64_t g = mul2(mul2(gv[v].p[i], kKeepW ? kept[v].p[i] : w.p[i]), r2);
        rv[v].p[i] = add2(fma2(s2, hv[v].p[i], g), rv[v].p[i]);
      }
      if (in(v)) {
        Vec8<S, false> o;
        o.set(rv[v]);
        o.store(dh + row * a.ld_dh + c);
        if (a.dx != nullptr) st_v4(a.dx + row * a.ld_dx + c, to_bf16(rv[v]));
      }
    }
  }
  if (part == nullptr) return;
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  float *s_dw = reinterpret_cast<float *>(smem);  // [teams - 1][cols]
  if (t.id > 0) {
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      if (!in(v)) continue;
      float *o = s_dw + (t.id - 1) * a.cols + c0 + 256 * v;
#pragma unroll
      for (int i = 0; i < 4; ++i) unpack2(dw[v].p[i], o[2 * i], o[2 * i + 1]);
    }
  }
  __syncthreads();
  if (t.id > 0) return;
  float *out = part + (int64_t)blockIdx.x * a.cols;
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int c = c0 + 256 * v;
    if (!in(v)) continue;
    for (int k = 0; k < teams - 1; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        dw[v].p[i] = add2(dw[v].p[i], pack2(s_dw[k * a.cols + c + 2 * i], s_dw[k * a.cols + c + 2 * i + 1]));
    Vec8<float, false> o;
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
  if (c < cols) {
    for (int p = k; p < parts; p += 8 * kSumRows) {
      float x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int q = p + u * kSumRows;
        x[u] = q < parts ? ld_f32(part + (int64_t)q * cols + c) : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) v += x[u];
    }
  }
  s[k][threadIdx.x] = v;
  __syncthreads();
  // row k of the transposed sums: one warp a column
  v = warp_sum(s[threadIdx.x][k]);
  const int col = blockIdx.x * 32 + k;
  if (threadIdx.x == 0 && col < cols) dw[col] = accumulate ? dw[col] + v : v;
}

// Warps of a row's team with `vpl` vectors of 8 a lane.
int team_warps(int cols, int vpl) { return (cols + 256 * vpl - 1) / (256 * vpl); }

template <int VPL, typename S, bool FULL>
cudaError_t norm_launch(const RmsNormArgs &a, int W, cudaStream_t st) {
  const int teams = std::max(1, 8 / W);
  const unsigned grid = (unsigned)((a.rows + teams - 1) / teams);
  const dim3 block(32 * W * teams);
  switch (a.codes) {
    case MOE_CODES_MX:
      return launch_dependent(rms_norm_kernel<VPL, S, MOE_CODES_MX, FULL>, grid, block, 0, st, a, W, teams);
    case MOE_CODES_ACT8:
      return launch_dependent(rms_norm_kernel<VPL, S, MOE_CODES_ACT8, FULL>, grid, block, 0, st, a, W, teams);
    default:
      return launch_dependent(rms_norm_kernel<VPL, S, MOE_CODES_NONE, FULL>, grid, block, 0, st, a, W, teams);
  }
}

// Rows of the stream that 8 elements at a time start on their own size.
bool whole8(const void *p, int64_t ld, int elem) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % (8 * elem) == 0 && ld % 8 == 0);
}

template <int VPL, typename S>
cudaError_t norm_launch(const RmsNormArgs &a, cudaStream_t st) {
  const int W = team_warps(a.cols, VPL), elem = (int)sizeof(S);
  const bool full = W * VPL * 256 == a.cols && whole8(a.residual, a.ld_res, elem) && whole8(a.h, a.ldh, elem);
  return full ? norm_launch<VPL, S, true>(a, W, st) : norm_launch<VPL, S, false>(a, W, st);
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

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
// keeps both has codes of the tensor it computed with.  All sums and products are fp32; h is
// rounded to the stream's type, as the residual stream goes on with it, y to bf16.
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

// Makes w a new value to the compiler, so that what it was unpacked to before is not kept.
MOE_DEVINL void afresh(uint4 &w) { asm volatile("" : "+r"(w.x), "+r"(w.y), "+r"(w.z), "+r"(w.w)); }

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
// where rows are aligned to that (WIDE; halves of 16 bytes cost up to a quarter of the
// bandwidth: 2712 columns 5.7 and 6.4 TB/s).
template <typename S, bool WIDE>
struct Vec8;

template <bool WIDE>
struct Vec8<uint16_t, WIDE> {
  uint4 a;
  MOE_DEVINL void zero() { a = make_uint4(0, 0, 0, 0); }
  MOE_DEVINL void load(const uint16_t *p) { a = ld_stream_v4(p); }
  MOE_DEVINL void take(const uint4 *p) { a = p[0]; }
  MOE_DEVINL void again() { afresh(a); }
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

template <bool WIDE>
struct Vec8<float, WIDE> {
  Pairs v;
  MOE_DEVINL void zero() { v.zero(); }
  MOE_DEVINL void load(const float *p) {
    if (WIDE) {
      float f[8];
      ld_stream_f32x8(p, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) v.p[i] = pack2(f[2 * i], f[2 * i + 1]);
    } else {
      v = from_f32(ld_stream_v4(p), ld_stream_v4(p + 4));
    }
  }
  MOE_DEVINL void take(const uint4 *p) { v = from_f32(p[0], p[1]); }
  MOE_DEVINL void again() {}
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
    if (WIDE) {
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

// How the operands fit a kernel: fp32 rows start on 32 bytes, and the team's lanes have the
// columns exactly.
enum { kAny = 0, kWide = 1, kFull = 2 };

// What bounds it: HBM for bf16 output (16384 x 4096: 79 us, 6800 GB/s); with codes the issue of
// instructions came first (290 for 8 values a lane before the arithmetic in pairs, 80 us).
template <int VPL, typename S, int CODES, int FIT>
__global__ void __launch_bounds__(VPL > 2 ? 512 : 1024)
rms_norm_kernel(const RmsNormArgs a, int W, int teams) {
  constexpr bool FULL = FIT == kFull;
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
  Vec8<S, FIT != kAny> hv[VPL];
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
// Rows come in by asynchronous copies, `stages` of them a team: a warp copies what its own
// lanes will read (h, dy, d_residual), so that a warp's barrier is enough and loads stay
// under way while a row's sums are taken (16384 x 4096 bf16: 79 us, 6800 GB/s; without: 106
// us).  The row at hand is held in registers, as it came, so that its place is free for the
// next one before the sums (read twice from shared memory: 99 us).  DIRECT (wide fp32 rows,
// which would not fit beside the weights): d_residual is loaded past shared memory.
// Threads of a SM, as their registers go: 128 a thread, fewer where the row at hand is unpacked
// a second time (TIGHT) instead of kept in fp32.
constexpr int bwd_threads(int vpl, int elem, bool tight) {
  return !tight || vpl == 4 ? 512 : elem == 4 || vpl == 2 ? 768 : 1024;
}

template <int VPL, typename S, bool DIRECT, bool TIGHT>
__global__ void __launch_bounds__(bwd_threads(VPL, sizeof(S), TIGHT))
rms_norm_bwd_kernel(const RmsNormBwdArgs a, int W, int teams, int stages, float *__restrict__ part) {
  constexpr int kWide = sizeof(S) / 2;             // copies of a warp for 8 elements a lane
  constexpr int kDy = (DIRECT ? 1 : 2) * VPL * kWide;
  constexpr int kCopies = kDy + VPL;               // of a warp and row, 512 bytes each
  __shared__ float red[2][2][32];
  // [stages][warps][kCopies][512], then (four vectors a lane) the lanes' weights, each its own
  extern __shared__ __align__(16) uint8_t smem[];
  const Team t(W);
  constexpr bool kKeepW = VPL <= 2;
  const int c0 = t.warp * (256 * VPL) + t.lane * 8;
  auto in = [&](int v) { return c0 + 256 * v < a.cols; };
  Pairs dw[VPL], kept[kKeepW ? VPL : 1];  // kept: the weights
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
            if (!DIRECT && res != nullptr)
              copy_async(to + ((VPL + v) * kWide + k) * 512, res + ahead * a.ld_dres + c);
          }
        }
        if (in(v)) copy_async(to + (kDy + v) * 512, a.dy + ahead * a.ld_dy + c0 + 256 * v);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ahead += step;
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
  uint4 *own_w = reinterpret_cast<uint4 *>(smem + stages * stage) + threadIdx.x;
  if (!kKeepW) {
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      Pairs w;
      w.zero();
      if (in(v)) w = load_w(a.w, a.w_dtype, c0 + 256 * v);
      own_w[2 * v * blockDim.x] = *reinterpret_cast<const uint4 *>(&w.p[0]);
      own_w[(2 * v + 1) * blockDim.x] = *reinterpret_cast<const uint4 *>(&w.p[2]);
    }
  }
  auto weight = [&](int v) {
    if (kKeepW) return kept[v];
    return from_f32(own_w[2 * v * blockDim.x], own_w[(2 * v + 1) * blockDim.x]);
  };
  int turn = 0, s = 0;
  for (; row < a.rows; row += step, turn ^= 1) {
    Vec8<S, false> hv[VPL], rv[VPL];
    uint4 dy[VPL];
    if (DIRECT) {
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        rv[v].zero();
        if (res != nullptr && in(v)) rv[v].load(res + row * a.ld_dres + c0 + 256 * v);
      }
    }
    // all but the rows ahead have landed
    if (stages == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (stages == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      hv[v].zero();
      if (!DIRECT) rv[v].zero();
      dy[v] = make_uint4(0, 0, 0, 0);
      if (in(v)) {
        const uint4 *at = reinterpret_cast<const uint4 *>(mine + s * stage);
        hv[v].take(at + v * (kWide * 32) + t.lane * kWide);
        if (!DIRECT && res != nullptr) rv[v].take(at + (VPL + v) * (kWide * 32) + t.lane * kWide);
        dy[v] = at[(kDy + v) * 32 + t.lane];
      }
    }
    __syncwarp();
    fetch(s);  // (every lane has what was there)
    if (++s == stages) s = 0;
    uint64_t ss2 = 0, gh2 = 0;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const Pairs f = hv[v].get(), g = from_bf16(dy[v]), w = weight(v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ss2 = fma2(f.p[i], f.p[i], ss2);
        gh2 = fma2(mul2(g.p[i], w.p[i]), f.p[i], gh2);
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
    // dh = r g + m (h r) + d_residual: h r and r mean(g h) are of ordinary size for any eps, r^3 is
    // not (a row of zeros, eps under 2e-26: infinity times 0).  r = 0: the squares pass fp32's range,
    // the forward's y is constant there, and the mean, which may be no number, is left out.
    const float m = r == 0.0f ? 0.0f : -(r * (r * (gh / (float)a.cols)));
    const uint64_t r2 = pack2(r, r), m2 = pack2(m, m);
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int c = c0 + 256 * v;
      if (TIGHT) {
        hv[v].again();
        afresh(dy[v]);
      }
      const Pairs f = hv[v].get(), g = from_bf16(dy[v]), w = weight(v);
      Pairs d = rv[v].get();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t n = mul2(f.p[i], r2);
        dw[v].p[i] = fma2(g.p[i], n, dw[v].p[i]);
        d.p[i] = add2(fma2(m2, n, mul2(mul2(g.p[i], w.p[i]), r2)), d.p[i]);
      }
      if (in(v)) {
        Vec8<S, false> o;
        o.set(d);
        o.store(dh + row * a.ld_dh + c);
        if (a.dx != nullptr) st_v4(a.dx + row * a.ld_dx + c, to_bf16(d));
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

template <int VPL, typename S, int FIT>
cudaError_t norm_launch(const RmsNormArgs &a, int W, cudaStream_t st) {
  const int teams = std::max(1, 8 / W);
  const unsigned grid = (unsigned)((a.rows + teams - 1) / teams);
  const dim3 block(32 * W * teams);
  switch (a.codes) {
    case MOE_CODES_MX:
      return launch_dependent(rms_norm_kernel<VPL, S, MOE_CODES_MX, FIT>, grid, block, 0, st, a, W, teams);
    case MOE_CODES_ACT8:
      return launch_dependent(rms_norm_kernel<VPL, S, MOE_CODES_ACT8, FIT>, grid, block, 0, st, a, W, teams);
    default:
      return launch_dependent(rms_norm_kernel<VPL, S, MOE_CODES_NONE, FIT>, grid, block, 0, st, a, W, teams);
  }
}

// Rows of which 8 elements at a time start on their own size.
template <typename S>
bool whole8(const void *p, int64_t ld) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % (8 * sizeof(S)) == 0 && ld % 8 == 0);
}

template <int VPL, typename S>
cudaError_t norm_launch(const RmsNormArgs &a, cudaStream_t st) {
  const int W = team_warps(a.cols, VPL);
  const bool wide = whole8<S>(a.residual, a.ld_res) && whole8<S>(a.h, a.ldh);
  if (wide && W * VPL * 256 == a.cols) return norm_launch<VPL, S, kFull>(a, W, st);
  if (wide && sizeof(S) == 4) return norm_launch<VPL, S, kWide>(a, W, st);
  return norm_launch<VPL, S, kAny>(a, W, st);
}

// Vectors a lane, by the matrix alone, so that y is the same number with codes and without.  One
// while its warps are some half of what the GPU holds, for the latency (1000 x 1024: 3.1 us and with
// codes 3.4, four vectors 3.9 and 4.3; 100 x 7168 3.0 and 4.2; but 600 x 4096 with codes 6.1 and
// 5.9).  Else four (16384 x 4096: 79 us, one or two 82) but where a row has not so many (256
// columns: one 73 us, four 96; 512: two 80, four 83).
template <typename S>
cudaError_t norm_by_size(const RmsNormArgs &a, cudaStream_t st) {
  const bool few = a.rows * team_warps(a.cols, 1) <= 36ll * num_sms();
  if (few ? a.cols <= 8192 : a.cols <= 256) return norm_launch<1, S>(a, st);
  if (few || a.cols <= 512) return norm_launch<2, S>(a, st);
  return norm_launch<4, S>(a, st);
}

// How the backward is laid out: a lane's vectors, a block's teams, blocks of a SM, rows ahead.
// One vector where a row has no more (bf16 256 columns: 69 us, with two 83; fp32 128: 61 and 89,
// but 256: 119 and 109), four past 8192 columns.  TIGHT with two vectors: blocks of which one
// leaves a good part of the SM without threads and two fit so (5000 columns: 96 us, else 116;
// 4096: 91 and 85).  With four vectors the weights are kept in shared memory (read twice a row
// from L2 16384 columns took 129 us).
struct BwdShape {
  int vpl, W, teams, threads, per_sm, stages;
  bool direct, tight;
  size_t smem;
  BwdShape(int cols, int elem) {
    vpl = cols <= 512 / elem ? 1 : cols <= 8192 ? 2 : 4;
    W = team_warps(cols, vpl);
    teams = std::max(1, 8 / W);
    threads = 32 * W * teams;
    const size_t weights = vpl == 4 ? (size_t)threads * vpl * 32 : 0;
    direct = (size_t)threads * 8 * vpl * (2 + elem * 2) + weights > kBwdSmem;
    tight = vpl != 2 || (elem == 2 && threads > 256 && threads <= 384);
    const size_t stage = (size_t)threads * 8 * vpl * (2 + elem * (direct ? 1 : 2));
    // as many blocks as leave each two rows
    per_sm = std::max(1, bwd_threads(vpl, elem, tight) / threads);
    while (per_sm > 1 && kBwdSmem / per_sm < 2 * stage) --per_sm;
    stages = (int)std::min<size_t>(3, (kBwdSmem / per_sm - weights) / stage);
    smem = std::max(stage * stages + weights, (size_t)(teams - 1) * cols * sizeof(float));
  }
  static constexpr size_t kBwdSmem = 216 << 10;
};

// Blocks that the backward is launched with at most, of either type (its rows of `part`).
int64_t bwd_parts(int64_t rows, int cols) {
  const BwdShape b(cols, 2), f(cols, 4);
  const int64_t teams = std::min(b.teams, f.teams);
  return std::min<int64_t>((rows + teams - 1) / teams, 160 * std::max(b.per_sm, f.per_sm));
}

template <auto Kernel>
cudaError_t allow_smem() {
  static PerDevice<cudaError_t> done;
  return done.get(current_device(), [] {
    return cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)BwdShape::kBwdSmem);
  });
}

template <int VPL, typename S, bool DIRECT, bool TIGHT>
cudaError_t bwd_kernel(const RmsNormBwdArgs &a, const BwdShape &b, unsigned grid, float *part, cudaStream_t st) {
  const cudaError_t e = allow_smem<rms_norm_bwd_kernel<VPL, S, DIRECT, TIGHT>>();
  if (e != cudaSuccess) return e;
  return launch_dependent(rms_norm_bwd_kernel<VPL, S, DIRECT, TIGHT>, grid, b.threads, b.smem, st, a, b.W,
                          b.teams, b.stages, part);
}

template <typename S>
cudaError_t bwd_launch(const RmsNormBwdArgs &a, float *part, cudaStream_t st) {
  const BwdShape b(a.cols, (int)sizeof(S));
  const unsigned grid = (unsigned)std::min<int64_t>((a.rows + b.teams - 1) / b.teams, (int64_t)std::min(num_sms(), 160) * b.per_sm);
  cudaError_t e;
  if (b.vpl == 1) e = bwd_kernel<1, S, false, true>(a, b, grid, part, st);
  else if (b.vpl == 4 && b.direct) e = bwd_kernel<4, float, true, true>(a, b, grid, part, st);
  else if (b.vpl == 4) e = bwd_kernel<4, S, false, true>(a, b, grid, part, st);
  else if (sizeof(S) == 2 && b.tight) e = bwd_kernel<2, uint16_t, false, true>(a, b, grid, part, st);
  else e = bwd_kernel<2, S, false, false>(a, b, grid, part, st);
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

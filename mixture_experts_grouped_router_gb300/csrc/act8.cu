// Activation checkpoints in 8 bits, and the SwiGLU backward that reads them.
//
// A block of 32 consecutive elements of a row keeps one bf16 scale and 32
// signed 8-bit codes:
//     s = (max |x|) / 127 rounded up to bf16,   q = rne(x / s),   x ~ q s
// so that |q| <= 127 and the error is at most s / 2 an element.  A block whose
// largest magnitude is under 2^-100 keeps s = 0 (and reads as zeros); one that
// holds a NaN or an infinity keeps a NaN scale (and reads as NaN).  8.5 bits an
// element: 0.53 of the bf16 tensor.
//
// From the saved H = [g | u] of a SwiGLU (Act = silu(g) u), with the codes'
// values g', u' and dAct, the backward writes
//     dg = dAct u' sig (1 + g' (1 - sig)),   du = dAct g' sig,   sig = sigmoid(g')
// and, recomputed for the weight gradient of the down-projection, Act' =
// g' sig u'.  No bf16 copy of H is made in between.
//
// Every kernel streams: a warp takes 256 columns of a row at a time (8 elements
// = 16 bytes a lane, 4 lanes a block, the block's maximum by two shuffles) and
// keeps two to four 16-byte loads a lane in flight.  What bounds them: HBM, the
// quantising ones the issue of some 14 instructions a value as well (32768 rows,
// measured copy 6676 GB/s):
//   swiglu_bwd, F = 14336       778 us, 6110 GB/s
//   swiglu_fwd, F = 14336       604 us, 6320 GB/s (652 with a residual step after each
//       quotient; five resident blocks were 3% faster by themselves, but forward and
//       backward in turn 1.4% slower)
//   dequantize, 4096 columns     69 us, 6000 GB/s
//   quantize,   4096 columns     67 us, 6130 GB/s (eight resident blocks of two
//       loads a lane; four of four: 7% slower)
// Eight loads a lane are slower everywhere (registers).
#include <algorithm>

#include "internal.h"
#include "lowbit.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

// The warps' walk over (row, chunk of 256 columns): chunk c of warp w is c0 + w,
// then steps of all warps; a step is taken by additions alone.
struct Walk {
  int row, d_row, ch, d_ch, n_ch;
  MOE_DEVINL Walk(int chunks) : n_ch(chunks) {
    const int warp = (int)((blockIdx.x * kThreads + threadIdx.x) >> 5);
    const int warps = (int)gridDim.x * (kThreads / 32);
    row = warp / chunks;
    ch = warp - row * chunks;
    d_row = warps / chunks;
    d_ch = warps - d_row * chunks;
  }
  MOE_DEVINL void step() {
    row += d_row;
    ch += d_ch;
    if (ch >= n_ch) {
      ch -= n_ch;
      ++row;
    }
  }
};

MOE_DEVINL int live_rows(const int32_t *offsets, int E, int rows) {
  if (offsets == nullptr) return rows;
  return min(max(ld_i32(offsets + E), 0), rows);
}

__global__ void __launch_bounds__(kThreads, 8)
act8_quantize_kernel(const uint16_t *__restrict__ x, int ldx, int rows, int cols,
                     const int32_t *__restrict__ offsets, int E, int8_t *__restrict__ q,
                     int ldq, uint16_t *__restrict__ s, int lds) {
  constexpr int kU = 2;
  const int lane = threadIdx.x & 31;
  grid_dependency_begin();
  const int R = live_rows(offsets, E, rows);
  Walk w((cols + 255) / 256);
  while (w.row < R) {
    uint4 v[kU];
    int at[kU];
    int col[kU];
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      at[i] = w.row;
      col[i] = w.ch * 256 + lane * 8;
      v[i] = make_uint4(0, 0, 0, 0);
      if (w.row < R && col[i] < cols) v[i] = ld_stream_v4(x + (int64_t)w.row * ldx + col[i]);
      w.step();
    }
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      uint32_t sb;
      const uint2 c = act8_quantize8(v[i], sb);
      if (at[i] < R && col[i] < cols) {
        *reinterpret_cast<uint2 *>(q + (int64_t)at[i] * ldq + col[i]) = c;
        if ((lane & 3) == 0) s[(int64_t)at[i] * lds + (col[i] >> 5)] = (uint16_t)sb;
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads)
act8_dequantize_kernel(const int8_t *__restrict__ q, int ldq, const uint16_t *__restrict__ s,
                       int lds, int rows, int cols, const int32_t *__restrict__ offsets,
                       int E, uint16_t *__restrict__ x, int ldx) {
  const int lane = threadIdx.x & 31;
  grid_dependency_begin();
  const int R = live_rows(offsets, E, rows);
  Walk w((cols + 255) / 256);
  while (w.row < R) {
    uint2 c[kUnroll];
    uint32_t sb[kUnroll];
    int at[kUnroll];
    int col[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      at[i] = w.row;
      col[i] = w.ch * 256 + lane * 8;
      if (w.row < R && col[i] < cols) {
        c[i] = ld_stream_v2(q + (int64_t)w.row * ldq + col[i]);
        sb[i] = ld_u16(s + (int64_t)w.row * lds + (col[i] >> 5));
      }
      w.step();
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      if (at[i] < R && col[i] < cols) {
        float v[8];
        act8_values8(c[i], sb[i], v);
        st_v4(x + (int64_t)at[i] * ldx + col[i], f32_to_bf16x8(v));
      }
    }
  }
}

// h [rows, 2F] -> act [rows, F], codes [rows, 2F], scales [rows, 2 nb] (nb =
// ceil(F / 32); the up half's blocks start at nb, so that no block straddles).
__global__ void __launch_bounds__(kThreads)
act8_swiglu_fwd_kernel(const uint16_t *__restrict__ h, int ldh, int rows, int F,
                       const int32_t *__restrict__ offsets, int E, uint16_t *__restrict__ act,
                       int lda, int8_t *__restrict__ q, int ldq,
                       uint16_t *__restrict__ s, int lds) {
  constexpr int kU = kUnroll / 2;  // two loads a chunk
  const int lane = threadIdx.x & 31;
  const int nb = (F + 31) / 32;
  grid_dependency_begin();
  const int R = live_rows(offsets, E, rows);
  Walk w((F + 255) / 256);
  while (w.row < R) {
    uint4 g[kU], u[kU];
    int at[kU];
    int col[kU];
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      at[i] = w.row;
      col[i] = w.ch * 256 + lane * 8;
      g[i] = u[i] = make_uint4(0, 0, 0, 0);
      if (w.row < R && col[i] < F) {
        g[i] = ld_stream_v4(h + (int64_t)w.row * ldh + col[i]);
        u[i] = ld_stream_v4(h + (int64_t)w.row * ldh + F + col[i]);
      }
      w.step();
    }
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      uint32_t sg, su;
      const uint2 cg = act8_quantize8(g[i], sg);
      const uint2 cu = act8_quantize8(u[i], su);
      float fg[8], fu[8];
      bf16x8_to_f32(g[i], fg);
      bf16x8_to_f32(u[i], fu);
#pragma unroll
      for (int j = 0; j < 8; ++j) fg[j] = fg[j] * sigmoid_f(fg[j]) * fu[j];
      if (at[i] < R && col[i] < F) {
        st_v4(act + (int64_t)at[i] * lda + col[i], f32_to_bf16x8(fg));
        int8_t *qr = q + (int64_t)at[i] * ldq + col[i];
        *reinterpret_cast<uint2 *>(qr) = cg;
        *reinterpret_cast<uint2 *>(qr + F) = cu;
        if ((lane & 3) == 0) {
          uint16_t *sr = s + (int64_t)at[i] * lds + (col[i] >> 5);
          sr[0] = (uint16_t)sg;
          sr[nb] = (uint16_t)su;
        }
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads)
act8_swiglu_bwd_kernel(const int8_t *__restrict__ q, int ldq, const uint16_t *__restrict__ s,
                       int lds, const uint16_t *__restrict__ dact, int ldda,
                       int rows, int F, const int32_t *__restrict__ offsets, int E,
                       uint16_t *__restrict__ dh, int lddh, uint16_t *__restrict__ act,
                       int lda) {
  constexpr int kU = kUnroll / 2;
  const int lane = threadIdx.x & 31;
  const int nb = (F + 31) / 32;
  grid_dependency_begin();
  const int R = live_rows(offsets, E, rows);
  Walk w((F + 255) / 256);
  while (w.row < R) {
    uint2 cg[kU], cu[kU];
    uint4 da[kU];
    uint32_t sg[kU], su[kU];
    int at[kU];
    int col[kU];
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      at[i] = w.row;
      col[i] = w.ch * 256 + lane * 8;
      if (w.row < R && col[i] < F) {
        const int8_t *qr = q + (int64_t)w.row * ldq + col[i];
        const uint16_t *sr = s + (int64_t)w.row * lds + (col[i] >> 5);
        cg[i] = ld_stream_v2(qr);
        cu[i] = ld_stream_v2(qr + F);
        da[i] = ld_stream_v4(dact + (int64_t)w.row * ldda + col[i]);
        sg[i] = ld_u16(sr);
        su[i] = ld_u16(sr + nb);
      }
      w.step();
    }
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      if (at[i] < R && col[i] < F) {
        float g[8], u[8], d[8], a[8];
        act8_values8(cg[i], sg[i], g);
        act8_values8(cu[i], su[i], u);
        bf16x8_to_f32(da[i], d);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float sig = sigmoid_f(g[j]);
          const float silu = g[j] * sig;
          const float ds = d[j] * sig;
          a[j] = silu * u[j];
          const float dg = ds * u[j] * (1.0f + g[j] * (1.0f - sig));
          u[j] = d[j] * silu;
          g[j] = dg;
        }
        uint16_t *o = dh + (int64_t)at[i] * lddh + col[i];
        st_v4(o, f32_to_bf16x8(g));
        st_v4(o + F, f32_to_bf16x8(u));
        if (act != nullptr) st_v4(act + (int64_t)at[i] * lda + col[i], f32_to_bf16x8(a));
      }
    }
  }
}

// Launches a kernel's walk over rows x chunks of 256 columns: as many blocks as
// there is work for, no more than the GPU holds at a time.
template <auto Kernel, typename... Args>
cudaError_t run(int64_t rows, int cols, cudaStream_t st, Args... args) {
  const int64_t warps = rows * ((cols + 255) / 256);
  const int64_t blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t most = (int64_t)num_sms() * blocks_per_sm<Kernel>(kThreads);
  return launch_dependent(Kernel, (unsigned)std::max<int64_t>(1, std::min(blocks, most)), kThreads,
                          0, st, args...);
}

}  // namespace

cudaError_t launch_act8_quantize(const uint16_t *x, int64_t ldx, int64_t rows, int cols,
                                 const int32_t *offsets, int E, int8_t *q, int64_t ldq,
                                 uint16_t *s, int64_t lds, cudaStream_t st) {
  return run<act8_quantize_kernel>(rows, cols, st, x, (int)ldx, (int)rows, cols, offsets, E, q,
      (int)ldq, s, (int)lds);
}

cudaError_t launch_act8_dequantize(const int8_t *q, int64_t ldq, const uint16_t *s, int64_t lds,
                                   int64_t rows, int cols, const int32_t *offsets, int E,
                                   uint16_t *x, int64_t ldx, cudaStream_t st) {
  return run<act8_dequantize_kernel>(rows, cols, st, q, (int)ldq, s, (int)lds, (int)rows, cols,
      offsets, E, x, (int)ldx);
}

cudaError_t launch_act8_swiglu_fwd(const uint16_t *h, int64_t ldh, int64_t rows, int F,
                                   const int32_t *offsets, int E, uint16_t *act, int64_t lda,
                                   int8_t *q, int64_t ldq, uint16_t *s, int64_t lds,
                                   cudaStream_t st) {
  return run<act8_swiglu_fwd_kernel>(rows, F, st, h, (int)ldh, (int)rows, F, offsets, E, act,
      (int)lda, q, (int)ldq, s, (int)lds);
}

cudaError_t launch_act8_swiglu_bwd(const int8_t *q, int64_t ldq, const uint16_t *s, int64_t lds,
                                   const uint16_t *dact, int64_t ldda, int64_t rows, int F,
                                   const int32_t *offsets, int E, uint16_t *dh, int64_t lddh,
                                   uint16_t *act, int64_t lda, cudaStream_t st) {
  return run<act8_swiglu_bwd_kernel>(rows, F, st, q, (int)ldq, s, (int)lds, dact, (int)ldda,
      (int)rows, F, offsets, E, dh, (int)lddh, act, (int)lda);
}

}  // namespace moe

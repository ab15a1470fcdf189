// Microscaled 4-bit floating point: quantisation of activations (gathered
// through the permutation in the same pass) and weights, the scale layout the
// tensor cores read, and the way back.
//
// Two formats, both with E2M1 elements (0, .5, 1, 1.5, 2, 3, 4, 6 and a sign),
// packed two a byte, the even column in the low nibble:
//   MXFP4  blocks of 32 along a row, scale 2^s as E8M0 (OCP Microscaling v1.0):
//          s = floor(log2 max|x|) - 2
//   NVFP4  blocks of 16, scale E4M3(max|x| / (6 g)), and one fp32 scale g of
//          the tensor (or of each expert's weight); an element's value is
//          code * scale * g
// Elements round to nearest even and saturate.  A block that holds a NaN or an
// infinity takes a NaN scale and zero codes, and reads as NaN.
//
// Scales sit in 512-byte atoms of 128 rows x 4 blocks, which tcgen05.cp brings
// to tensor memory as they are: row r0 + 32 r1, block j at byte 16 r0 + 4 r1 +
// j; the atoms of a row of atoms follow one another, ceil(cols / (4 block)) of
// them, the last one's spare blocks zero.  Row maps: GROUPED (activations) and
// EXPERTS (weights), each group or expert padded to whole atoms, and SWIGLU, the
// fused up-projection with 32 gate rows and 32 up rows in turn.
//
// The kernels stream: a warp takes four chunks of 256 columns of a row (a lane 16
// bytes of each) and loads the next row's before it works on them.  What bounds
// them, 32768 rows of 4096 gathered from 16384 tokens, NVFP4, measured copy 6676 GB/s:
//   quantise    43 us with the linking (single launches 42 and 6): 208 MB would take 31;
//       the issue of some 16 instructions a value (two chunks a warp, or five or more
//       resident blocks, which leaves fewer registers: 54 to 72 us)
//   dequantise  58 us in a single launch, 6000 GB/s: HBM, mostly its writes
#include <algorithm>

#include "internal.h"
#include "lowbit.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;  // chunks of 256 columns a warp holds at a time
constexpr int kMaxE = 256;

// Padded row of row r of rows = E G under the maps that need no offsets.
MOE_DEVINL int weight_row(int r, int G, int row_map) {
  const int e = r / G, n = r - e * G;
  int m = n;
  if (row_map == MOE_FP4_ROWS_SWIGLU) {
    const int F = G / 2;
    const int f = n < F ? n : n - F;
    m = f / 32 * 64 + (n < F ? 0 : 32) + f % 32;
  }
  return e * ((G + 127) / 128 * 128) + m;
}

// The groups' first rows and their padded starts (sizes rounded up to 128), by
// the first warp of a block.  The offsets are clamped to [0, rows] and to their
// running maximum, so that a bad table names no row or atom that is not there.
struct Groups {
  int off[kMaxE + 1];
  int pad[kMaxE];
};

MOE_DEVINL void scan_groups(Groups &gr, const int32_t *offsets, int E, int64_t rows) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    auto offset = [&](int e) {
      return (int)min(max((int64_t)ld_i32(offsets + e), (int64_t)0), rows);
    };
    int top = offset(0), carry = 0;  // running maximum, padded rows so far
    for (int c0 = 0; c0 < E; c0 += 32) {
      const int e = c0 + lane;
      int hi = e < E ? offset(e + 1) : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, hi, o);
        if (lane >= o) hi = max(hi, y);
      }
      hi = max(hi, top);
      int lo = __shfl_up_sync(0xffffffffu, hi, 1);
      if (lane == 0) lo = top;
      const int p = (hi - lo + 127) / 128 * 128;
      int incl = p;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (e < E) {
        gr.off[e] = lo;
        gr.pad[e] = carry + incl - p;
        if (e == E - 1) gr.off[E] = hi;
      }
      carry += __shfl_sync(0xffffffffu, incl, 31);
      top = __shfl_sync(0xffffffffu, hi, 31);
    }
  }
}

// Padded row of row r < off[E], in the group that holds it (-1 before the first
// group); e: the group of an earlier row, advanced.
MOE_DEVINL int grouped_row(const Groups &gr, int &e, int r) {
  while (gr.off[e + 1] <= r) ++e;
  return gr.off[e] <= r ? gr.pad[e] + (r - gr.off[e]) : -1;
}

// A warp's walk over (row, segment of 4 chunks): additions only.
struct Walk {
  int row, seg, d_row, d_seg, segs;
  MOE_DEVINL Walk(int segments) : segs(segments) {
    const int warp = (int)((blockIdx.x * kThreads + threadIdx.x) >> 5);
    const int warps = (int)gridDim.x * kWarps;
    row = warp / segs;
    seg = warp - row * segs;
    d_row = warps / segs;
    d_seg = warps - d_row * segs;
  }
  MOE_DEVINL void step() {
    row += d_row;
    seg += d_seg;
    if (seg >= segs) {
      seg -= segs;
      ++row;
    }
  }
};

// The scale codes of a warp's chunk (the lane's block code in c) as the words
// of its atoms: a word is 4 blocks, 8 lanes of two per block (NVFP4) or 16
// lanes of four (MXFP4); every lane of a word returns it.
template <int FMT>
MOE_DEVINL uint32_t scale_word(uint32_t c, int lane) {
  constexpr int kSh = FMT == MOE_FP4_NV ? 1 : 2;  // log2 of lanes a block
  uint32_t v = c << (8 * ((lane >> kSh) & 3));
  v |= __shfl_xor_sync(0xffffffffu, v, 1 << kSh);
  v |= __shfl_xor_sync(0xffffffffu, v, 2 << kSh);
  return v;
}

// A warp's 4 chunks of 256 columns of a row (a lane 8 values of each, 16 bytes in,
// 4 bytes of codes out): the codes, and the words of the scale atoms (4 blocks
// each; the lanes that share a word all hold it).
template <int FMT, bool FEW>
MOE_DEVINL void quantize_chunks(const uint4 *w, int c0, int cols, int lane, float g, float inv6,
                                uint32_t *codes, uint32_t *words) {
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int c = c0 + 256 * i;
    codes[i] = words[i] = 0;
    if (c - lane * 8 >= cols) break;  // the whole chunk
    uint32_t a = amax_bits8(w[i]);
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
    if (FMT != MOE_FP4_NV) a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
    float inv, v[8];
    const uint32_t code =
        fp4_block_scale<FMT>(__uint_as_float(a << 16), g, 6.0f * g, inv6, inv);
    bf16x8_to_f32(w[i], v);
    codes[i] = fp4_codes8<FMT, FEW>(v, inv, code, g);
    words[i] = scale_word<FMT>(c < cols ? code : 0u, lane);
  }
}

template <int FMT>
MOE_DEVINL void quantize_piece(const uint4 *w, int c0, int cols, int lane, float g, float inv6,
                               uint32_t *codes, uint32_t *words) {
  if (FMT == MOE_FP4_MX || fp4_few_bits(g))
    quantize_chunks<FMT, true>(w, c0, cols, lane, g, inv6, codes, words);
  else
    quantize_chunks<FMT, false>(w, c0, cols, lane, g, inv6, codes, words);
}

// Stores a piece as row r, padded row pr.
template <int FMT>
MOE_DEVINL void store_piece(const uint32_t *codes, const uint32_t *words, int c0, int cols,
                            int lane, int r, int pr, int ac, uint8_t *q, int ldq,
                            uint8_t *sf) {
  constexpr int kLanes = FMT == MOE_FP4_NV ? 8 : 16;  // lanes of a word
  uint8_t *qr = q + (int64_t)r * ldq + (c0 >> 1);
  // atoms of 4 blocks follow one another 512 bytes apart
  uint8_t *sr = sf + fp4_scale_byte(pr, c0 / fp4_block(FMT), ac);
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    if (c0 + 256 * i < cols) {
      *reinterpret_cast<uint32_t *>(qr + 128 * i) = codes[i];
      if (lane % kLanes == 0)
        *reinterpret_cast<uint32_t *>(sr + i * (256 / fp4_atom_cols(FMT)) * 512) = words[i];
    }
  }
}

// A warp's piece of source row src (zeros where there is none).
MOE_DEVINL void load_piece(const uint16_t *x, int ldx, int src, int c0, int cols,
                           uint4 *w) {
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    w[i] = make_uint4(0, 0, 0, 0);
    if (src >= 0 && c0 + 256 * i < cols) w[i] = ld_stream_v4(x + (int64_t)src * ldx + c0 + 256 * i);
  }
}

// One warp, one piece of a row; the next row's loads are issued before this one
// is quantised, the first row's before the groups are scanned.
template <int FMT, bool GROUPED>
__global__ void __launch_bounds__(kThreads)
fp4_quantize_kernel(const uint16_t *__restrict__ x, int ldx, int src_rows,
                    const int32_t *__restrict__ row_index, int index_div, int rows, int cols,
                    int row_map, const int32_t *__restrict__ offsets, int E,
                    const float *__restrict__ gscale, uint8_t *__restrict__ q, int ldq,
                    uint8_t *__restrict__ sf, int32_t *dev_status) {
  __shared__ Groups gr;
  const int lane = threadIdx.x & 31;
  const int ac = (cols + fp4_atom_cols(FMT) - 1) / fp4_atom_cols(FMT);
  const int G = rows / max(E, 1);
  grid_dependency_begin();
  Walk w((cols + 256 * kUnroll - 1) / (256 * kUnroll));
  // the source row of row w.row (-1: zeros; one that x does not have likewise)
  auto source = [&](bool &bad) {
    int src = -1;
    if (w.row < rows) {
      src = w.row;
      if (row_index != nullptr) {
        const int i = ld_i32(row_index + w.row);
        src = i < 0 ? -1 : i / index_div;
      }
    }
    bad = src >= src_rows;
    return bad ? -1 : src;
  };
  uint4 cur[kUnroll];
  bool bad;
  load_piece(x, ldx, source(bad), w.seg * (256 * kUnroll) + lane * 8, cols, cur);
  int R = rows;
  if (GROUPED) {
    scan_groups(gr, offsets, E, rows);
    __syncthreads();
    R = gr.off[E];
  }
  const float g1 = FMT == MOE_FP4_NV && GROUPED && gscale != nullptr ? ld_f32(gscale) : 1.0f;
  const float inv6_1 = __frcp_rn(6.0f * g1);
  int e = 0;
  while (w.row < R) {
    const int r = w.row, c0 = w.seg * (256 * kUnroll) + lane * 8;
    if (bad && lane == 0) moe_set_status(dev_status, MOE_ERR_DEVICE);
    uint4 next[kUnroll];
    w.step();
    load_piece(x, ldx, source(bad), w.seg * (256 * kUnroll) + lane * 8, cols, next);
    const float g = FMT == MOE_FP4_NV && !GROUPED && gscale != nullptr ? ld_f32(gscale + r / G) : g1;
    const float inv6 = GROUPED ? inv6_1 : __frcp_rn(6.0f * g);
    const int pr = GROUPED ? grouped_row(gr, e, r) : weight_row(r, G, row_map);
    if (pr >= 0) {
      uint32_t codes[kUnroll], words[kUnroll];
      quantize_piece<FMT>(cur, c0, cols, lane, g, inv6, codes, words);
      store_piece<FMT>(codes, words, c0, cols, lane, r, pr, ac, q, ldq, sf);
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) cur[i] = next[i];
  }
}

// Top-k routing gathers every token k times.  With many rows each token is
// quantised once and stored k times instead: fp4_link_kernel threads the rows of
// a source row into a list (next[p] = the row before p and p's padded row), and
// fp4_quantize_linked_kernel walks the source rows.  Rows of zeros are spread over
// kZeroLists lists of their own.  The lists' order varies from run to run; what is
// stored does not.
constexpr int kZeroLists = 512;

__global__ void __launch_bounds__(kThreads)
fp4_link_kernel(const int32_t *__restrict__ row_index, int index_div, int64_t src_rows, int rows,
                const int32_t *__restrict__ offsets, int E, int32_t *__restrict__ head,
                int2 *__restrict__ next, int32_t *dev_status) {
  __shared__ Groups gr;
  grid_dependency_begin();
  scan_groups(gr, offsets, E, rows);
  __syncthreads();
  const int R = gr.off[E];
  int e = 0;
  for (int p = blockIdx.x * kThreads + threadIdx.x; p < R; p += gridDim.x * kThreads) {
    const int pr = grouped_row(gr, e, p);
    if (pr < 0) continue;
    const int i = ld_i32(row_index + p);
    int64_t src = i < 0 ? -1 : i / index_div;
    if (src >= src_rows) {
      moe_set_status(dev_status, MOE_ERR_DEVICE);
      src = -1;
    }
    if (src < 0) src = src_rows + p % kZeroLists;
    next[p] = make_int2(atomicExch(head + src, p), pr);
  }
}

template <int FMT>
__global__ void __launch_bounds__(kThreads)
fp4_quantize_linked_kernel(const uint16_t *__restrict__ x, int ldx, int src_rows, int cols,
                           const float *__restrict__ gscale, const int32_t *__restrict__ head,
                           const int2 *__restrict__ next, uint8_t *__restrict__ q, int ldq,
                           uint8_t *__restrict__ sf) {
  const int lane = threadIdx.x & 31;
  const int ac = (cols + fp4_atom_cols(FMT) - 1) / fp4_atom_cols(FMT);
  grid_dependency_begin();
  const int lists = src_rows + kZeroLists;
  Walk w((cols + 256 * kUnroll - 1) / (256 * kUnroll));
  auto load = [&](uint4 *v, int &p) {
    p = -1;
    if (w.row < lists) p = ld_i32(head + w.row);
    load_piece(x, ldx, p >= 0 && w.row < src_rows ? w.row : -1,
               w.seg * (256 * kUnroll) + lane * 8, cols, v);
  };
  const float g = FMT == MOE_FP4_NV && gscale != nullptr ? ld_f32(gscale) : 1.0f;
  const float inv6 = __frcp_rn(6.0f * g);
  uint4 cur[kUnroll];
  int p;
  load(cur, p);
  while (w.row < lists) {
    const int c0 = w.seg * (256 * kUnroll) + lane * 8;
    int at = p;
    int2 nx = make_int2(-1, 0);
    if (at >= 0) nx = ld_i32x2(next + at);
    uint4 ahead[kUnroll];
    w.step();
    load(ahead, p);
    if (at >= 0) {
      uint32_t codes[kUnroll], words[kUnroll];
      quantize_piece<FMT>(cur, c0, cols, lane, g, inv6, codes, words);
      while (at >= 0) {
        const int r = at, pr = nx.y;
        at = nx.x;
        if (at >= 0) nx = ld_i32x2(next + at);
        store_piece<FMT>(codes, words, c0, cols, lane, r, pr, ac, q, ldq, sf);
      }
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) cur[i] = ahead[i];
  }
}

// The way back: values (code * scale * g, rounded once to bf16).
template <int FMT, bool GROUPED>
__global__ void __launch_bounds__(kThreads)
fp4_dequantize_kernel(const uint8_t *__restrict__ q, int ldq, const uint8_t *__restrict__ sf,
                      int rows, int cols, int row_map, const int32_t *__restrict__ offsets, int E,
                      const float *__restrict__ gscale, uint16_t *__restrict__ x, int ldx) {
  __shared__ Groups gr;
  const int lane = threadIdx.x & 31;
  const int ac = (cols + fp4_atom_cols(FMT) - 1) / fp4_atom_cols(FMT);
  const int G = rows / max(E, 1);
  grid_dependency_begin();
  int R = rows;
  if (GROUPED) {
    scan_groups(gr, offsets, E, rows);
    __syncthreads();
    R = gr.off[E];
  }
  const float g1 = FMT == MOE_FP4_NV && GROUPED && gscale != nullptr ? ld_f32(gscale) : 1.0f;
  int e = 0;
  for (Walk w((cols + 256 * kUnroll - 1) / (256 * kUnroll)); w.row < R; w.step()) {
    const int r = w.row, c0 = w.seg * (256 * kUnroll) + lane * 8;
    const int pr = GROUPED ? grouped_row(gr, e, r) : weight_row(r, G, row_map);
    if (pr < 0) continue;
    const uint8_t *qr = q + (int64_t)r * ldq + (c0 >> 1);
    const uint8_t *sr = sf + fp4_scale_byte(pr, c0 / fp4_block(FMT), ac);
    uint32_t codes[kUnroll], sc[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      codes[i] = sc[i] = 0;
      if (c0 + 256 * i < cols) {
        codes[i] = ld_u32(qr + 128 * i);
        sc[i] = ld_u8(sr + i * (256 / fp4_atom_cols(FMT)) * 512);
      }
    }
    const float g = FMT == MOE_FP4_NV && !GROUPED && gscale != nullptr ? ld_f32(gscale + r / G) : g1;
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      if (c0 + 256 * i < cols) {
        float v[8];
        e2m1x8_to_f32(codes[i], v);
        // code times scale is exact (6 significant bits): one rounding by g, one to bf16
        const float t = fp4_scale_value(sc[i], FMT);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = FMT == MOE_FP4_NV ? v[j] * t * g : v[j] * t;
        st_v4(x + (int64_t)r * ldx + c0 + 256 * i, f32_to_bf16x8(v));
      }
    }
  }
}

// Weights w [E, K, N] (contraction down the rows) to K-major codes [E, N, K]:
// a block transposes 64 x 64 elements through shared memory; a thread then
// quantises 32 consecutive k of one column.  Run once when weights are laid out.
constexpr int kWT = 64;

template <int FMT>
__global__ void __launch_bounds__(128)
fp4_quantize_weights_kernel(const uint16_t *__restrict__ w, int K, int N, int row_map,
                            const float *__restrict__ gscale, uint8_t *__restrict__ q,
                            uint8_t *__restrict__ sf) {
  __shared__ uint16_t tile[kWT][kWT + 2];
  const int e = blockIdx.z, k0 = blockIdx.y * kWT, n0 = blockIdx.x * kWT;
  const uint16_t *src = w + (int64_t)e * K * N;
  for (int i = threadIdx.x; i < kWT * kWT; i += 128) {
    const int kk = i / kWT, nn = i % kWT;
    tile[kk][nn] = k0 + kk < K && n0 + nn < N ? src[(int64_t)(k0 + kk) * N + n0 + nn] : 0;
  }
  __syncthreads();
  const int nn = threadIdx.x & 63, kb = (threadIdx.x >> 6) * 32;
  const int n = n0 + nn, k = k0 + kb;
  if (n >= N) return;
  constexpr int kB = fp4_block(FMT);
  const int ac = (K + fp4_atom_cols(FMT) - 1) / fp4_atom_cols(FMT);
  const int pr = weight_row(e * N + n, N, row_map);
  const float g = FMT != MOE_FP4_NV || gscale == nullptr ? 1.0f : __ldg(gscale + e);
  uint32_t codes[4];
#pragma unroll
  for (int b = 0; b < 32 / kB; ++b) {
    uint32_t a = 0;
#pragma unroll
    for (int j = 0; j < kB; ++j) a = max(a, (uint32_t)tile[kb + b * kB + j][nn] & 0x7FFFu);
    float inv, v[kB];
    const uint32_t code = fp4_block_scale<FMT>(__uint_as_float(a << 16), g, 6.0f * g,
                                               __frcp_rn(6.0f * g), inv);
#pragma unroll
    for (int j = 0; j < kB; ++j)
      v[j] = __uint_as_float((uint32_t)tile[kb + b * kB + j][nn] << 16);
#pragma unroll
    for (int j = 0; j < kB / 8; ++j)
      codes[b * (kB / 8) + j] = fp4_few_bits(g) ? fp4_codes8<FMT, true>(v + 8 * j, inv, code, g)
                                                : fp4_codes8<FMT, false>(v + 8 * j, inv, code, g);
    const int blk = k / kB + b;
    if (blk < 4 * ac) sf[fp4_scale_byte(pr, blk, ac)] = k < K ? (uint8_t)code : (uint8_t)0;
  }
  if (k < K)
    *reinterpret_cast<uint4 *>(q + ((int64_t)e * N + n) * (K / 2) + k / 2) =
        make_uint4(codes[0], codes[1], codes[2], codes[3]);
  // the spare blocks of the last atom past this tile's columns (MXFP4 atoms
  // hold two tiles): zero
  if (kb == 0 && k0 + kWT >= K)
    for (int blk = (k0 + kWT) / kB; blk < 4 * ac; ++blk) sf[fp4_scale_byte(pr, blk, ac)] = 0;
}

// Row-order scales [rows, nb] of a 4-bit checkpoint into atoms (a thread one
// word of 4 blocks).
__global__ void __launch_bounds__(kThreads)
fp4_arrange_scales_kernel(const uint8_t *__restrict__ s, int64_t rows, int nb, int G,
                          int row_map, uint8_t *__restrict__ sf) {
  const int ac = (nb + 3) / 4;
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < rows * ac; i += stride) {
    const int64_t r = i / ac;
    const int b = (int)(i - r * ac) * 4;
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (b + j < nb) w |= (uint32_t)__ldg(s + r * nb + b + j) << (8 * j);
    *reinterpret_cast<uint32_t *>(sf + fp4_scale_byte(weight_row((int)r, G, row_map), b, ac)) = w;
  }
}

// A kernel as a value that a lambda can take.
template <auto Kernel>
struct K {
  static constexpr auto value = Kernel;
};

// Launches a kernel's walk over rows x segments of 4 chunks: as many blocks as
// there is work for, no more than the GPU holds at a time.
template <auto Kernel, typename... Args>
cudaError_t run(int64_t rows, int cols, cudaStream_t st, Args... args) {
  const int64_t warps = rows * ((cols + 256 * kUnroll - 1) / (256 * kUnroll));
  const int64_t most = (int64_t)num_sms() * blocks_per_sm<Kernel>(kThreads);
  const int64_t blocks = std::min((warps + kWarps - 1) / kWarps, most);
  return launch_dependent(Kernel, (unsigned)std::max<int64_t>(1, blocks), kThreads, 0, st,
                          args...);
}

}  // namespace

int64_t fp4_atom_rows(int64_t rows, int row_map, int E) {
  if (row_map == MOE_FP4_ROWS_GROUPED) return f8_padded_rows(rows, E) / 128;
  return (int64_t)E * ((rows / E + 127) / 128);
}

// Linked quantisation pays from so many gathered values on, for its two more
// launches (about 5 us): NVFP4, 32768 rows of 4096 from 16384 tokens 69 us directly, 43
// linked; MXFP4, 6216 rows of 7168 from 777 tokens 25 and 14 us; at 2^25 values, 8192
// rows of 4096 from 4096 tokens, 19.8 and 18.5 (MXFP4 19.5 and 17.4); at 2^24 the two are
// even, 4096 rows of 4096 from 2048 tokens 12.0 and 12.5, from 1024 11.8 and 11.6.
constexpr int64_t kLinkFrom = 1 << 24;

size_t fp4_quantize_workspace_bytes(int64_t src_rows, int64_t rows) {
  return (size_t)rows * sizeof(int2) + (size_t)(src_rows + kZeroLists) * sizeof(int32_t);
}

cudaError_t launch_fp4_quantize(const uint16_t *x, int64_t ldx, int64_t src_rows,
                                const int32_t *row_index, int index_div, int64_t rows, int cols,
                                int fmt, int row_map, const int32_t *offsets, int E,
                                const float *gscale, uint8_t *q, int64_t ldq, uint8_t *sf,
                                void *ws, size_t ws_bytes, int32_t *dev_status, cudaStream_t st) {
  const bool grouped = row_map == MOE_FP4_ROWS_GROUPED;
  if (grouped && row_index != nullptr && rows >= 2 * src_rows && rows * cols >= kLinkFrom &&
      ws != nullptr && ws_bytes >= fp4_quantize_workspace_bytes(src_rows, rows)) {
    int2 *next = static_cast<int2 *>(ws);
    int32_t *head = reinterpret_cast<int32_t *>(next + rows);
    cudaError_t e = cudaMemsetAsync(head, 0xFF, (size_t)(src_rows + kZeroLists) * 4, st);
    if (e != cudaSuccess) return e;
    const int lg = (int)std::min<int64_t>((rows + kThreads - 1) / kThreads, (int64_t)num_sms() * 4);
    e = launch_dependent(fp4_link_kernel, lg, kThreads, 0, st, row_index, index_div, src_rows,
                         (int)rows, offsets, E, head, next, dev_status);
    if (e != cudaSuccess) return e;
    auto link = [&](auto kernel) {
      return run<kernel.value>(src_rows + kZeroLists, cols, st, x, (int)ldx, (int)src_rows, cols,
                               gscale, (const int32_t *)head, (const int2 *)next, q, (int)ldq, sf);
    };
    return fmt == MOE_FP4_NV ? link(K<fp4_quantize_linked_kernel<MOE_FP4_NV>>{})
                             : link(K<fp4_quantize_linked_kernel<MOE_FP4_MX>>{});
  }
  auto go = [&](auto kernel) {
    return run<kernel.value>(rows, cols, st, x, (int)ldx, (int)src_rows, row_index, index_div,
                             (int)rows, cols, row_map, offsets, E, gscale, q, (int)ldq, sf,
                             dev_status);
  };
  if (fmt == MOE_FP4_NV)
    return grouped ? go(K<fp4_quantize_kernel<MOE_FP4_NV, true>>{})
                   : go(K<fp4_quantize_kernel<MOE_FP4_NV, false>>{});
  return grouped ? go(K<fp4_quantize_kernel<MOE_FP4_MX, true>>{})
                 : go(K<fp4_quantize_kernel<MOE_FP4_MX, false>>{});
}

cudaError_t launch_fp4_dequantize(const uint8_t *q, int64_t ldq, const uint8_t *sf, int64_t rows,
                                  int cols, int fmt, int row_map, const int32_t *offsets, int E,
                                  const float *gscale, uint16_t *x, int64_t ldx,
                                  cudaStream_t st) {
  const bool grouped = row_map == MOE_FP4_ROWS_GROUPED;
  auto go = [&](auto kernel) {
    return run<kernel.value>(rows, cols, st, q, (int)ldq, sf, (int)rows, cols, row_map, offsets, E,
                             gscale, x, (int)ldx);
  };
  if (fmt == MOE_FP4_NV)
    return grouped ? go(K<fp4_dequantize_kernel<MOE_FP4_NV, true>>{})
                   : go(K<fp4_dequantize_kernel<MOE_FP4_NV, false>>{});
  return grouped ? go(K<fp4_dequantize_kernel<MOE_FP4_MX, true>>{})
                 : go(K<fp4_dequantize_kernel<MOE_FP4_MX, false>>{});
}

cudaError_t launch_fp4_quantize_weights(const uint16_t *w, int E, int K, int N, int fmt,
                                        int row_map, const float *gscale, uint8_t *q, uint8_t *sf,
                                        cudaStream_t st) {
  const dim3 grid((N + kWT - 1) / kWT, (K + kWT - 1) / kWT, E);
  if (fmt == MOE_FP4_NV)
    fp4_quantize_weights_kernel<MOE_FP4_NV><<<grid, 128, 0, st>>>(w, K, N, row_map, gscale, q, sf);
  else
    fp4_quantize_weights_kernel<MOE_FP4_MX><<<grid, 128, 0, st>>>(w, K, N, row_map, gscale, q, sf);
  return cudaGetLastError();
}

cudaError_t launch_fp4_arrange_scales(const uint8_t *s, int64_t rows, int nb, int E, int row_map,
                                      uint8_t *sf, cudaStream_t st) {
  const int64_t words = rows * ((nb + 3) / 4);
  const int grid = (int)std::max<int64_t>(
      1, std::min<int64_t>((words + kThreads - 1) / kThreads, (int64_t)num_sms() * 8));
  fp4_arrange_scales_kernel<<<grid, kThreads, 0, st>>>(s, rows, nb, (int)(rows / E), row_map, sf);
  return cudaGetLastError();
}

}  // namespace moe

// Grouped GEMM of the expert FFN on 4-bit block-scaled codes (MXFP4, NVFP4):
// for every expert e, rows [off_e, off_e+1) of A times B_e^T, both K-major E2M1
// codes with their scales applied by the tensor cores
// (tcgen05.mma kind::mxf4nvf4.block_scale), fp32 accumulators in tensor memory.
//
// The product runs transposed: the weight's rows are the MMA's M (256, a pair of
// CTAs), the expert's tokens its N, 16 to 256 in steps of 16.  An expert's last
// tokens then cost what they are (a row tile of tokens would round them up to
// 256), a single token costs N = 16, and the weights, which are what few tokens
// wait for, fill every stage.
//
// Epilogues: plain (times the tensors' fp32 scales, to bf16 or fp32), and the
// SwiGLU forward, which quantises Act = silu(g) u to 4 bits straight from the
// fp32 accumulators, so that the down-projection's operand leaves the kernel as
// codes and scales instead of bf16 that another pass would read again.  Gate and
// up rows alternate in blocks of 32 along M: one warp holds a block's gates, its
// neighbour the ups.  A block of 32 weight rows x 32 tokens is turned through
// shared memory, and leaves as rows of tokens.
//
// With many rows an expert and a short contraction the SwiGLU product runs the
// other way round (kRows: M = 256 tokens, N = 192 weight rows): a thread then holds
// a token's gates and ups of 32 features and quantises them without the shared
// memory whose bandwidth the turned blocks share with the MMAs' operands.
//
// Persistent; clusters of two CTAs issue 2-SM MMAs (M = 256, K = 64 codes = 32
// bytes).  A stage is a K block of 256 codes (one 128-byte swizzle row a row): a
// CTA's 128 weight rows 16 KB, its half of the tokens up to 16 KB (in boxes of 32
// rows), and the K block's scale atoms (512 bytes of 128 rows x 4 blocks): 4
// (NVFP4) or 2 (MXFP4) for the weight rows and twice as many for 256 tokens.
//   warp 0     TMA producer
//   warp 1     tensor memory, and in the leader CTA the MMA issue: the atoms
//              to tensor memory (tcgen05.cp), then four MMAs.  A tile's shape comes
//              from the producer with the tile's first stage
//   warps 2-9  epilogue, two per quarter of the tensor-memory lanes, which take the
//              tile's chunks of 32 tokens in turn (kRows: warps 2-5)
// Tensor memory: two accumulators of 256 columns, at 0 and at 160, that share 96.
// The epilogue reads those first, and the next tile's products wait until it has
// (for some 700 cycles) if either tile needs them: one tile of 256 tokens instead of two
// of 192 and 64 saves a pass over the weights (8192 rows of 32 experts, NVFP4:
// 7168 x 4096 133 -> 110 us) and takes longer MMAs a K block (32768 rows of 8,
// 14336 x 4096 606 -> 546 us).  kRows: two of 192.
// The scale slots are in the columns that they leave: 48 columns a K block (NVFP4, 2
// slots) or 24 (MXFP4, 4).  A slot is rewritten after the MMAs that read it are
// done: their commit arrives on the full barrier of the K block that takes the slot
// next, beside the stage's copies, so that the issuer has one barrier to wait for.
// That wait and the issue set the pace below 192 tokens (there a K block's MMAs take 384
// cycles, at 256 512; its issue some 280 and its wait 60): the next barrier is
// tested between two blocks, the issuing warp stays uniform, elect_one() choosing the
// lane, its descriptors differ by constants, and it looks up no tile (those two:
// 1095 -> 1046 us MXFP4, 1345 -> 1222 NVFP4, 32768 rows, 4096 x 28672 with SwiGLU;
// two K blocks an iteration were no faster).  The epilogue hands its columns back by
// arrivals that order no memory: releasing ones waited for its global stores (8192
// rows of 32 experts, NVFP4: 7168 x 4096 110 -> 100 us, 2048 x 7168 90 -> 68 us).
// At 8 experts and 32768 rows: 14336 x 4096 0.51 ms = 7.5 PFLOP/s (MXFP4), 0.53 ms = 7.3
// (NVFP4); 4096 x 28672 with SwiGLU 1.07 and 1.14 ms (ragged groups), 7.2 and 6.7.
// Few tokens wait for the weights: 3 or 4 each of 32 experts, 7168 x 4096 80 us, 6.2 TB/s.
// A tile of one K block and up to 32 tokens takes 0.75 us (SwiGLU 0.84): tiles are looked
// up by a ballot and the scales of the weights are in shared memory (1.32 -> 1.02 us),
// and the two warps of a quarter change places from tile to tile (-> 0.75).
// Every wait is bounded; on time-out the CTA winds down and reports
// MOE_ERR_TIMEOUT through dev_status.
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "internal.h"
#include "lowbit.cuh"
#include "tc_fp4_sm103.cuh"

namespace moe {
namespace {

constexpr int BW = 256;        // weight rows of a tile (the pair's M)
constexpr int BT = 256;        // most tokens of a tile (N)
constexpr int kRowBytes = 128; // one K block of a row: 256 codes
constexpr int kKSteps = 4;     // MMAs a K block
constexpr int W_BYTES = BW / 2 * kRowBytes;
constexpr int kStgBytes = 4096;  // staging of an epilogue warp: one 32 x 32 fp32 block
constexpr int kMaxE = 256;
constexpr int kTmemCols = 512;

// EPI: MOE_EPI_NONE, MOE_EPI_SWIGLU_FWD, or kRows (SwiGLU with tokens as M, whose
// epilogue needs no staging).
constexpr int kRows = 3;
constexpr int BR = 192;        // its weight rows of a tile (N): 96 features

template <int FMT, int EPI>
struct Lay {
  static constexpr int epi_warps = EPI == kRows ? 4 : 8;
  static constexpr int threads = 64 + 32 * epi_warps;
  static constexpr int stages = EPI == kRows ? 6 : 5;
  static constexpr int t_bytes = (EPI == kRows ? BR : BT) / 2 * kRowBytes;
  static constexpr int atoms = 256 / fp4_atom_cols(FMT);  // atom columns a K block
  static constexpr int sfw_bytes = atoms * 512;
  static constexpr int sft_bytes = 2 * sfw_bytes;
  static constexpr int stage_bytes = (W_BYTES + t_bytes + sfw_bytes + sft_bytes + 1023) / 1024 * 1024;
  static constexpr int sf_cols = atoms * 12;               // tensor-memory columns a slot
  // the second accumulator's first column, and the scale slots'
  static constexpr int acc_step = EPI == kRows ? BR : 160;
  static constexpr int sf_base = acc_step + (EPI == kRows ? BR : BT);
  static constexpr int sf_slots = (kTmemCols - sf_base) / sf_cols;
  static_assert(sf_slots <= stages, "a commit names a K block's next user by its stage");
  static constexpr int stg_offset = stages * stage_bytes;
  static constexpr int book_offset =
      stg_offset + (EPI == kRows ? 0 : epi_warps * kStgBytes);
};

constexpr int kMaxStages = 6;

struct Book {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t shared_read;  // the columns that both accumulators use have been read
  uint64_t drain;
  uint32_t tmem_base;
  uint32_t shape[kMaxStages];  // mma_shape of the tile that begins in the stage
  int abort_flag;
  int total_tiles;
  int off[kMaxE + 1];        // group offsets, clamped to [0, rows_cap]
  int cum[kMaxE + 1];        // per-expert tile prefix
  uint16_t poff[kMaxE + 1];  // padded group starts in units of 128 rows
  float gb[kMaxE];           // the weights' fp32 scales
};

template <int FMT, int EPI>
constexpr int smem_bytes() {
  return 1024 + Lay<FMT, EPI>::book_offset + (int)((sizeof(Book) + 127) / 128 * 128);
}
static_assert(smem_bytes<MOE_FP4_NV, MOE_EPI_NONE>() <= 232448, "shared memory of one CTA");
static_assert(smem_bytes<MOE_FP4_MX, MOE_EPI_NONE>() <= 232448, "shared memory of one CTA");
static_assert(smem_bytes<MOE_FP4_NV, kRows>() <= 232448, "shared memory of one CTA");

struct Fp4Params {
  int E, rows_cap, N, F, w_tiles, w_atoms, kblocks;
  const int32_t *offsets;
  void *C;
  int64_t ldc;
  int c_f32;
  uint8_t *Q2;        // SwiGLU: codes and scale atoms of Act
  int64_t ldq2;
  uint8_t *sf2;
  int ac2;            // atom columns of Act
  int atom_rows2;     // atom rows of Act
  const float *g2;    // fp32 scale that Act is quantised with (or null: 1)
  const float *ga, *gb;  // fp32 scales of A (one) and B (one an expert), or null: 1
  int32_t *dev_status;
  uint64_t wait_limit_ns;
  int stall_loads;
  int early;          // offsets and weights may be read before the kernel before is done
};

struct Maps {
  CUtensorMap w;     // weight codes
  CUtensorMap t[4];  // token codes, boxes of 32, 64, 96 and 128 rows
  CUtensorMap sw;    // weight scale atoms
  CUtensorMap st[2]; // token scale atoms, boxes of one and two atom rows
  CUtensorMap c;     // plain output (no other form reads it)
};

struct TileInfo {
  int e, w_idx;      // expert, weight tile
  int t0;            // first token within the group (a multiple of 64)
  int row0, tokens;  // its row, and the tile's tokens (1 to 256)
  int n;             // tokens rounded up to the MMA's step of 16
};

MOE_DEVINL int group_offset(const Fp4Params &p, int e) {
  return min(max(ld_i32(p.offsets + e), 0), p.rows_cap);
}

// The expert of tile t: the last one whose tiles begin at or before it (a warp's
// lanes look at one expert each; the result is uniform).
MOE_DEVINL int tile_expert(const Book &bk, const Fp4Params &p, int t) {
  int n = 0;
  for (int e0 = 0; e0 < p.E; e0 += 32) {
    const int e = e0 + (int)(threadIdx.x & 31);
    n += __popc(__ballot_sync(0xffffffffu, e < p.E && bk.cum[e] <= t));
  }
  return n - 1;
}

// Tile t: an expert's token tiles follow one another under one weight tile, so
// that the pairs that run at a time share its rows in L2.  They are as few as can be
// and of like size, in steps of 64 tokens: 192 and up to 192 rather than 256 and up
// to 128 (the scale atoms of their tokens then start in row 0 or in row 64).
MOE_DEVINL TileInfo decode_tile(const Book &bk, const Fp4Params &p, int t) {
  TileInfo ti;
  ti.e = tile_expert(bk, p, t);
  const int off = tc::uniform(bk.off[ti.e]);
  const int size = tc::uniform(max(bk.off[ti.e + 1], off)) - off;
  const int local = t - tc::uniform(bk.cum[ti.e]);
  ti.w_idx = local;
  ti.t0 = 0;
  ti.tokens = size;
  if (size > BT) {
    const int tt = (size + BT - 1) / BT;
    const int step = ((size + tt - 1) / tt + 63) & ~63;
    ti.w_idx = local / tt;
    ti.t0 = (local - ti.w_idx * tt) * step;
    ti.tokens = min(size - ti.t0, step);
  }
  ti.row0 = off + ti.t0;
  ti.n = (ti.tokens + 15) / 16 * 16;
  return ti;
}

// The tile's first token sits in row 0 of an atom, or in row 64 (two scale
// columns on); whether its tokens reach into a second one.
MOE_DEVINL int scale_shift(const TileInfo &ti) { return ti.t0 & 127 ? 2 : 0; }
MOE_DEVINL bool second_atom(const TileInfo &ti) { return scale_shift(ti) * 32 + ti.n > 128; }

// A tile's MMAs as the producer hands them to the issuing warp: N, the scale
// column that the tokens start in, whether they reach into a second atom.
MOE_DEVINL uint32_t mma_shape(int n, int shift, bool second) {
  return (uint32_t)n | (uint32_t)shift << 16 | (uint32_t)second << 24;
}

// ---------------------------------------------------------------- epilogue
// Thread `r`'s 32 values become column r of a 32 x 32 block (block row j = value
// j), as the TMA store reads it: bf16 rows of 64 bytes under the 64-byte swizzle.
// Lanes r and r ^ 1 trade a value a row pair and write 32-bit words, free of
// bank conflicts.
MOE_DEVINL void stage_bf16_t(uint8_t *buf, int r, const float *v) {
  const bool odd = r & 1;
  const int off = ((r >> 1) & 3) * 4;  // byte of the word within its 16-byte chunk
  const int chunk = r >> 3;
#pragma unroll
  for (int m = 0; m < 16; ++m) {
    const float recv = __shfl_xor_sync(0xffffffffu, odd ? v[2 * m] : v[2 * m + 1], 1);
    const int n = 2 * m + (odd ? 1 : 0);
    const __nv_bfloat162 w = odd ? __floats2bfloat162_rn(recv, v[2 * m + 1])
                                 : __floats2bfloat162_rn(v[2 * m], recv);
    *reinterpret_cast<__nv_bfloat162 *>(buf + n * 64 + ((chunk ^ ((n >> 1) & 3)) << 4) + off) = w;
  }
}

// The same in fp32: rows of 128 bytes under the 128-byte swizzle.
MOE_DEVINL void stage_f32_t(uint8_t *buf, int r, const float *v) {
#pragma unroll
  for (int j = 0; j < 32; ++j)
    *reinterpret_cast<float *>(buf + j * 128 + (((r >> 2) ^ (j & 7)) << 4) + (r & 3) * 4) = v[j];
}

// 16 fp32 values from 16 h on of row r of such a block.
MOE_DEVINL void unstage_f32_16(const uint8_t *buf, int r, int h, float *v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 w = *reinterpret_cast<const float4 *>(buf + r * 128 + (((4 * h + i) ^ (r & 7)) << 4));
    v[4 * i] = w.x;
    v[4 * i + 1] = w.y;
    v[4 * i + 2] = w.z;
    v[4 * i + 3] = w.w;
  }
}

// Two neighbouring epilogue warps (a block's gates and its ups) meet.
MOE_DEVINL void pair_sync(int pair) {
  asm volatile("bar.sync %0, 64;" ::"r"(1 + pair) : "memory");
}

// The same, with one verdict for both.
MOE_DEVINL bool pair_agree(bool ok, int pair) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, 64, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)ok), "r"(1 + pair)
      : "memory");
  return r != 0;
}

// A warp's chunks of 32 tokens, every other one from `first` on (the two warps of a
// quarter change places from tile to tile, so that those of one chunk overlap), those of the columns that the two
// accumulators share first: the last ones of the lower accumulator (a = 0), the first
// ones of the upper.  Its first two are loaded together, after which the next tile's
// products may take the shared columns; then one is always on its way.
struct Chunks {
  uint32_t taddr;
  int n, a, first;  // chunks of the tile, accumulator
  uint32_t cur[32], nxt[32];

  MOE_DEVINL int at(int i) const { return a ? i : n - 1 - i; }
  MOE_DEVINL void begin(uint32_t shared_read, int lane) {
    if (first < n) tc::tmem_ld32_issue(taddr + at(first) * 32, cur);
    if (first + 2 < n) tc::tmem_ld32_issue(taddr + at(first + 2) * 32, nxt);
    tc::tmem_wait_ld(cur);
    tc::reg_after(nxt);
    tc::tc_fence_before();
    __syncwarp();
    if (lane == 0) tc::mbar_arrive_cluster_relaxed(shared_read);
  }
  // after chunk i's values have been taken
  MOE_DEVINL void advance(int i) {
    tc::tmem_wait_ld(nxt);
#pragma unroll
    for (int j = 0; j < 32; ++j) cur[j] = nxt[j];
    if (i + 4 < n) tc::tmem_ld32_issue(taddr + at(i + 4) * 32, nxt);
  }
};

// SwiGLU: warp q holds the gates (q even) or ups (q odd) of 32 features for the
// tile's tokens.  A chunk of 32 tokens goes through the two warps' staging; a
// thread then has one token's gates and ups of 16 features, which are a block of
// NVFP4 or half a block of MXFP4, whose other half is its neighbour's.  The
// values are continuous, so that no quotient sits on a tie and a product with the
// reciprocal decides as the quotient would.
template <int FMT>
MOE_DEVINL void epilogue_swiglu(const Book &bk, const Fp4Params &p, const TileInfo &ti, float sc,
                                float g2, float inv6, Chunks &ch, int crank, int q, int sub,
                                int lane, uint8_t *stg_pair) {
  const int F = p.F;
  // the pair of warps' 32 features
  const int f0 = ti.w_idx * (BW / 2) + crank * (BW / 4) + (q >> 1) * 32;
  if (f0 >= F) return;
  const int pair = 2 * sub + (q >> 1);
  const int tok = (q & 1) * 16 + (lane >> 1), h = lane & 1;
  const int fh = f0 + 16 * h;  // this thread's features
#pragma unroll 1
  for (int i = ch.first; i < ch.n; i += 2) {
    const int c = ch.at(i);
    {
      float v[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(ch.cur[j]) * sc;
      if (i > ch.first) pair_sync(pair);  // both warps are done with the last chunk
      stage_f32_t(stg_pair + (q & 1) * kStgBytes, lane, v);
    }
    ch.advance(i);
    pair_sync(pair);
    float g[16], u[16];
    unstage_f32_16(stg_pair, tok, h, g);
    unstage_f32_16(stg_pair + kStgBytes, tok, h, u);
    const int t = c * 32 + tok;  // token of the tile
    const int64_t row = (int64_t)ti.row0 + t;
    const bool valid = t < ti.tokens;
    if (p.C != nullptr && valid) {  // H in bf16 as well
      uint16_t *H = static_cast<uint16_t *>(p.C) + row * p.ldc + fh;
      st_v4(H, f32_to_bf16x8(g));
      st_v4(H + 8, f32_to_bf16x8(g + 8));
      st_v4(H + F, f32_to_bf16x8(u));
      st_v4(H + F + 8, f32_to_bf16x8(u + 8));
    }
    float a = 0.0f;
    bool finite = true;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      g[j] = g[j] * sigmoid_f(g[j]) * u[j];
      const float m = fabsf(g[j]);
      finite &= m <= 3.402823466e38f;
      a = fmaxf(a, m);
    }
    if (!finite) a = __uint_as_float(0x7F800000u);
    if (FMT != MOE_FP4_NV) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
    float inv;
    const uint32_t scale = fp4_block_scale<FMT>(a, g2, 6.0f * g2, inv6, inv);
#pragma unroll
    for (int j = 0; j < 16; ++j) g[j] *= inv;
    const uint32_t lo = inv == 0.0f ? 0u : cvt_e2m1x8(g);
    const uint32_t hi = inv == 0.0f ? 0u : cvt_e2m1x8(g + 8);
    // the row's place in Act's scale atoms
    const int pr = ti.t0 + t;
    const int arow = (int)bk.poff[ti.e] + (pr >> 7);
    if (valid && arow < p.atom_rows2) {
      *reinterpret_cast<uint2 *>(p.Q2 + row * p.ldq2 + (fh >> 1)) = make_uint2(lo, hi);
      uint8_t *srow = p.sf2 + (int64_t)arow * p.ac2 * 512 + (pr & 31) * 16 + ((pr >> 5) & 3) * 4;
      const int b = fh / fp4_block(FMT);
      if (FMT == MOE_FP4_NV || h == 0) srow[(b >> 2) * 512 + (b & 3)] = (uint8_t)scale;
      if (f0 + 32 >= F && h == 0)  // the last atom's spare blocks
        for (int x = F / fp4_block(FMT); x < 4 * p.ac2; ++x)
          srow[(x >> 2) * 512 + (x & 3)] = 0;
    }
  }
}

// Plain: warp q holds 32 output columns of the tile's tokens.
MOE_DEVINL void epilogue_plain(const Fp4Params &p, const TileInfo &ti, float sc, Chunks &ch,
                               int crank, int q, int sub, int lane, uint8_t *stg,
                               const CUtensorMap *m0) {
  const int nc = ti.w_idx * BW + crank * (BW / 2) + q * 32;
  if (nc >= p.N) return;
#pragma unroll 1
  for (int i = ch.first; i < ch.n; i += 2) {
    const int c = ch.at(i);
    float v[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(ch.cur[j]) * sc;
    ch.advance(i);
    const int left = ti.tokens - c * 32;  // rows of this block that are the tile's
    const int r0 = ti.row0 + c * 32;
    // bf16 blocks take the staging's halves in turn (from the first one on, once
    // the last tile's stores have read them), fp32 ones all of it
    uint8_t *buf = p.c_f32 ? stg : stg + (i >> 1 & 1) * 2048;
    if (lane == 0) {
      if (p.c_f32 || i == ch.first) tc::bulk_wait_read0();
      else tc::bulk_wait_read<1>();
    }
    __syncwarp();
    if (p.c_f32) stage_f32_t(buf, lane, v);
    else stage_bf16_t(buf, lane, v);
    if (left >= 32) {
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tc::tma_store_2d(m0, buf, nc, r0);
        tc::bulk_commit();
      }
    } else {  // rows past the group are the next expert's
      __syncwarp();
      // a row's 16-byte chunks: 4 (bf16) or 8 (fp32), one a lane
      const int sh = p.c_f32 ? 3 : 2, es = p.c_f32 ? 4 : 2;
      const int k = lane & ((1 << sh) - 1), first = lane >> sh, step = 32 >> sh;
      const bool in = nc + k * (16 / es) < p.N;
      uint8_t *o = static_cast<uint8_t *>(p.C) +
                   ((int64_t)(r0 + first) * p.ldc + nc) * es + k * 16;
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const int r = first + x * step;
        if (r < left && in) {
          const int at =
              p.c_f32 ? r * 128 + ((k ^ (r & 7)) << 4) : r * 64 + ((k ^ ((r >> 1) & 3)) << 4);
          st_v4(o + (int64_t)x * step * p.ldc * es, *reinterpret_cast<const uint4 *>(buf + at));
        }
      }
      __syncwarp();
    }
  }
}

// ------------------------------------------- SwiGLU with many rows an expert
// The same pipeline with the roles exchanged: a CTA's 128 tokens are its share of
// M, the pair's 192 weight rows N, 96 to a CTA, alternating gates and ups in blocks
// of 32.  A tile of 192 rows starts in row 0 or 64 of its scale atoms.
struct RowTile {
  int e, m_idx, n_idx, row0, row_end;
};

constexpr int kGroupPairs = 16;  // raster group: token-tile pairs that share weight rows in L2

MOE_DEVINL RowTile decode_row_tile(const Book &bk, const Fp4Params &p, int t, int crank) {
  RowTile ti;
  ti.e = tile_expert(bk, p, t);
  const int local = t - tc::uniform(bk.cum[ti.e]);
  ti.row0 = tc::uniform(bk.off[ti.e]);
  ti.row_end = max(tc::uniform(bk.off[ti.e + 1]), ti.row0);
  const int mp = (ti.row_end - ti.row0 + 255) / 256;
  const int group = kGroupPairs * p.w_tiles;
  const int g = local / group;
  const int within = local - g * group;
  const int gm = min(kGroupPairs, mp - g * kGroupPairs);
  ti.n_idx = within / gm;
  ti.m_idx = 2 * (g * kGroupPairs + (within - ti.n_idx * gm)) + crank;
  ti.row0 += ti.m_idx * 128;
  return ti;
}

// 32 values of a row -> 16 bytes of codes and the chunk's scale codes (NVFP4:
// two bytes, MXFP4: one).
template <int FMT>
MOE_DEVINL uint4 quantize_chunk(float *v, float g, float inv6, uint32_t &scale) {
  constexpr int kB = fp4_block(FMT);
  uint32_t codes[4];
  scale = 0;
#pragma unroll
  for (int b = 0; b < 32 / kB; ++b) {
    float a = 0.0f;
    bool finite = true;
#pragma unroll
    for (int j = 0; j < kB; ++j) {
      const float m = fabsf(v[b * kB + j]);
      finite &= m <= 3.402823466e38f;
      a = fmaxf(a, m);
    }
    float inv;
    scale |= fp4_block_scale<FMT>(finite ? a : __uint_as_float(0x7F800000u), g, 6.0f * g, inv6,
                                  inv)
             << (8 * b);
#pragma unroll
    for (int j = 0; j < kB; ++j) v[b * kB + j] *= inv;
#pragma unroll
    for (int j = 0; j < kB / 8; ++j)
      codes[b * (kB / 8) + j] = inv == 0.0f ? 0u : cvt_e2m1x8(v + b * kB + 8 * j);
  }
  return make_uint4(codes[0], codes[1], codes[2], codes[3]);
}

template <int FMT>
MOE_DEVINL void epilogue_rows(const Book &bk, const Fp4Params &p, const RowTile &ti, float sc,
                              float g2, float inv6, uint32_t taddr, int q, int sub, int subs,
                              int lane) {
  const int64_t row = (int64_t)ti.row0 + q * 32 + lane;
  const bool valid = row < ti.row_end;
  if (ti.row0 + q * 32 >= ti.row_end) return;  // no row of this warp is the expert's
  const int F = p.F;
  const int f0 = ti.n_idx * (BR / 2);
  // the row's place in Act's scale atoms
  const int arow = (int)bk.poff[ti.e] + ti.m_idx;
  uint8_t *srow = p.sf2 + (int64_t)arow * p.ac2 * 512 + lane * 16 + q * 4;
  const bool put = valid && arow < p.atom_rows2;
#pragma unroll 1
  for (int c = sub; c < BR / 64; c += subs) {
    const int nc = f0 + c * 32;
    if (nc >= F) break;
    float g[32], u[32];
    {
      uint32_t rg[32], ru[32];
      tc::tmem_ld32_issue(taddr + c * 64, rg);
      tc::tmem_ld32_issue(taddr + c * 64 + 32, ru);
      tc::tmem_wait_ld(rg);
      tc::reg_after(ru);
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        g[j] = __uint_as_float(rg[j]) * sc;
        u[j] = __uint_as_float(ru[j]) * sc;
      }
    }
    if (p.C != nullptr && valid) {  // H in bf16 as well
      uint16_t *H = static_cast<uint16_t *>(p.C) + row * p.ldc + nc;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        st_v4(H + 8 * j, f32_to_bf16x8(g + 8 * j));
        st_v4(H + F + 8 * j, f32_to_bf16x8(u + 8 * j));
      }
    }
#pragma unroll
    for (int j = 0; j < 32; ++j) g[j] = g[j] * sigmoid_f(g[j]) * u[j];
    uint32_t scale;
    const uint4 codes = quantize_chunk<FMT>(g, g2, inv6, scale);
    if (put) {
      st_v4(p.Q2 + row * p.ldq2 + (nc >> 1), codes);
      const int b = nc / fp4_block(FMT);
      uint8_t *s = srow + (b >> 2) * 512 + (b & 3);
      if (FMT == MOE_FP4_NV) *reinterpret_cast<uint16_t *>(s) = (uint16_t)scale;
      else *s = (uint8_t)scale;
      if (nc + 32 >= F)  // the last atom's spare blocks
        for (int x = F / fp4_block(FMT); x < 4 * p.ac2; ++x)
          srow[(x >> 2) * 512 + (x & 3)] = 0;
    }
  }
}

// ------------------------------------------------------------------ kernel
template <int FMT, int EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Lay<FMT, EPI>::threads, 1)
gmm_fp4_kernel(const __grid_constant__ Maps m, const Fp4Params p) {
  using L = Lay<FMT, EPI>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Book &bk = *reinterpret_cast<Book *>(smem + L::book_offset);
  volatile int *abort_flag = &bk.abort_flag;
  const int warp = tc::uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int crank = (int)tc::cluster_ctarank();
  const int cid = (int)tc::cluster_id_x();
  const int ncl = (int)tc::nclusters_x();
  constexpr uint16_t kPair = 0x3;
  constexpr int kStages = L::stages;
  const bool leader = crank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(&bk.full[s], 2);  // the stage's copies, and a free scale slot
      tc::mbar_init(&bk.empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      tc::mbar_init(&bk.tfull[a], 1);
      tc::mbar_init(&bk.tempty[a], 2 * L::epi_warps);
    }
    tc::mbar_init(&bk.shared_read, 2 * L::epi_warps);
    tc::mbar_init(&bk.drain, 1);
    bk.abort_flag = 0;
    tc::fence_mbar_init();
  }
  if (warp == 2 && lane == 0) {
    // (those that the launch has encoded: kRows loads its tokens by the last box alone)
    tc::tma_prefetch(&m.w);
    tc::tma_prefetch(&m.t[EPI == kRows ? 3 : 0]);
    tc::tma_prefetch(&m.sw);
    tc::tma_prefetch(&m.st[0]);
    if (EPI == MOE_EPI_NONE) tc::tma_prefetch(&m.c);
  }
  if (warp == 1) {
    tc::tmem_alloc_2sm(&bk.tmem_base, kTmemCols);
    tc::tmem_relinquish_2sm();
  }
  // The work above overlaps the end of the kernel before; with `early` so do the
  // tile counts and the first weights' copies (each role then waits for itself).
  const bool early = EPI != kRows && p.early;
  if (!early) grid_dependency_begin();
  for (int e = (int)threadIdx.x - 32; e < p.E; e += L::threads - 32)
    if (e >= 0) bk.gb[e] = p.gb != nullptr ? ld_f32(p.gb + e) : 1.0f;
  if (warp == 0) {
    // per-expert tile counts and padded sizes, and their exclusive scans
    int carry = 0, pcarry = 0;
    for (int c0 = 0; c0 < p.E; c0 += 32) {
      const int e = c0 + lane;
      int tiles = 0, padded = 0;
      if (e < p.E) {
        const int lo = group_offset(p, e), hi = group_offset(p, e + 1);
        const int size = max(hi - lo, 0);
        bk.off[e] = lo;
        if (e == p.E - 1) bk.off[p.E] = hi;
        padded = (size + 127) / 128;
        tiles = (EPI == kRows ? (size + 255) / 256 : (size + BT - 1) / BT) * p.w_tiles;
        if (hi < lo) moe_set_status(p.dev_status, MOE_ERR_DEVICE);
      }
      int incl = tiles, pincl = padded;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        const int py = __shfl_up_sync(0xffffffffu, pincl, o);
        if (lane >= o) {
          incl += y;
          pincl += py;
        }
      }
      if (e < p.E) {
        bk.cum[e] = carry + incl - tiles;
        bk.poff[e] = (uint16_t)(pcarry + pincl - padded);
      }
      carry += __shfl_sync(0xffffffffu, incl, 31);
      pcarry += __shfl_sync(0xffffffffu, pincl, 31);
    }
    if (lane == 0) {
      bk.cum[p.E] = carry;
      bk.total_tiles = carry;
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::cluster_sync();
  tc::tc_fence_after();
  const uint32_t tmem = (uint32_t)tc::uniform((int)bk.tmem_base);
  const int total = tc::uniform(bk.total_tiles);

  if (early && warp != 0) grid_dependency_begin();
  if (warp == 0) {
    if (!p.stall_loads) {
      uint32_t issued = 0;
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = cid; t < total && ok && EPI == kRows; t += ncl) {
        const RowTile ti = decode_row_tile(bk, p, t, crank);
        const int tok_sf = (int)bk.poff[ti.e] + ti.m_idx;
        const int wgt_sf = ti.e * p.w_atoms + ti.n_idx * BR / 128;
        // a CTA past the expert's rows loads none: its products are not stored
        const bool own = ti.row0 < ti.row_end;
        const bool both = ti.row0 + (1 - 2 * crank) * 128 < ti.row_end;  // the other CTA's
        const int tx = (own + both) * (W_BYTES + L::sfw_bytes) + 2 * (L::t_bytes + L::sft_bytes);
        for (int kb = 0; kb < p.kblocks; ++kb) {
          if (!tc::mbar_wait_warp(&bk.empty[s], ph ^ 1, abort_flag, p.wait_limit_ns)) {
            ok = false;
            break;
          }
          if (tc::elect_one()) {
            uint8_t *st = smem + s * L::stage_bytes;
            const uint32_t fb = tc::mapa_shared(tc::smem_u32(&bk.full[s]), 0);
            if (leader) {
              if (kb == 0) bk.shape[s] = mma_shape(BR, ti.n_idx & 1 ? 2 : 0, true);
              tc::mbar_expect_tx(&bk.full[s], tx);
            }
            const int k = kb * kRowBytes;
            if (own) {
              tc::tma_load_2d_2sm(st, &m.t[3], fb, k, ti.row0);
              tc::tma_load_3d_2sm(st + W_BYTES + L::t_bytes, &m.st[0], fb, 0, kb * L::atoms, tok_sf);
            }
#pragma unroll
            for (int i = 0; i < 3; ++i) {  // three of the tile's six blocks of 32 rows
              const int b = 3 * crank + i;
              tc::tma_load_5d_2sm(st + W_BYTES + i * 4096, &m.w, fb, k, 0, b & 1,
                                  3 * ti.n_idx + (b >> 1), ti.e);
            }
            tc::tma_load_3d_2sm(st + W_BYTES + L::t_bytes + L::sfw_bytes, &m.sw, fb, 0,
                                kb * L::atoms, wgt_sf);
          }
          __syncwarp();
          ++issued;
          if (++s == kStages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      int done = 0;  // K blocks of the first tile that are issued
      TileInfo next;
      if (EPI != kRows && cid < total) next = decode_tile(bk, p, cid);
      for (int t = cid; t < total && ok && EPI != kRows; t += ncl) {
        const TileInfo ti = next;
        bool looked = t + ncl >= total;  // the next tile is looked up between copies
        // this CTA's half of the tokens, rounded up to 32 rows
        const int trow = ti.row0 + crank * (ti.n / 2);
        const int tbox = (ti.n / 2 + 31) / 32;
        const int sbox = second_atom(ti) ? 2 : 1;  // their scale atoms
        const int trow_sf = (int)bk.poff[ti.e] + (ti.t0 >> 7);
        const int wrow_sf = ti.e * p.w_atoms + 2 * ti.w_idx + crank;
        const int tx = 2 * (W_BYTES + tbox * 4096 + (1 + sbox) * L::sfw_bytes);  // the pair's
        auto load_weights = [&](int st, int kb) {
          uint8_t *sw = smem + st * L::stage_bytes;
          const uint32_t fb = tc::mapa_shared(tc::smem_u32(&bk.full[st]), 0);
          if (leader) {
            if (kb == 0) bk.shape[st] = mma_shape(ti.n, scale_shift(ti), second_atom(ti));
            tc::mbar_expect_tx(&bk.full[st], tx);
          }
          const int k = kb * kRowBytes;
          if (EPI == MOE_EPI_SWIGLU_FWD)  // 32 gate rows, 32 up rows, twice
            tc::tma_load_5d_2sm(sw, &m.w, fb, k, 0, 0, 4 * ti.w_idx + 2 * crank, ti.e);
          else
            tc::tma_load_3d_2sm(sw, &m.w, fb, k, ti.w_idx * BW + crank * (BW / 2), ti.e);
          tc::tma_load_3d_2sm(sw + W_BYTES + L::t_bytes, &m.sw, fb, 0, kb * L::atoms, wrow_sf);
        };
        auto load_tokens = [&](int st, int kb) {
          uint8_t *sw = smem + st * L::stage_bytes;
          const uint32_t fb = tc::mapa_shared(tc::smem_u32(&bk.full[st]), 0);
          tc::tma_load_2d_2sm(sw + W_BYTES, &m.t[tbox - 1], fb, kb * kRowBytes, trow);
          tc::tma_load_3d_2sm(sw + W_BYTES + L::t_bytes + L::sfw_bytes, &m.st[sbox - 1], fb, 0,
                              kb * L::atoms, trow_sf);
        };
        if (early && t == cid) {
          // the stages are free: their weights first, the tokens once they are there
          done = min(p.kblocks, kStages);
          if (tc::elect_one())
            for (int kb = 0; kb < done; ++kb) load_weights(kb, kb);
          __syncwarp();
          grid_dependency_begin();
          if (tc::elect_one())
            for (int kb = 0; kb < done; ++kb) load_tokens(kb, kb);
          __syncwarp();
          issued = done;
          s = done == kStages ? 0 : done;
          ph = done == kStages ? 1 : 0;
        }
        for (int kb = t == cid ? done : 0; kb < p.kblocks; ++kb) {
          if (!tc::mbar_wait_warp(&bk.empty[s], ph ^ 1, abort_flag, p.wait_limit_ns)) {
            ok = false;
            break;
          }
          if (tc::elect_one()) {
            load_weights(s, kb);
            load_tokens(s, kb);
          }
          __syncwarp();
          ++issued;
          if (++s == kStages) {
            s = 0;
            ph ^= 1;
          }
          if (!looked) next = decode_tile(bk, p, t + ncl);
          looked = true;
        }
        if (!looked) next = decode_tile(bk, p, t + ncl);
      }
      // every issued copy has landed before the CTA may exit (both CTAs' copies
      // complete on the leader's barriers)
      if (leader)
        for (uint32_t i = issued > (uint32_t)kStages ? issued - kStages : 0; i < issued; ++i)
          tc::mbar_wait_drain(&bk.full[i % kStages], (i / kStages) & 1, p.wait_limit_ns / 4);
    }
  } else if (warp == 1 && leader) {
    uint32_t acc_it = 0;
    int before = 0;     // N of the tile before
    int s = 0;          // ring slot of the next K block
    uint32_t ph = 0;
    int slot = 0;       // its scale slot
    bool ready = false; // its barrier has been seen complete
    bool ok = true;
    // descriptors of codes and scales at address 0, and the ring in their units
    const uint64_t dcodes = tc::sdesc(0, 16, 1024), dscales = tc::sdesc_plain(0, 0, 128);
    const uint32_t ring = (uint32_t)tc::uniform((int)(tc::smem_u32(smem) >> 4));
    constexpr uint32_t kTok = W_BYTES / 16, kSfw = kTok + L::t_bytes / 16,
                       kSft = kSfw + L::sfw_bytes / 16;
    // the first K blocks find their scale slots free
    if (tc::elect_one())
      for (int i = 0; i < L::sf_slots; ++i) tc::mbar_arrive(&bk.full[i]);
    __syncwarp();
    for (int t = cid; t < total && ok; t += ncl) {
      const uint32_t a = acc_it & 1;
      const uint32_t aph = (acc_it >> 1) & 1;
      uint32_t id0 = 0, id2 = 0, shift = 0;
      bool second = false;
      if (!tc::mbar_wait_warp(&bk.tempty[a], aph ^ 1, abort_flag, p.wait_limit_ns)) break;
      tc::tc_fence_after();
      const uint32_t d_tmem = tmem + a * L::acc_step;
      for (int kb = 0; kb < p.kblocks; ++kb) {
        if (!__all_sync(0xffffffffu, ready) &&
            !tc::mbar_wait_warp(&bk.full[s], ph, abort_flag, p.wait_limit_ns)) {
          ok = false;
          break;
        }
        const int s1 = s + 1 == kStages ? 0 : s + 1;
        const uint32_t ph1 = s1 == 0 ? ph ^ 1 : ph;
        tc::tc_fence_after();
        if (kb == 0) {
          const uint32_t shape = (uint32_t)tc::uniform((int)bk.shape[s]);
          const int n = shape & 0xffff;
          id0 = tc::idesc_fp4(BW, n, FMT == MOE_FP4_NV, 0);
          id2 = tc::idesc_fp4(BW, n, FMT == MOE_FP4_NV, 2);
          shift = shape >> 16 & 0xff;
          second = shape >> 24;
          // where this tile and the one before share columns, those have to be read
          if (EPI != kRows && acc_it > 0 && (a ? before : n) > L::acc_step) {
            ok = tc::mbar_wait_warp(&bk.shared_read, (acc_it - 1) & 1, abort_flag,
                                    p.wait_limit_ns);
            if (!ok) break;
            tc::tc_fence_after();
          }
          before = n;
        }
        if (tc::elect_one()) {
          const uint32_t w = ring + s * (L::stage_bytes / 16);
          const uint32_t at = tmem + L::sf_base + slot * L::sf_cols;
#pragma unroll
          for (int j = 0; j < L::atoms; ++j) {
            tc::tmem_cp_32x128b_x4_2sm(at + 12 * j, tc::desc_at(dscales, w + kSfw + 32 * j));
            tc::tmem_cp_32x128b_x4_2sm(at + 12 * j + 4, tc::desc_at(dscales, w + kSft + 32 * j));
            if (second)
              tc::tmem_cp_32x128b_x4_2sm(at + 12 * j + 8,
                                         tc::desc_at(dscales, w + kSft + 32 * (L::atoms + j)));
          }
#pragma unroll
          for (int kk = 0; kk < kKSteps; ++kk) {
            const int j = kk * L::atoms / kKSteps;  // atom of this step
            // MXFP4: two steps share an atom, two bytes of its scale words each
            tc::umma_fp4_2sm<FMT == MOE_FP4_NV>(
                d_tmem, tc::desc_at(dcodes, w + 2 * kk), tc::desc_at(dcodes, w + kTok + 2 * kk),
                L::atoms == kKSteps || !(kk & 1) ? id0 : id2, at + 12 * j, at + 12 * j + 4 + shift,
                (kb | kk) != 0);
          }
          tc::umma_commit_2sm_mc(&bk.empty[s], kPair);
          // this block's scale slot is free for the block sf_slots further
          const int sn = s + L::sf_slots;
          tc::umma_commit_2sm_mc(&bk.full[sn < kStages ? sn : sn - kStages], 0x1);
        }
        __syncwarp();
        ready = tc::mbar_test(&bk.full[s1], ph1);
        if (++slot == L::sf_slots) slot = 0;
        s = s1;
        ph = ph1;
      }
      if (!ok) break;
      if (tc::elect_one()) tc::umma_commit_2sm_mc(&bk.tfull[a], kPair);
      __syncwarp();
      ++acc_it;
    }
    if (tc::elect_one()) tc::umma_commit_2sm_mc(&bk.drain, 0x1);
    __syncwarp();
    tc::mbar_wait_drain(&bk.drain, 0, p.wait_limit_ns);
  } else if (warp >= 2) {
    const int q = warp & 3;           // the tensor-memory lanes that it may read
    const int sub = (warp - 2) >> 2;  // its chunks of 32 tokens: every other one
    uint8_t *stg = smem + L::stg_offset;
    const float ga = p.ga != nullptr ? ld_f32(p.ga) : 1.0f;
    const float g2 = FMT == MOE_FP4_NV && p.g2 != nullptr ? ld_f32(p.g2) : 1.0f;
    const float inv6 = __frcp_rn(6.0f * g2);
    uint32_t acc_it = 0;
    for (int t = cid; t < total; t += ncl) {
      TileInfo ti;
      RowTile rt;
      if (EPI == kRows) rt = decode_row_tile(bk, p, t, crank);
      else ti = decode_tile(bk, p, t);
      const float sc = ga * bk.gb[EPI == kRows ? rt.e : ti.e];
      const uint32_t a = acc_it & 1;
      const uint32_t aph = (acc_it >> 1) & 1;
      // the two warps of a pair give up together (one barrier between them below)
      bool go = tc::mbar_wait_warp(&bk.tfull[a], aph, abort_flag, p.wait_limit_ns);
      if (EPI == MOE_EPI_SWIGLU_FWD) go = pair_agree(go, 2 * sub + (q >> 1));
      if (!go) break;
      tc::tc_fence_after();
      const uint32_t taddr = tmem + a * L::acc_step + (static_cast<uint32_t>(q * 32) << 16);
      if (EPI == kRows) {
        epilogue_rows<FMT>(bk, p, rt, sc, g2, inv6, taddr, q, sub, L::epi_warps / 4, lane);
      } else {
        Chunks ch;
        ch.taddr = taddr;
        ch.n = (ti.tokens + 31) / 32;
        ch.a = a;
        ch.first = sub ^ (int)a;
        ch.begin(tc::mapa_shared(tc::smem_u32(&bk.shared_read), 0), lane);
        if (EPI == MOE_EPI_SWIGLU_FWD)
          epilogue_swiglu<FMT>(bk, p, ti, sc, g2, inv6, ch, crank, q, sub, lane,
                               stg + (2 * sub + (q >> 1)) * 2 * kStgBytes);
        else
          epilogue_plain(p, ti, sc, ch, crank, q, sub, lane, stg + (4 * sub + q) * kStgBytes,
                         &m.c);
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive_cluster_relaxed(tc::mapa_shared(tc::smem_u32(&bk.tempty[a]), 0));
      ++acc_it;
    }
    if (lane == 0) tc::bulk_wait0();
    __syncwarp();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::cluster_sync();
  tc::tc_fence_after();
  if (warp == 1) tc::tmem_dealloc_2sm(tmem, kTmemCols);
  if (threadIdx.x == 0 && bk.abort_flag) moe_set_status(p.dev_status, MOE_ERR_TIMEOUT);
}

// --------------------------------------------------------------- host side
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// Map of `rank` dimensions, dims[0] contiguous, strides in bytes.
bool make_map(CUtensorMap *m, const void *base, CUtensorMapDataType type, int rank,
              const uint64_t *dims, const uint64_t *strides, const uint32_t *box,
              CUtensorMapSwizzle swizzle) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t d[5], st[4];
  cuuint32_t b[5], es[5] = {1, 1, 1, 1, 1};
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
  }
  for (int i = 0; i < rank - 1; ++i) st[i] = strides[i];
  return fn(m, type, rank, const_cast<void *>(base), d, st, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of packed codes: boxes of 128 bytes (256 codes) x `box_rows` rows.
bool make_code_map(CUtensorMap *m, const uint8_t *base, int rank, int64_t bytes, int64_t rows,
                   int64_t ld, int64_t groups, int64_t group_stride, int box_rows) {
  const uint64_t dims[3] = {(uint64_t)bytes, (uint64_t)rows, (uint64_t)groups};
  const uint64_t st[2] = {(uint64_t)ld, (uint64_t)group_stride};
  const uint32_t box[3] = {kRowBytes, (uint32_t)box_rows, 1};
  return make_map(m, base, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, dims, st, box,
                  CU_TENSOR_MAP_SWIZZLE_128B);
}

// Scale atoms as [atom rows, atom columns, 128 words]; past the last atom
// column the fill is zero, the scale of the codes that are not there.
bool make_scale_map(CUtensorMap *m, const uint8_t *base, int64_t ac, int64_t ar, int atoms,
                    int box_rows) {
  const uint64_t dims[3] = {128, (uint64_t)ac, (uint64_t)ar};
  const uint64_t st[2] = {512, (uint64_t)ac * 512};
  const uint32_t box[3] = {128, (uint32_t)atoms, (uint32_t)box_rows};
  return make_map(m, base, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, dims, st, box,
                  CU_TENSOR_MAP_SWIZZLE_NONE);
}

bool make_out_map(CUtensorMap *m, const void *base, bool f32, int64_t cols, int64_t rows,
                  int64_t ld) {
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows};
  const uint64_t st[1] = {(uint64_t)ld * (f32 ? 4 : 2)};
  const uint32_t box[2] = {32, 32};
  return make_map(m, base, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                  2, dims, st, box, f32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

template <int FMT, int EPI>
moe_status_t launch(const Maps &m, const Fp4Params &p, int64_t tiles_upper,
                    cudaStream_t s) {
  constexpr int kSmem = smem_bytes<FMT, EPI>();
  constexpr int kThreads = Lay<FMT, EPI>::threads;
  struct Setup {
    cudaError_t err;
    int max_clusters;  // clusters of two CTAs that the device holds at a time
  };
  static PerDevice<Setup> known;
  const Setup setup = known.get(current_device(), [] {
    Setup u{cudaFuncSetAttribute(gmm_fp4_kernel<FMT, EPI>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem),
            0};
    if (u.err != cudaSuccess) return u;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (unsigned)num_sms());
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    if (cudaOccupancyMaxActiveClusters(&u.max_clusters, gmm_fp4_kernel<FMT, EPI>, &cfg) !=
            cudaSuccess ||
        u.max_clusters <= 0) {
      cudaGetLastError();
      u.max_clusters = num_sms() / 2;
    }
    return u;
  });
  if (setup.err != cudaSuccess) {
    set_error("moe_gmm_fp4: cannot reserve %d bytes of shared memory: %s", kSmem,
              cudaGetErrorString(setup.err));
    return MOE_ERR_CUDA;
  }
  const int grid = 2 * (int)std::max<int64_t>(1, std::min<int64_t>(setup.max_clusters, tiles_upper));
  const cudaError_t e = launch_dependent(gmm_fp4_kernel<FMT, EPI>, grid, kThreads, kSmem, s, m, p);
  if (e != cudaSuccess) {
    set_error("moe_gmm_fp4 launch: %s", cudaGetErrorString(e));
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // namespace

// SwiGLU with tokens as M (kRows): where K is so short that the turned epilogue (some
// 9000 cycles a tile of 256 tokens) is what a tile waits for, from as many rows an
// expert on as fill its tile of 256 tokens.  us with tokens / weights as M, ragged
// groups:
//   16 experts of 1024 x 4096, MXFP4, 128 rows each 19.3 / 17.9, 256: 24.4 / 27.7,
//     1024: 61.7 / 70.3, 4096: 207 / 244;  NVFP4, 256: 29.6 / 36.0, 4096: 252 / 284
//   of 2560 x 8192, MXFP4, 192: 42.2 / 41.1, 256: 51.0 / 55.4, 4096: 439 / 501
//   of 3584 x 8192, MXFP4, 256: 65.2 / 62.0, 1024: 169 / 159, 4096: 561 / 546
//   8 of 4096 x 28672, MXFP4, 512: 183 / 165, 4096: 1097 / 1071
constexpr int kRowsFrom = 256, kRowsMaxK = 2816;

moe_status_t launch_gmm_fp4(const GmmFp4Args &a, cudaStream_t s) {
  const bool swiglu = a.epilogue == MOE_EPI_SWIGLU_FWD;
  const bool nv = a.fmt == MOE_FP4_NV;
  const int acols = fp4_atom_cols(a.fmt);
  const int atoms = 256 / acols;
  Fp4Params p{};
  p.E = a.E;
  p.rows_cap = (int)a.rows_cap;
  p.N = a.N;
  p.F = swiglu ? a.N / 2 : a.N;
  const bool rows =
      swiglu && a.rows_cap >= (int64_t)kRowsFrom * a.E && a.K <= kRowsMaxK;
  p.w_tiles = rows ? (a.N + BR - 1) / BR : (a.N + BW - 1) / BW;
  p.w_atoms = (a.N + 127) / 128;
  p.kblocks = (a.K + 255) / 256;
  p.offsets = a.offsets;
  p.C = a.C;
  p.ldc = a.ldc;
  p.c_f32 = a.c_dtype == MOE_DTYPE_F32;
  p.Q2 = a.Q2;
  p.ldq2 = a.ldq2;
  p.sf2 = a.sf2;
  p.ac2 = (p.F + acols - 1) / acols;
  p.atom_rows2 = (int)(f8_padded_rows(a.rows_cap, a.E) / 128);
  p.g2 = a.g2;
  p.ga = a.ga;
  p.gb = a.gb;
  p.dev_status = a.dev_status;
  p.wait_limit_ns = wait_limit_ns();
  p.stall_loads = test_stall_loads();
  p.early = a.early;
  Maps m{};
  const int64_t ac = (a.K + acols - 1) / acols;
  const int64_t stride_b = a.E > 1 ? a.stride_b : (int64_t)a.N * a.ldb;
  bool ok = make_scale_map(&m.sw, a.sfb, ac, (int64_t)a.E * p.w_atoms, atoms, 1) &&
            make_scale_map(&m.st[0], a.sfa, ac, p.atom_rows2, atoms, 1) &&
            (rows || a.rows_cap <= 128 ||
             make_scale_map(&m.st[1], a.sfa, ac, p.atom_rows2, atoms, 2));
  // the boxes that a tile of at most rows_cap tokens can need (an encoding takes the
  // host about as long as a launch)
  const int boxes = (int)(std::min<int64_t>((a.rows_cap + 15) / 16 * 16, BT) + 63) / 64;
  for (int i = rows ? 3 : 0; i < (rows ? 4 : boxes); ++i)
    ok = ok && make_code_map(&m.t[i], a.A, 2, a.K / 2, a.rows_cap, a.lda, 1, 0, 32 * (i + 1));
  if (rows)  // weights in boxes of 32 rows, their atoms two rows
    ok = ok && make_scale_map(&m.sw, a.sfb, ac, (int64_t)a.E * p.w_atoms, atoms, 2);
  if (swiglu) {
    // [E][F / 32][gate, up][32] rows: a box takes two blocks of 32 gates and 32 ups
    const uint64_t dims[5] = {(uint64_t)a.K / 2, 32, 2, (uint64_t)p.F / 32, (uint64_t)a.E};
    const uint64_t st[4] = {(uint64_t)a.ldb, (uint64_t)p.F * a.ldb, 32 * (uint64_t)a.ldb,
                            (uint64_t)stride_b};
    const uint32_t nb = rows ? 1 : 2;
    const uint32_t box[5] = {kRowBytes, 32, nb, nb, 1};
    ok = ok && make_map(&m.w, a.B, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, dims, st, box,
                        CU_TENSOR_MAP_SWIZZLE_128B);
  } else {
    ok = ok && make_code_map(&m.w, a.B, 3, a.K / 2, a.N, a.ldb, a.E, stride_b, BW / 2) &&
         make_out_map(&m.c, a.C, p.c_f32, a.N, a.rows_cap, a.ldc);
  }
  if (!ok) {
    set_error("moe_gmm_fp4: cannot encode a TMA descriptor");
    return MOE_ERR_CUDA;
  }
  // token tiles: at most one partly filled an expert that has rows
  const int64_t live = std::min<int64_t>(a.E, a.rows_cap);
  const int64_t tiles_upper = ((a.rows_cap + BT - 1) / BT + live) * p.w_tiles;
  if (rows)
    return nv ? launch<MOE_FP4_NV, kRows>(m, p, tiles_upper, s)
              : launch<MOE_FP4_MX, kRows>(m, p, tiles_upper, s);
  if (swiglu)
    return nv ? launch<MOE_FP4_NV, MOE_EPI_SWIGLU_FWD>(m, p, tiles_upper, s)
              : launch<MOE_FP4_MX, MOE_EPI_SWIGLU_FWD>(m, p, tiles_upper, s);
  return nv ? launch<MOE_FP4_NV, MOE_EPI_NONE>(m, p, tiles_upper, s)
            : launch<MOE_FP4_MX, MOE_EPI_NONE>(m, p, tiles_upper, s);
}

}  // namespace moe

// Grouped GEMM of the expert FFN on 4-bit block-scaled codes (MXFP4, NVFP4):
// for every expert e, rows [off_e, off_e+1) of A times B_e^T, both K-major E2M1
// codes with their scales applied by the tensor cores
// (tcgen05.mma kind::mxf4nvf4.block_scale), fp32 accumulators in tensor memory.
//
// Epilogues: plain (times the tensors' fp32 scales, to bf16 or fp32), and the
// SwiGLU forward, which quantises Act = silu(g) u to 4 bits straight from the
// fp32 accumulators: a thread holds a row's 32 columns, so that a block's
// maximum needs no other thread, and the down-projection's operand leaves
// the kernel as 16 bytes of codes and one or two scale bytes instead of 64
// bytes of bf16 that another pass would read again.
//
// Persistent; clusters of two CTAs issue 2-SM MMAs (M = 256, N = 192, K = 64
// codes = 32 bytes).  A stage is a K block of 256 codes (one 128-byte swizzle
// row a tile row): A 16 KB and half of B 12 KB a CTA, and the K block's scale
// atoms (512 bytes of 128 rows x 4 blocks): 4 (NVFP4) or 2 (MXFP4) for A and
// twice as many for B's 192 columns.
//   warp 0     TMA producer
//   warp 1     tensor memory, and in the leader CTA the MMA issue: the atoms
//              to tensor memory (tcgen05.cp), then four MMAs
//   warps 2-5  epilogue, one per quarter of the tensor-memory lanes
// Tensor memory: two accumulators of 192 columns, and scale slots in the 128
// columns that they leave: 48 columns a K block (NVFP4, 2 slots) or 24 (MXFP4,
// 5).  A slot is rewritten after the MMAs that read it are done: their commit
// arrives on the full barrier of the K block that takes the slot next, beside the
// stage's copies, so that the issuer has one barrier to wait for.  That wait and
// the issue set the pace (a K block's MMAs take about 300 cycles): the next
// barrier is tested before a block's MMAs are issued, and the issuing warp stays
// uniform, elect_one() choosing the lane.  8 experts, 32768 rows, 4096 x 28672:
// lane == 0 in place of elect_one() 2.41 ms, a second wait for the slot 1.36 ms.
// Every wait is bounded; on time-out the CTA winds down and reports
// MOE_ERR_TIMEOUT through dev_status.
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "internal.h"
#include "lowbit.cuh"
#include "tc_sm103.cuh"

namespace moe {
namespace {

constexpr int BM = 128;        // rows of a CTA's A tile
constexpr int BN = 192;        // columns of the pair's tile
constexpr int kRowBytes = 128; // one K block of a tile row: 256 codes
constexpr int kKSteps = 4;     // MMAs a K block
constexpr int kStages = 6;
constexpr int A_BYTES = BM * kRowBytes;
constexpr int B_BYTES = BN / 2 * kRowBytes;
constexpr int kEpiWarps = 4;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kStgBytes = 4096;  // staging of an epilogue warp
constexpr int kMaxE = 256;
constexpr int kGroupPairs = 16;  // raster group: row-tile pairs that share B columns in L2
constexpr int kTmemCols = 512;

template <int FMT>
struct Lay {
  static constexpr int atoms = 256 / fp4_atom_cols(FMT);  // atom columns a K block
  static constexpr int sfa_bytes = atoms * 512;
  static constexpr int sfb_bytes = 2 * sfa_bytes;
  static constexpr int tx_bytes = A_BYTES + B_BYTES + sfa_bytes + sfb_bytes;
  static constexpr int stage_bytes = (tx_bytes + 1023) / 1024 * 1024;
  static constexpr int sf_cols = atoms * 12;               // tensor-memory columns a slot
  static constexpr int sf_slots = (kTmemCols - 2 * BN) / sf_cols;
  static_assert(sf_slots <= kStages, "a commit names a K block's next user by its stage");
  static constexpr int stg_offset = kStages * stage_bytes;
  static constexpr int book_offset = stg_offset + kEpiWarps * kStgBytes;
};

struct Book {
  uint64_t full[kStages];
  uint64_t empty[kStages];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  int total_tiles;
  int cum[kMaxE + 1];        // per-expert tile prefix
  uint16_t poff[kMaxE + 1];  // padded group starts in units of 128 rows
};

template <int FMT>
constexpr int smem_bytes() {
  return 1024 + Lay<FMT>::book_offset + (int)((sizeof(Book) + 127) / 128 * 128);
}
static_assert(smem_bytes<MOE_FP4_NV>() <= 232448, "shared memory of one CTA");

struct Fp4Params {
  int E, rows_cap, N, F, n_tiles, kblocks;
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
};

struct TileInfo {
  int e, m_idx, n_idx, row0, row_end;
};

MOE_DEVINL int group_offset(const Fp4Params &p, int e) {
  return min(max(ld_i32(p.offsets + e), 0), p.rows_cap);
}

// Tile t: the two CTAs of a pair take row tiles 2 pm and 2 pm + 1 of an expert
// and one column tile (the second may lie past the expert's rows).
MOE_DEVINL TileInfo decode_tile(const Book &bk, const Fp4Params &p, int t, int crank) {
  int lo = 0, hi = p.E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (bk.cum[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  TileInfo ti;
  ti.e = lo;
  const int local = t - bk.cum[lo];
  ti.row0 = group_offset(p, lo);
  ti.row_end = max(group_offset(p, lo + 1), ti.row0);
  const int mp = ((ti.row_end - ti.row0 + BM - 1) / BM + 1) / 2;
  const int group = kGroupPairs * p.n_tiles;
  const int g = local / group;
  const int within = local - g * group;
  const int gm = min(kGroupPairs, mp - g * kGroupPairs);
  ti.n_idx = within / gm;
  ti.m_idx = 2 * (g * kGroupPairs + (within - ti.n_idx * gm)) + crank;
  ti.row0 += ti.m_idx * BM;
  return ti;
}

// Rows of A that a CTA loads for a tile of `valid` rows, in boxes of 32 (the
// others keep what the stage held: their products are not stored).
MOE_DEVINL int rows_loaded(int valid) {
  return valid > BM - 32 ? BM : valid > 0 ? (valid + 31) / 32 * 32 : 0;
}

// ---------------------------------------------------------------- epilogue
// One thread's 32-value row segment staged as the TMA store reads it (64-byte
// swizzle for bf16, 128-byte for fp32).
MOE_DEVINL void stage_bf16(uint8_t *buf, int r, const float *v) {
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<uint4 *>(buf + r * 64 + ((c ^ ((r >> 1) & 3)) << 4)) =
        f32_to_bf16x8(v + 8 * c);
}

MOE_DEVINL void stage_f32(uint8_t *buf, int r, const float *v) {
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<uint4 *>(buf + r * 128 + ((c ^ (r & 7)) << 4)) =
        make_uint4(__float_as_uint(v[4 * c]), __float_as_uint(v[4 * c + 1]),
                   __float_as_uint(v[4 * c + 2]), __float_as_uint(v[4 * c + 3]));
}

// 32 values of a row -> 16 bytes of codes and the chunk's scale codes (NVFP4:
// two bytes, MXFP4: one).  The values are continuous, so that no quotient sits
// on a tie and a product with the reciprocal decides as the quotient would.
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
    float t, inv;
    scale |= fp4_block_scale<FMT>(finite ? a : __uint_as_float(0x7F800000u), g, 6.0f * g, inv6, t,
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

template <int FMT, int EPI>
MOE_DEVINL void epilogue(const Book &bk, const Fp4Params &p, const TileInfo &ti, uint32_t taddr,
                         int q, int lane, uint8_t *stg, const CUtensorMap *m0,
                         const CUtensorMap *m1) {
  const float sc = (p.ga != nullptr ? ld_f32(p.ga) : 1.0f) *
                   (p.gb != nullptr ? ld_f32(p.gb + ti.e) : 1.0f);
  const int wrow0 = ti.row0 + q * 32;
  const int64_t row = (int64_t)wrow0 + lane;
  const bool valid = row < ti.row_end;
  const bool bulk = wrow0 + 32 <= ti.row_end;
  if (wrow0 >= ti.row_end) return;  // no row of this warp is the expert's
  if (EPI == MOE_EPI_SWIGLU_FWD) {
    const int F = p.F;
    const int n0 = ti.n_idx * (BN / 2);
    const float g2 = FMT == MOE_FP4_NV && p.g2 != nullptr ? ld_f32(p.g2) : 1.0f;
    const float inv6 = __frcp_rn(6.0f * g2);
    // the row's place in Act's scale atoms
    const int arow = (int)bk.poff[ti.e] + ti.m_idx;
    uint8_t *srow = p.sf2 + (int64_t)arow * p.ac2 * 512 + lane * 16 + q * 4;
    const bool put = valid && arow < p.atom_rows2;
#pragma unroll 1
    for (int c = 0; c < BN / 64; ++c) {
      const int nc = n0 + c * 32;
      if (nc >= F) break;
      float g[32], u[32];
      {
        uint32_t rg[32], ru[32];
        tc::tmem_ld32_issue(taddr + c * 32, rg);
        tc::tmem_ld32_issue(taddr + BN / 2 + c * 32, ru);
        tc::tmem_wait_ld(rg);
        tc::reg_after(ru);
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          g[j] = __uint_as_float(rg[j]) * sc;
          u[j] = __uint_as_float(ru[j]) * sc;
        }
      }
      if (p.C != nullptr) {  // H in bf16 as well
        if (bulk) {
          if (lane == 0) tc::bulk_wait_read0();
          __syncwarp();
          stage_bf16(stg, lane, g);
          stage_bf16(stg + 2048, lane, u);
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tc::tma_store_2d(m0, stg, nc, wrow0);
            tc::tma_store_2d(m1, stg + 2048, nc, wrow0);
            tc::bulk_commit();
          }
        } else if (valid) {
          uint16_t *H = static_cast<uint16_t *>(p.C) + row * p.ldc + nc;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            st_v4(H + 8 * j, f32_to_bf16x8(g + 8 * j));
            st_v4(H + F + 8 * j, f32_to_bf16x8(u + 8 * j));
          }
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
    return;
  }
  const int N = p.N;
  const int n0 = ti.n_idx * BN;
  int slot = 0;
#pragma unroll 1
  for (int c = 0; c < BN / 32; ++c) {
    const int nc = n0 + c * 32;
    if (nc >= N) break;
    float v[32];
    tc::tmem_ld32(taddr + c * 32, v);
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] *= sc;
    if (bulk) {
      // bf16 blocks take the staging's halves in turn, fp32 ones all of it
      uint8_t *buf = p.c_f32 ? stg : stg + slot * 2048;
      if (lane == 0) {
        if (p.c_f32) tc::bulk_wait_read0();
        else tc::bulk_wait_read<1>();
      }
      __syncwarp();
      if (p.c_f32) stage_f32(buf, lane, v);
      else stage_bf16(buf, lane, v);
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tc::tma_store_2d(m0, buf, nc, wrow0);
        tc::bulk_commit();
      }
      slot ^= 1;
    } else if (valid) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = nc + j * 8;
        if (n >= N) break;
        if (p.c_f32) {
          float *o = static_cast<float *>(p.C) + row * p.ldc + n;
          st_v4(o, make_uint4(__float_as_uint(v[8 * j]), __float_as_uint(v[8 * j + 1]),
                              __float_as_uint(v[8 * j + 2]), __float_as_uint(v[8 * j + 3])));
          st_v4(o + 4, make_uint4(__float_as_uint(v[8 * j + 4]), __float_as_uint(v[8 * j + 5]),
                                  __float_as_uint(v[8 * j + 6]), __float_as_uint(v[8 * j + 7])));
        } else {
          st_v4(static_cast<uint16_t *>(p.C) + row * p.ldc + n, f32_to_bf16x8(v + 8 * j));
        }
      }
    }
  }
}

// ------------------------------------------------------------------ kernel
template <int FMT, int EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
gmm_fp4_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
               const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
               const __grid_constant__ CUtensorMap tmC0, const __grid_constant__ CUtensorMap tmC1,
               const __grid_constant__ CUtensorMap tmA32, const Fp4Params p) {
  using L = Lay<FMT>;
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
  const bool leader = crank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(&bk.full[s], 2);  // the stage's copies, and a free scale slot
      tc::mbar_init(&bk.empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      tc::mbar_init(&bk.tfull[a], 1);
      tc::mbar_init(&bk.tempty[a], 2 * kEpiWarps);
    }
    tc::mbar_init(&bk.drain, 1);
    bk.abort_flag = 0;
    tc::fence_mbar_init();
  }
  if (warp == 2 && lane == 0) {
    tc::tma_prefetch(&tmA);
    tc::tma_prefetch(&tmB);
    tc::tma_prefetch(&tmSA);
    tc::tma_prefetch(&tmSB);
    tc::tma_prefetch(&tmC0);
    tc::tma_prefetch(&tmA32);
  }
  if (warp == 1) {
    tc::tmem_alloc_2sm(&bk.tmem_base, kTmemCols);
    tc::tmem_relinquish_2sm();
  }
  grid_dependency_begin();  // the work above overlaps the end of the kernel before
  if (warp == 0) {
    // per-expert tile counts and padded sizes, and their exclusive scans
    int carry = 0, pcarry = 0;
    for (int c0 = 0; c0 < p.E; c0 += 32) {
      const int e = c0 + lane;
      int tiles = 0, padded = 0;
      if (e < p.E) {
        const int lo = group_offset(p, e), hi = group_offset(p, e + 1);
        const int size = max(hi - lo, 0);
        padded = (size + BM - 1) / BM;
        tiles = (padded + 1) / 2 * p.n_tiles;
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

  if (warp == 0) {
    if (!p.stall_loads) {
      uint32_t issued = 0;
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = cid; t < total && ok; t += ncl) {
        const TileInfo ti = decode_tile(bk, p, t, crank);
        const int nrow = EPI == MOE_EPI_SWIGLU_FWD
                             ? (crank == 0 ? 0 : p.F) + ti.n_idx * (BN / 2)
                             : ti.n_idx * BN + crank * (BN / 2);
        const int arow = (int)bk.poff[ti.e] + ti.m_idx;
        const int brow = 2 * (ti.e * p.n_tiles + ti.n_idx);
        const int left = ti.row_end - ti.row0;  // rows from this CTA's first on
        const int rows = rows_loaded(left);
        // the leader's barrier counts the pair's copies
        const int tx = 2 * (L::tx_bytes - A_BYTES) + (rows + rows_loaded(left - BM)) * kRowBytes;
        for (int kb = 0; kb < p.kblocks; ++kb) {
          if (!tc::mbar_wait_warp(&bk.empty[s], ph ^ 1, abort_flag, p.wait_limit_ns)) {
            ok = false;
            break;
          }
          if (tc::elect_one()) {
            uint8_t *sa = smem + s * L::stage_bytes;
            const uint32_t fb = tc::mapa_shared(tc::smem_u32(&bk.full[s]), 0);
            if (leader) tc::mbar_expect_tx(&bk.full[s], tx);
            if (rows == BM) {
              tc::tma_load_3d_2sm(sa, &tmA, fb, kb * kRowBytes, ti.row0, 0);
            } else {
              for (int r = 0; r < rows; r += 32)
                tc::tma_load_3d_2sm(sa + r * kRowBytes, &tmA32, fb, kb * kRowBytes, ti.row0 + r,
                                    0);
            }
            tc::tma_load_3d_2sm(sa + A_BYTES, &tmB, fb, kb * kRowBytes, nrow, ti.e);
            tc::tma_load_3d_2sm(sa + A_BYTES + B_BYTES, &tmSA, fb, 0, kb * L::atoms, arow);
            tc::tma_load_3d_2sm(sa + A_BYTES + B_BYTES + L::sfa_bytes, &tmSB, fb, 0,
                                kb * L::atoms, brow);
          }
          __syncwarp();
          ++issued;
          if (++s == kStages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      // every issued copy has landed before the CTA may exit (both CTAs' copies
      // complete on the leader's barriers)
      if (leader)
        for (uint32_t i = issued > (uint32_t)kStages ? issued - kStages : 0; i < issued; ++i)
          tc::mbar_wait_drain(&bk.full[i % kStages], (i / kStages) & 1, p.wait_limit_ns / 4);
    }
  } else if (warp == 1 && leader) {
    uint32_t acc_it = 0;
    int s = 0;          // ring slot of the next K block
    uint32_t ph = 0;
    int slot = 0;       // its scale slot
    bool ready = false; // its barrier has been seen complete
    bool ok = true;
    // the first K blocks find their scale slots free
    if (tc::elect_one())
      for (int i = 0; i < L::sf_slots; ++i) tc::mbar_arrive(&bk.full[i]);
    __syncwarp();
    for (int t = cid; t < total && ok; t += ncl) {
      const uint32_t a = acc_it & 1;
      const uint32_t aph = (acc_it >> 1) & 1;
      if (!tc::mbar_wait_warp(&bk.tempty[a], aph ^ 1, abort_flag, p.wait_limit_ns)) break;
      tc::tc_fence_after();
      const uint32_t d_tmem = tmem + a * BN;
      for (int kb = 0; kb < p.kblocks; ++kb) {
        if (!__all_sync(0xffffffffu, ready) &&
            !tc::mbar_wait_warp(&bk.full[s], ph, abort_flag, p.wait_limit_ns)) {
          ok = false;
          break;
        }
        const int s1 = s + 1 == kStages ? 0 : s + 1;
        const uint32_t ph1 = s1 == 0 ? ph ^ 1 : ph;
        ready = tc::mbar_test(&bk.full[s1], ph1);
        tc::tc_fence_after();
        if (tc::elect_one()) {
          const uint32_t sa = tc::smem_u32(smem + s * L::stage_bytes);
          const uint64_t ad = tc::sdesc(sa, 16, 1024);
          const uint64_t bd = tc::sdesc(sa + A_BYTES, 16, 1024);
          const uint32_t sfa = sa + A_BYTES + B_BYTES;
          const uint32_t sfb = sfa + L::sfa_bytes;
          const uint32_t sft = tmem + 2 * BN + slot * L::sf_cols;
#pragma unroll
          for (int j = 0; j < L::atoms; ++j) {
            tc::tmem_cp_32x128b_x4_2sm(sft + 12 * j, tc::sdesc_plain(sfa + 512 * j, 0, 128));
            tc::tmem_cp_32x128b_x4_2sm(sft + 12 * j + 4, tc::sdesc_plain(sfb + 512 * j, 0, 128));
            tc::tmem_cp_32x128b_x4_2sm(sft + 12 * j + 8,
                                       tc::sdesc_plain(sfb + 512 * (L::atoms + j), 0, 128));
          }
#pragma unroll
          for (int kk = 0; kk < kKSteps; ++kk) {
            const int j = kk * L::atoms / kKSteps;            // atom of this step
            const int id = L::atoms == kKSteps ? 0 : (kk & 1) * 2;  // byte of its scale words
            tc::umma_fp4_2sm<FMT == MOE_FP4_NV>(d_tmem, ad + 2 * kk, bd + 2 * kk,
                                               tc::idesc_fp4(2 * BM, BN, FMT == MOE_FP4_NV, id),
                                               sft + 12 * j, sft + 12 * j + 4, (kb | kk) != 0);
          }
          tc::umma_commit_2sm_mc(&bk.empty[s], kPair);
          // this block's scale slot is free for the block sf_slots further
          const int sn = s + L::sf_slots;
          tc::umma_commit_2sm_mc(&bk.full[sn < kStages ? sn : sn - kStages], 0x1);
        }
        __syncwarp();
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
    const int q = warp & 3;
    uint8_t *stg = smem + L::stg_offset + (warp - 2) * kStgBytes;
    uint32_t acc_it = 0;
    for (int t = cid; t < total; t += ncl) {
      const TileInfo ti = decode_tile(bk, p, t, crank);
      const uint32_t a = acc_it & 1;
      const uint32_t aph = (acc_it >> 1) & 1;
      if (!tc::mbar_wait_warp(&bk.tfull[a], aph, abort_flag, p.wait_limit_ns)) break;
      tc::tc_fence_after();
      epilogue<FMT, EPI>(bk, p, ti, tmem + a * BN + (static_cast<uint32_t>(q * 32) << 16), q, lane,
                         stg, &tmC0, &tmC1);
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive_cluster(tc::mapa_shared(tc::smem_u32(&bk.tempty[a]), 0));
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
  cuuint64_t d[3], st[2];
  cuuint32_t b[3], es[3] = {1, 1, 1};
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
bool make_code_map(CUtensorMap *m, const uint8_t *base, int64_t bytes, int64_t rows, int64_t ld,
                   int64_t groups, int64_t group_stride, int box_rows) {
  const uint64_t dims[3] = {(uint64_t)bytes, (uint64_t)rows, (uint64_t)groups};
  const uint64_t st[2] = {(uint64_t)ld, (uint64_t)group_stride};
  const uint32_t box[3] = {kRowBytes, (uint32_t)box_rows, 1};
  return make_map(m, base, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, dims, st, box,
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
moe_status_t launch(const CUtensorMap *m, const Fp4Params &p, int64_t tiles_upper,
                    cudaStream_t s) {
  constexpr int kSmem = smem_bytes<FMT>();
  static std::once_flag once;
  static cudaError_t attr_err = cudaSuccess;
  static int max_clusters = 0;
  std::call_once(once, [] {
    attr_err = cudaFuncSetAttribute(gmm_fp4_kernel<FMT, EPI>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (attr_err != cudaSuccess) return;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (unsigned)num_sms());
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    if (cudaOccupancyMaxActiveClusters(&max_clusters, gmm_fp4_kernel<FMT, EPI>, &cfg) !=
            cudaSuccess ||
        max_clusters <= 0) {
      cudaGetLastError();
      max_clusters = num_sms() / 2;
    }
  });
  if (attr_err != cudaSuccess) {
    set_error("moe_gmm_fp4: cannot reserve %d bytes of shared memory: %s", kSmem,
              cudaGetErrorString(attr_err));
    return MOE_ERR_CUDA;
  }
  const int grid = 2 * (int)std::max<int64_t>(1, std::min<int64_t>(max_clusters, tiles_upper));
  const cudaError_t e = launch_dependent(gmm_fp4_kernel<FMT, EPI>, grid, kThreads, kSmem, s, m[0],
                                         m[1], m[2], m[3], m[4], m[5], m[6], p);
  if (e != cudaSuccess) {
    set_error("moe_gmm_fp4 launch: %s", cudaGetErrorString(e));
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // namespace

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
  p.n_tiles = swiglu ? (p.F + BN / 2 - 1) / (BN / 2) : (a.N + BN - 1) / BN;
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
  CUtensorMap m[7];
  const int64_t ac = (a.K + acols - 1) / acols;
  const int64_t stride_b = a.E > 1 ? a.stride_b : (int64_t)a.N * a.ldb;
  bool ok = make_code_map(&m[0], a.A, a.K / 2, a.rows_cap, a.lda, 1, a.rows_cap * a.lda, BM) &&
            make_code_map(&m[1], a.B, a.K / 2, a.N, a.ldb, a.E, stride_b, BN / 2) &&
            make_scale_map(&m[2], a.sfa, ac, p.atom_rows2, atoms, 1) &&
            make_scale_map(&m[3], a.sfb, ac, 2 * (int64_t)a.E * p.n_tiles, atoms, 2);
  ok = ok && make_code_map(&m[6], a.A, a.K / 2, a.rows_cap, a.lda, 1, a.rows_cap * a.lda, 32);
  if (swiglu && a.C != nullptr) {
    const uint16_t *H = static_cast<const uint16_t *>(a.C);
    ok = ok && make_out_map(&m[4], H, false, p.F, a.rows_cap, a.ldc) &&
         make_out_map(&m[5], H + p.F, false, p.F, a.rows_cap, a.ldc);
  } else if (!swiglu) {
    ok = ok && make_out_map(&m[4], a.C, p.c_f32, a.N, a.rows_cap, a.ldc);
    m[5] = m[4];
  } else {
    m[4] = m[5] = m[0];
  }
  if (!ok) {
    set_error("moe_gmm_fp4: cannot encode a TMA descriptor");
    return MOE_ERR_CUDA;
  }
  // pairs of row tiles: at most one partly filled pair an expert that has rows
  const int64_t live = std::min<int64_t>(a.E, a.rows_cap);
  const int64_t tiles_upper = ((a.rows_cap + 2 * BM - 1) / (2 * BM) + live) * p.n_tiles;
  if (swiglu)
    return nv ? launch<MOE_FP4_NV, MOE_EPI_SWIGLU_FWD>(m, p, tiles_upper, s)
              : launch<MOE_FP4_MX, MOE_EPI_SWIGLU_FWD>(m, p, tiles_upper, s);
  return nv ? launch<MOE_FP4_NV, MOE_EPI_NONE>(m, p, tiles_upper, s)
            : launch<MOE_FP4_MX, MOE_EPI_NONE>(m, p, tiles_upper, s);
}

}  // namespace moe

// sm_103a building blocks of the 4-bit GEMM beside those of tc_sm103.cuh:
// uniform issue, non-blocking barrier tests, the kind::mxf4nvf4 MMA.
#pragma once
#include "tc_sm103.cuh"

namespace moe {
namespace tc {

// Whether the phase with the given parity has completed, without waiting.
MOE_DEVINL bool mbar_test(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// One arrival on a barrier of this CTA.
MOE_DEVINL void mbar_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// One arrival on a barrier of the cluster that orders no memory: what it hands over
// are tensor-memory columns, whose reads tcgen05.wait::ld and the fence before it
// have ended.  A releasing arrival would also wait for the warp's global stores,
// some 2000 cycles.
MOE_DEVINL void mbar_arrive_cluster_relaxed(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// tma_load_3d_2sm for five dimensions.
MOE_DEVINL void tma_load_5d_2sm(void *dst, const CUtensorMap *map, uint32_t bar, int c0, int c1,
                                int c2, int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}

// A shared-memory descriptor whose address is `units` of 16 bytes past that of d.
// The sum stays in the low word, so that a K block's descriptors differ from one
// register by constants.
MOE_DEVINL uint64_t desc_at(uint64_t d, uint32_t units) {
  return (d & 0xffffffff00000000ull) | ((uint32_t)d + units);
}

// True in one lane of a converged warp.  Tensor-core and TMA instructions take
// their operands from uniform registers.  Issued behind `if (elect_one())` by a warp
// whose control flow and operands are uniform they cost far less than behind
// `if (lane == 0)`: the 4-bit GEMM, which issues 10 to 16 of them a K block, ran
// 32768 rows of 4096 x 28672 in 1.36 ms with the one and in 2.41 ms with the other.
MOE_DEVINL bool elect_one() {
  uint32_t pred;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(pred));
  return pred != 0;
}

// A value that every lane holds alike, as one the compiler knows to be uniform.
MOE_DEVINL int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// Instruction descriptor of kind::mxf4nvf4 with block scaling, fp32
// accumulation, both operands K-major E2M1 (format 1): bits 4-5 and 29-30 the
// first byte of B's / A's 32-bit scale words that this MMA uses (scale_vec::4X
// takes the whole word, id 0; scale_vec::2X two bytes, id 0 or 2), 23 scale
// format (0 = UE4M3, 1 = UE8M0), 17-22 N >> 3, 27-28 M >> 7, 31 K (0 = 64).
__host__ __device__ constexpr uint32_t idesc_fp4(int M, int N, bool nv, int sf_id) {
  return (static_cast<uint32_t>(sf_id) << 4) | (1u << 7) | (1u << 10) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(!nv) << 23) |
         (static_cast<uint32_t>(M >> 7) << 27) | (static_cast<uint32_t>(sf_id) << 29);
}

// 4-bit block-scaled MMA over both CTAs of the pair (K = 64 codes): one E4M3
// scale per 16 codes (NV) or one E8M0 scale per 32.
template <bool NV>
MOE_DEVINL void umma_fp4_2sm(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                             uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
  if (NV)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X"
        " [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem),
        "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::2X"
        " [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem),
        "r"(accumulate)
        : "memory");
}

}  // namespace tc
}  // namespace moe

// Where the sequences' balance loss keeps what its blocks leave one another.
#pragma once
#include <cstddef>
#include <cstdint>

namespace moe {

// First the blocks' terms of the two losses (pairs of fp32, 8 bytes at a time), of as many blocks as
// there are or a sequence each and two; then their parts of P, [blocks + B, E] fp32.  The caller's
// memory is aligned to 4 bytes: the terms start at the next multiple of 8.
struct SeqAuxLayout {
  void *terms_at, *part_at;
  size_t bytes;
  SeqAuxLayout(void *p, int64_t blocks, int E, int B) {
    const size_t slots = (size_t)blocks + (size_t)B, terms = 8 * (slots + 2);
    const uintptr_t at = (reinterpret_cast<uintptr_t>(p) + 7) & ~(uintptr_t)7;
    terms_at = reinterpret_cast<void *>(at);
    part_at = reinterpret_cast<void *>(at + terms);
    bytes = 16 + terms + 4 * slots * (size_t)E;
  }
};

}  // namespace moe

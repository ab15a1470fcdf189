"""The balance loss's workspace may start on any 4 bytes: csrc/seqaux_layout.h compiled on the host and
laid out at every such address."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mixture_experts_grouped_router_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <initializer_list>
#include "seqaux_layout.h"

int main() {
  int wrong = 0;
  for (uintptr_t p = 4096; p < 4096 + 32; p += 4)
    for (int64_t blocks : {0, 1, 7, 1280})
      for (int E : {1, 2, 33, 256})
        for (int B : {1, 2, 501, 65536}) {
          const moe::SeqAuxLayout w((void *)p, blocks, E, B), aligned((void *)4096, blocks, E, B);
          const uintptr_t terms = (uintptr_t)w.terms_at, part = (uintptr_t)w.part_at;
          const size_t slots = (size_t)blocks + B;
          wrong += terms % 8 != 0 || part % 4 != 0;
          wrong += terms < p || part < terms + 8 * (slots + 2);
          wrong += part + 4 * slots * E > p + w.bytes;
          wrong += w.bytes != aligned.bytes;  // what the caller asked for
        }
  std::printf("wrong %d\n", wrong);
  return wrong != 0;
}
"""


def test_pairs_start_on_eight_bytes(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-I" + CSRC, str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,B", [(2000, 64, 2, 3), (300, 256, 8, 60), (100, 8, 2, 1)])
@pytest.mark.parametrize("sigmoid", [0, 1])
def test_a_workspace_off_eight_bytes(T, E, k, B, sigmoid):
    """By chunks, by sequences and by one block: the same numbers from any address."""
    import torch
    from mixture_experts_grouped_router_gb300 import _lib as L
    gen = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, E, generator=gen, device="cuda")
    idx = x.topk(k, 1).indices.to(torch.int32)
    off = (torch.arange(B + 1, device="cuda") * T // B).to(torch.int32)
    nb = L.moe_seq_aux_loss_workspace_bytes(T, E, B)
    got = []
    for shift in (0, 4, 8, 12):
        whole = torch.full((nb + 32,), 0xAB, dtype=torch.uint8, device="cuda")
        counts, tokens = (torch.empty(s, dtype=torch.int32, device="cuda") for s in (B * E, B))
        probs, loss, d = torch.empty(B, E, device="cuda"), torch.empty(2, device="cuda"), torch.empty_like(x)
        L.moe_seq_aux_loss(x, idx, off, sigmoid, 0.3, 0.05, counts, tokens, probs, loss,
                           whole[shift:shift + nb], d_logits=d)
        assert (whole[:shift] == 0xAB).all() and (whole[shift + nb:] == 0xAB).all()
        got.append((counts, tokens, probs, loss, d))
    assert torch.isfinite(got[0][3]).all()
    for g in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], g))

"""Static rules on the CUDA sources of the dense attention calls (CPU only).

- A lane leaves a bounded wait on its own clock, so lanes of a warp may disagree on whether its limit
  ran out. The code behind a wait has instructions that the whole warp has to reach together (tensor
  memory accesses, votes, barriers): each wait is followed by a vote that makes the outcome one.
"""
import os

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "hierarchical_sparse_attention_index_gb300", "csrc")


def lines(name):
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        return [x.split("//")[0] for x in f.read().splitlines()]


def test_the_warp_votes_after_each_bounded_wait():
    waits = 0
    for name in ("paged_rows.cu", "prompt_attn.cu"):
        src = lines(name)
        for i, x in enumerate(src):
            if "wait_bar(" in x:
                waits += 1
                assert any("__all_sync(0xffffffffu, ok)" in y for y in src[i:i + 7]), f"{name}:{i + 1}: no vote behind the wait"
    assert waits > 0

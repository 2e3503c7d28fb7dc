"""Static rules on the CUDA sources of the dense attention calls (CPU only).

- A lane leaves a bounded wait on its own clock, so lanes of a warp may disagree on whether its limit
  ran out. The code behind a wait has instructions that the whole warp has to reach together (tensor
  memory accesses, votes, barriers): each wait is followed by a vote that makes the outcome one.
- What the dense calls' headers define is used, and defined once.
"""
import os
import re

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


def test_helpers_are_used_and_defined_once():
    files = ("hsa_dense.h", "hsa_softmax.cuh", "hsa_flash.cuh", "hsa_paged.cuh", "paged_write.cu", "paged_attn.cu", "paged_rows.cu",
             "prompt_attn.cu")
    text = {name: "\n".join(lines(name)) for name in files}
    defined = {}
    for name, t in text.items():
        if name.endswith(".cuh"):
            for x in re.findall(r"__forceinline__ [\w:]+ (\w+)\(", t) + re.findall(r"^constexpr \w+ (k\w+) =", t, re.M):
                defined.setdefault(x, []).append(name)
    assert defined
    for x, where in defined.items():
        uses = sum(len(re.findall(rf"\b{x}\b", t)) for t in text.values())
        assert len(where) == 1 and uses > 1, f"{x} of {where}: defined {len(where)} times, named {uses} times"
        for name in files:
            if name.endswith(".cu"):
                again = re.search(rf"(?:__forceinline__ [\w:]+ {x}\(|^constexpr \w+ {x} =)", text[name], re.M)
                assert not again, f"{name} defines {x} of {where[0]} again"

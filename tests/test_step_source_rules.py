"""Static rules on the CUDA sources of the speculative step's calls (CPU only): what their headers define is used and defined once,
and the kernel that hands registers from group to group takes no more than its launch holds."""
import os
import re

from tests.test_dense_source_rules import lines

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "hierarchical_sparse_attention_index_gb300", "csrc")
HEADERS = ("hsa_four.cuh", "hsa_rows.cuh", "hsa_paged_warp.cuh")


def test_helpers_are_used_and_defined_once():
    text = {name: "\n".join(lines(name)) for name in sorted(os.listdir(CSRC)) if name.endswith((".cu", ".cuh", ".h"))}
    found = 0
    for header in HEADERS:
        names = re.findall(r"__forceinline__ (?:constexpr )?[\w:]+ (\w+)\(", text[header]) + re.findall(r"^constexpr \w+ (k\w+) =", text[header], re.M)
        for x in names:
            found += 1
            assert sum(len(re.findall(rf"\b{x}\b", t)) for t in text.values()) > 1, f"{header}: {x} is not used"
    assert found > 20


def test_register_shares():
    """Each role of the tcgen05 decode kernel goes on with whole groups of 8 registers, and their sum is at most the launch's."""
    src = "\n".join(lines("paged_rows.cu"))
    groups = re.findall(r"kThreads = (\d+) \* 32.*?kLaunchRegs = (\d+), kSoftRegs = (\d+), kIssueRegs = (\d+), kOutRegs = (\d+), kLastRegs = (\d+);", src, re.S)
    assert len(groups) == 2
    for warps, launch, soft, issue, out, last in (map(int, g) for g in groups):
        shares = [soft, soft, issue, out] + [last] * (warps // 4 - 4)
        assert all(x % 8 == 0 for x in shares) and sum(shares) <= launch * (warps // 4) and launch * warps * 32 <= 65536

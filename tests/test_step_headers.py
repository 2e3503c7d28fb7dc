"""What the headers of the speculative step's calls define has one definition where it can be seen: the headers share namespace hsa,
so no other header may hold the name, and no source that includes them, nor do they hold it twice. And it is used somewhere."""
import os
import re

from tests.test_dense_source_rules import CSRC, lines

HEADERS = ("hsa_four.cuh", "hsa_rows.cuh", "hsa_paged_warp.cuh")
FUNCTION = r"(?:__forceinline__|inline|constexpr|cudaError_t) (?:constexpr )?(?:[\w:]+ )?{}\("


def definitions(name, text):
    """Places where `name` is defined as a function (templates with their only form) or a constant."""
    return len(re.findall(r"^(?:template <[^\n]*>\n)?(?:static )?(?:__\w+__ )*" + FUNCTION.format(name), text, re.M)) + \
        len(re.findall(rf"^(?:static )?constexpr [\w:]+ {name}\b(?!\()", text, re.M))


def test_one_definition_and_a_use():
    text = {n: "\n".join(lines(n)) for n in sorted(os.listdir(CSRC)) if n.endswith((".cu", ".cuh", ".h"))}
    sees = {n: set(re.findall(r'#include "(\w+\.cuh?h?)"', t)) for n, t in text.items()}
    names = 0
    for header in HEADERS:
        here = set(re.findall(r"__forceinline__ (?:constexpr )?[\w:]+ (\w+)\(", text[header])) | set(re.findall(r"^constexpr [\w:]+ (\w+)\b", text[header], re.M)) | \
            set(re.findall(r"^cudaError_t (\w+)\(", text[header], re.M))
        for x in sorted(here):
            names += 1
            assert definitions(x, text[header]) == 1, f"{header} defines {x} {definitions(x, text[header])} times"
            for other, t in text.items():
                if other != header and (other.endswith((".cuh", ".h")) or header in sees[other]):
                    assert definitions(x, t) == 0, f"{other} defines {x} of {header} again"
            uses = sum(len(re.findall(rf"\b{x}\b", t)) for t in text.values()) - definitions(x, text[header])
            assert uses > 0, f"{header}: {x} is not used"
    assert names > 25

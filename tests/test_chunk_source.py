"""What no run can show of csrc/attn_chunk.cu: a commit covers the products of the thread that issues it, so
products and commits have to come from one lane, and elect.sync does not say which lane it picks."""
import os
import re

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "decoder_only_transformer_layer_b200",
                   "csrc", "attn_chunk.cu")


def elected_blocks(src):
    """The bodies of `if (elected()) { .. }`."""
    out = []
    for m in re.finditer(r"if \(elected\(\)( && ok)?\) \{", src):
        depth, at = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(src[at], 0)
            at += 1
        out.append((m.end(), at))
    return out


def test_products_and_commits_are_the_elected_lanes():
    src = open(SRC).read()
    kernel = src[src.index("chunk_attn_kernel("):]
    blocks = elected_blocks(kernel)
    calls = list(re.finditer(r"\b(mma_ss|mma_ts|tc_commit)\(", kernel))
    assert {m.group(1) for m in calls} == {"mma_ss", "mma_ts", "tc_commit"}
    for m in calls:
        assert any(a <= m.start() < b for a, b in blocks), kernel[m.start():m.start() + 60]
    # a commit in assembly of its own elects its lane
    for asm in re.findall(r"asm volatile\((.*?)\);", src, re.S):
        if "tcgen05.commit" in asm:
            assert "elect.sync _|e" in asm and "@e tcgen05.commit" in asm

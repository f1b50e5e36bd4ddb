"""Rules of the PTX ISA and of bounded waits that the cache's kernels keep, read off their sources: what
would break them could fault or hang a GPU, so it is not tried there."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_decoding_gb300", "csrc")


def source(name):
    """A source file without its comments."""
    return re.sub(r"/\*.*?\*/|//[^\n]*", "", open(os.path.join(CSRC, name)).read(), flags=re.S)


def block(text, head):
    """The text from `head` to the end of the braces that open after it."""
    at = text.index(head)
    depth, i = 0, text.index("{", at)
    for j in range(i, len(text)):
        depth += (text[j] == "{") - (text[j] == "}")
        if depth == 0:
            return text[at:j + 1]
    raise AssertionError(f"no end of {head}")


def test_warpgroups_meet_in_one_register_instruction():
    """setmaxnreg is .sync.aligned: all warps of a warpgroup execute the same instruction."""
    kernel = block(source("kv4_prompt.cu"), "attn_prompt_kernel(const Kv4 c")
    assert re.findall(r"setmaxnreg_(?:inc|dec)<(\w+)>\(\);", kernel) == ["kSoftRegs", "kUnpackRegs", "kMmaRegs"]
    # the branches that lead to them part whole warpgroups
    warps = [int(x) for x in re.findall(r"constexpr int kMmaWarp = (\d+);", source("kv4_prompt.cu"))]
    assert warps and warps[0] % 4 == 0
    roles = re.findall(r"\n    (?:\} else )?(if \([^\n]*\)|else) \{\s*setmaxnreg|\n    \} (else) \{\s*setmaxnreg", kernel)
    assert [a or b for a, b in roles] == ["if (warp < 8)", "if (warp < kMmaWarp)", "else"]

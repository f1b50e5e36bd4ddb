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


def test_prompt_roles_end_after_a_wait_that_ran_out():
    """A thread whose wait ran out goes on with polls. It must not use a piece of work that may not be
    there, write over one that is read, or meet others at a barrier without a bound."""
    kernel = block(source("kv4_prompt.cu"), "attn_prompt_kernel(const Kv4 c")
    roles = kernel[kernel.index("setmaxnreg_inc"):]
    roles = roles[:roles.rindex("__syncthreads()")]
    for unbounded in ("bar.sync", "barrier.sync", "__syncthreads", "while (!mbar"):
        assert unbounded not in roles, unbounded
    get = block(kernel, "const auto get_piece")
    assert "dead = __any_sync(~0u, dead);" in get
    assert re.search(r"if \(dead\)\s*w\.nblk = w\.n0 = w\.n1 = 0;", get)  # no piece
    # the other reader of the ring, and its writer
    assert re.search(r"nblk = dead \? 0 : sh\.piece", roles)
    assert re.search(r"if \(dead\)\s*break;\s*sh\.piece\[p % kRing\] = w;", roles)
    # the MMAs in flight are waited for once more before the tensor memory is given back
    assert re.search(r"if \(n > 0\) \{\s*dead = false;\s*wait\(sh\.k_empty", roles)


def test_rows_kernel_waits_for_its_copies_after_a_wait_that_ran_out():
    """No copy may be in flight when its shared memory is used for the parts or given back, and no barrier
    may be armed again before its copy is there: after a wait that ran out the warp asks for no more cells."""
    kernel = block(source("kv4_attn.cu"), "attn_rows_kernel(const Kv4 c")
    assert re.search(r"int mine = !dead && ", kernel)
    rest = kernel[kernel.index("kv4_wait(bars + 8 * st"):]
    out = block(rest, "if (__any_sync(~0u, dead))")
    assert rest.index("if (__any_sync(~0u, dead))") < rest.index("const uint32_t filled")
    assert re.search(r"for \(int z = x; z < x \+ S && z < mine; \+\+z\) \{\s*dead = false;\s*kv4_wait\(", out)
    assert re.search(r"dead = true;\s*mine = x;\s*break;", out)


def test_append_reads_q_as_memory_that_it_writes():
    """q_out may be q: loads by the read-only path are for memory that no thread of the kernel writes."""
    text = source("kv4.cu")
    turn = block(text, "void append_q(")
    assert re.findall(r"(\w+)<N>\(a\.q \+", turn) == ["load_own"]
    own = block(text, "Raw<N> load_own(")
    assert "ldg" not in own and ".nc" not in own

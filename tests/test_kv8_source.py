"""Rules of the PTX ISA and of bounded waits that the kernels over the 8-bit cache keep, read off their sources: what
would break them could fault or hang a GPU, so it is not tried there."""
import re

from tests.test_kv4_source import block, source


def test_warpgroups_meet_in_one_register_instruction():
    """setmaxnreg is .sync.aligned: all warps of a warpgroup execute the same instruction."""
    text = source("kv8_prompt.cu")
    kernel = block(text, "kv8_prompt_kernel(const Kv4 c")
    assert re.findall(r"setmaxnreg_(?:inc|dec)<(\w+)>\(\);", kernel) == ["kSoftRegs", "kUnpackRegs", "kMmaRegs"]
    # the branches that lead to them part whole warpgroups
    (warps,) = [int(x) for x in re.findall(r"constexpr int kMmaWarp = (\d+);", text)]
    assert warps % 4 == 0
    roles = re.findall(r"\n    (?:\} else )?(if \([^\n]*\)|else) \{\s*setmaxnreg|\n    \} (else) \{\s*setmaxnreg",
                       re.sub(r"\n\s*\n", "\n", kernel))
    assert [a or b for a, b in roles] == ["if (warp < 8)", "if (warp < kMmaWarp)", "else"]
    # what is taken is what the launch gave (a share above it would wait for ever)
    value = {k: int(v) for k, v in re.findall(r"\b(k\w+) = (\d+)\b", text)}
    assert 256 * value["kSoftRegs"] + 128 * value["kUnpackRegs"] + 128 * value["kMmaRegs"] <= 512 * value["kLaunchRegs"] <= 65536


def test_prompt_roles_end_after_a_wait_that_ran_out():
    """A thread whose wait ran out goes on with polls. It must not use a piece of work that may not be
    there, write over one that is read, or meet others at a barrier without a bound."""
    kernel = block(source("kv8_prompt.cu"), "kv8_prompt_kernel(const Kv4 c")
    roles = kernel[kernel.index("setmaxnreg_inc"):]
    roles = roles[:roles.rindex("__syncthreads()")]
    for unbounded in ("bar.sync", "barrier.sync", "__syncthreads", "while (!mbar", "cp.async.wait_group"):
        assert unbounded not in roles, unbounded
    get = block(kernel, "const auto get_piece")
    assert "dead = __any_sync(~0u, dead);" in get
    assert re.search(r"if \(dead\)\s*w\.nblk = w\.n0 = w\.n1 = 0;", get)  # no piece
    # the softmax warps and the MMA warp read the ring in place, and its writer
    assert re.search(r"dead = __any_sync\(~0u, dead\);\s*const Piece &w = sh\.piece[^;]*;\s*const bool none = dead \|\| w\.nblk == 0;", roles)
    assert re.search(r"nblk = dead \? 0 : sh\.piece", roles)
    assert re.search(r"if \(dead\)\s*break;\s*sh\.piece\[p % kRing\] = w;", roles)
    # the MMAs in flight are waited for once more before the tensor memory is given back, and a role's copies
    # before it ends
    assert re.search(r"if \(n > 0\) \{\s*dead = false;\s*wait\(sh\.k_empty", roles)
    assert re.search(r"while \(w\.nblk > 0 \|\| more\);\s*async_copies_wait\(\);", roles)


def test_kernels_of_few_rows_wait_for_their_copies_after_a_wait_that_ran_out():
    """No copy may be in flight when its shared memory is used for the parts or given back, and no barrier
    may be armed again before its copy is there: after a wait that ran out the warp asks for no more cells."""
    text = source("kv8_attn.cu")
    for name, mine in (("kv8_rows_kernel(const Kv4 c", r"int mine = !dead && "), ("kv8_lists_kernel(const Kv4 c", r"int mine = dead \|\| ")):
        kernel = block(text, name)
        assert re.search(mine, kernel)
        rest = kernel[kernel.index("kv4_wait(bars + 8 * st"):]
        out = block(rest, "if (__any_sync(~0u, dead))")
        assert rest.index("if (__any_sync(~0u, dead))") < rest.index("if (have >> st & 1u)")
        assert re.search(r"for \(int z = x; z < x \+ S && z < mine; \+\+z\) \{\s*dead = false;\s*kv4_wait\(", out)
        assert re.search(r"dead = true;\s*mine = x;\s*break;", out)


def test_clusters_leave_and_write_together():
    """Shared memory of another CTA is written only after all have started (a wait before the first store) and
    before the first one can leave (a meeting after the last); a CTA returns with its whole cluster."""
    kernel = block(source("kv8_select.cu"), "select_kernel(const Kv4 c")
    order = [kernel.index(x) for x in ("cluster_arrive();", "cluster_wait();", "return;", "st_cluster_f32(", "cluster_sync();", "if (rank > 0)")]
    assert order == sorted(order)
    # between the meetings no CTA returns by its rank, nor by a thread's own condition
    before = kernel[:kernel.index("cluster_sync();")]
    assert [x.strip() for x in re.findall(r"if \(([^\n]*)\)\s*return;", before)] == ["unit >= a.units || i >= b.n_seqs || nth < 0", "nt <= 0"]


def test_append_reads_q_as_memory_that_it_writes():
    """q_out may be q: loads by the read-only path are for memory that no thread of the kernel writes."""
    text = source("kv8.cu")
    turn = block(text, "void append_q(")
    assert re.findall(r"load_raw<N, (\w+)>\(a\.q \+", turn) == ["true"]
    load = block(text, "Raw<N> load_raw(")
    assert re.findall(r"kOwn \? \*\(const (\w+) \*\)at : __ldg", load) == ["uint4", "uint2"]

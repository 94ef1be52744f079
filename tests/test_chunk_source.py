"""What the tensor-core chunk kernel's source must keep to, checked without a GPU: rules of the instruction set whose
violation may hang a GPU, so that no test runs into one."""

import os
import re

from asymmetric_bit_kv_b200.build import CSRC

SOURCE = open(os.path.join(CSRC, "kvq_chunk_tc.cu")).read()


def _kernel():
    at = SOURCE.index("chunk_tc_kernel(const __grid_constant__")
    return SOURCE[at:SOURCE.index("\n}\n", at)]


def test_a_warpgroup_executes_one_setmaxnreg():
    """All threads of a warpgroup must execute the same setmaxnreg: each stands first in a branch on the warpgroup, and
    the warpgroups' registers add up to what the block is launched with."""
    kernel = _kernel()
    assert "const int group = warp >> 2;" in kernel
    found = re.findall(r"(?:if \((.*)\)|else) \{\n\s*asm volatile\(\"setmaxnreg\.(inc|dec)\.sync\.aligned\.u32 (\d+);", kernel)
    assert len(found) == kernel.count("setmaxnreg.")
    threads = int(re.search(r"kThreads = (\d+);", SOURCE)[1])
    regs = []
    for g in range(threads // 128):
        for cond, _, n in found:
            assert re.fullmatch(r"group < \d+|", cond), cond
            if not cond or g < int(cond.split()[-1]):
                regs.append(int(n))
                break
    assert len(regs) == threads // 128
    launched = 65536 // threads // 8 * 8
    assert sum(regs) <= launched * len(regs), (regs, launched)


def _function(name):
    at = SOURCE.index(name + "(const ChunkParams& p")
    return SOURCE[at:SOURCE.index("\n}\n", at)]


def test_copies_in_flight_are_waited_for_however_an_item_ends():
    """A warp that gives up a wait ends the others' waits, so that nobody may be left to wait for the last copies into
    shared memory and the last products: whoever issued them does, after its last one, before the block ends."""
    for name in ("copy_parts", "produce_exact"):
        body = _function(name)
        for exit_ in re.finditer("return (true|false);", body):
            # between the last copy issued (or the failed wait) and the return
            before = body[:exit_.start()]
            at = max(before.rfind("bulk_g2s("), before.rfind("cp.async"), before.rfind("mbar_wait"))
            assert "mbar_drain(" in before[at:], (name, exit_[0])
    kernel = _kernel()
    products = kernel[kernel.index("issue_products("):]
    products = products[:products.index("copy_parts(")]
    assert not re.search(r"!issue_products|if \([^)]*\) tc_commit\(bar\.drain\)", products.replace("if (elect_one())", ""))
    assert products.index("tc_commit(bar.drain)") < products.index("mbar_drain(bar.drain, 0)")


def test_a_build_with_fewer_registers_is_refused_on_the_host():
    """A warpgroup that asks for more registers than the block was launched with waits forever: the launcher compares the
    compiled kernel's count with the shares before its first launch."""
    kernel, at = _kernel(), SOURCE.index("cudaError_t launch_chunk_tc(")
    launcher = SOURCE[at:SOURCE.index("chunk_tc_kernel<<<", at)]
    assert "numRegs" in launcher and "kLaunchRegisters" in launcher
    shares = [int(n) for n in re.findall(r"setmaxnreg\.\w+\.sync\.aligned\.u32 (\d+);", kernel)]
    per_group = [shares[0], shares[0], shares[1], shares[1], shares[2]]
    assert int(re.search(r"kLaunchRegisters = (\d+);", SOURCE)[1]) * len(per_group) >= sum(per_group)

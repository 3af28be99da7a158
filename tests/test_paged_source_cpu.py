"""What the paged kernels' safety rests on and no run can show: read from their source."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sliding_window_gqa_prep_gb300", "csrc")


def kernels():
    """(file, name, body without comments) of every __global__ function."""
    for f in sorted(os.listdir(CSRC)):
        if not f.endswith(".cu"):
            continue
        with open(os.path.join(CSRC, f)) as h:
            s = re.sub(r"//[^\n]*|/\*.*?\*/", "", h.read(), flags=re.S)
        for part in s.split("__global__")[1:]:
            name = re.search(r"(\w+)\s*\((?:const|\w+Params)", part)
            yield f, name.group(1) if name else "?", part


def test_tmem_is_allocated_after_the_wait():
    """A kernel launched ahead of the end of the one in front must not hold tensor memory while
    it waits: the kernel in front may still have its own to allocate on the same SM, and neither
    would ever go on."""
    found = 0
    for f, name, body in kernels():
        at = body.find("tc_alloc(")
        if at < 0:
            continue
        found += 1
        wait = body.find("pdl_wait()")
        assert 0 <= wait < at, (f, name)
    assert found >= 4


@pytest.mark.parametrize("name", ["griddepcontrol.wait", "tcgen05.alloc"])
def test_the_wrappers_are_what_the_kernels_use(name):
    """The instructions stand in their wrappers alone, so that the order above is the order."""
    n = 0
    for f in os.listdir(CSRC):
        with open(os.path.join(CSRC, f)) as h:
            n += h.read().count(name + (";" if name.startswith("grid") else "."))
    assert n == 1


def test_register_shares_are_checked():
    """Registers that setmaxnreg hands out come from what the CTA was launched with. The shares stand
    against the launch's at compile time, and the compiler's count is checked before the first launch:
    a build with fewer (other flags, another compiler) is an error, not a hang."""
    users = [f for f in sorted(os.listdir(CSRC)) if "setmaxnreg." in open(os.path.join(CSRC, f)).read()]
    assert users == ["swa_paged_chunk.cu"]
    with open(os.path.join(CSRC, users[0])) as h:
        s = h.read()
    assert re.search(r"static_assert\([^;]*R_SOFT[^;]*R_REST[^;]*THREADS \* REGS", s)
    assert 'setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(C::R_REST)' in s
    assert 'setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(C::R_SOFT)' in s
    assert re.search(r"allow_smem<paged_chunk_kernel<T, D>>\([^;]*ChunkCfg<D>::REGS\)", s)

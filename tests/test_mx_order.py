"""What orders the MXFP4 kernels' accesses and no result shows: looks at the sources, on the CPU.

The kernels begin before the preceding kernel of the stream has ended, so what that one writes
must not be read through the non-coherent path (its data may not change during a kernel, and a cache
line from before the wait would be stale)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "decode_w4a16_g128_b200", "csrc")
FILES = sorted(glob.glob(os.path.join(CSRC, "mx*.cuh")))


def code(path):
    return re.sub(r"//[^\n]*", "", open(path).read())


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_no_load_through_the_non_coherent_path(path):
    found = re.findall(r"__ldg\b|ldg_nc\w*|\.global\.nc\b|__restrict__", code(path))
    assert not found, found


def test_the_files_are_there():
    assert len(FILES) == 5


def test_codes_are_released_behind_a_warp_barrier():
    """A codes slot is handed back by one lane's arrival: between the warp's loads of it and that arrival
    there has to be a barrier that orders memory, which a vote is not."""
    text = code(os.path.join(CSRC, "mx_gemm.cuh"))
    at = [m.start() for m in re.finditer(r"mbar_arrive\(&w_empty", text)]
    assert len(at) == 2
    loads = text.index("c[q] = lds128(src[q])")
    for a in at:
        assert "__syncwarp();" in text[loads:a]


@pytest.mark.parametrize("name,roles", [("mx_gemm.cuh", ("codes to BF16", "- epilogue")),
                                        ("mx_a4.cuh", ("- scales\n", "epilogue: half of the columns"))])
def test_a_warp_gives_up_as_one(name, roles):
    """Warps that wait with all lanes and then take part in collective instructions must not have some of
    them leave: their waits are those with one outcome for the warp."""
    text = open(os.path.join(CSRC, name)).read()
    for role in roles:
        at = [m.start() for m in re.finditer("------ *" + role if role[0] != "-" else "-----" + role, text)]
        assert at, role
        section = text[at[-1]:]
        section = section[:section.find("} else if") if "} else if" in section else len(section)]
        assert "mbar_wait_warp(" in section and not re.search(r"\bmbar_wait(_spin|_cluster)?\(", section), role

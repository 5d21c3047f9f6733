"""The DRAM traffic that bench.py reports is a capture, taken while the kernel's sources are the ones that it was made of;
csrc/sm100.cuh is one of them for every kernel of the gated linear attention passes."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "chunkwise_gated_linear_gla_gb300", "csrc")


def test_the_shared_header_holds_what_the_shared_kernels_use():
    """A helper of one operator's kernels alone lies beside them: in the shared header it would only make the other
    kernels' captures out of date."""
    with open(os.path.join(CSRC, "sm100.cuh")) as f:
        head = f.read()
    names = set(re.findall(r"__device__ __forceinline__ [\w ]+?\b(\w+)\(", head))
    assert "mbar_wait" in names and "tmem_ld16" in names
    rest, delta = "", ""
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        name = os.path.basename(path)
        with open(path) as f:
            if name.startswith("gla_delta"):
                delta += f.read()
            elif name != "sm100.cuh":
                rest += f.read()
    used = lambda n, text: len(re.findall(r"\b%s\b" % n, text))  # noqa: E731
    alone = [n for n in sorted(names) if used(n, delta) and not used(n, rest) and used(n, head) < 2]
    assert not alone, alone

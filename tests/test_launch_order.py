"""The order of a kernel's set-up and the release of the next kernel.

A kernel may be started early, beside the one before it on the stream, as soon
as every CTA of that one has called pdl_launch_dependents(); it then waits for
the earlier kernel's end.  A CTA that has not got its tensor memory by then
could find it taken by such a waiting kernel, and neither would ever go on.  So
a CTA calls pdl_launch_dependents() only when its allocation is known to be
done: behind a barrier of the CTA that the allocating warp reaches after it.
"""
import glob
import os
import re

from conftest import ROOT

CSRC = os.path.join(ROOT, "bit_gemm_quant_b200", "csrc")


def kernels():
    """(file, kernel name, body) of every __global__ function that allocates tensor memory."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for part in re.split(r"\b__global__\b", text)[1:]:
            body = part[:part.find("\n}\n")]
            if "tmem_alloc(" in body:
                yield os.path.basename(path), re.search(r"(\w+_kernel)\(", body).group(1), body


def test_dependents_start_behind_the_allocation():
    found = list(kernels())
    assert {f for f, _, _ in found} == {"gemm_tc.cu", "mx_gemm.cu", "experts_tc.cu"}
    for path, name, body in found:
        alloc, release = body.find("tmem_alloc("), body.find("pdl_launch_dependents()")
        assert body.count("tmem_alloc(") == 1 and body.count("pdl_launch_dependents()") == 1, (path, name)
        assert 0 <= alloc < body.find("__syncthreads()", alloc) < release, (path, name)

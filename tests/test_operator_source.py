"""What a run cannot show without a fault: where the kernels' sources put a wait."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "vector_codebook_codec_b200", "csrc")


def _kernels():
    for path in (os.path.join(CSRC, "qamw_cross_entropy.cu"), os.path.join(CSRC, "qamw_mx4_gemm.cu")):
        with open(path) as f:
            source = re.sub(r"//[^\n]*", "", f.read())
        for body in re.split(r"__global__", source)[1:]:
            body = body[:body.index("\n}")]
            if "griddep_wait" in body:
                yield os.path.basename(path), re.search(r"(\w+_kernel)\(", body).group(1), body


@pytest.mark.parametrize("file,name,body", [pytest.param(*k, id=k[1]) for k in _kernels()])
def test_a_dependent_kernel_waits_before_its_roles_part(file, name, body):
    """A kernel that may start beside the one before it waits for it with all threads: a role's bounded wait that
    began earlier would count that kernel's time, and could give up while it still runs."""
    assert body.count("griddep_wait") == 1
    wait = body.index("griddep_wait")
    roles = [m.start() for m in re.finditer(r"\n  if \(warp == 0\) \{\n", body)]
    bounded = [m.start() for m in re.finditer(r"tc::wait(_warp)?\(|mbar_wait\(", body)]
    assert all(wait < w for w in bounded)
    # at the body's own indent, so that every thread comes by
    line = body[body.rindex("\n", 0, wait) + 1:wait]
    assert re.fullmatch(r"  (if \(g\.after_quantize\) )?tc::", line), line
    if roles:
        assert wait < roles[-1]

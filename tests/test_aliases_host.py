"""Tensors that a header lets be the same memory are not declared restrict where
they are written: the qualifier would promise the compiler otherwise."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp4_weight_mixture_02_amd", "csrc")


def _kernels():
    """Each kernel's name and its parameters."""
    out = {}
    for path in glob.glob(os.path.join(CSRC, "*.hip")):
        src = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__[^;{]*?\bvoid\s+(\w+)\s*\(", src, re.S):
            depth, at = 1, m.end()
            while depth:
                depth += {"(": 1, ")": -1}.get(src[at], 0)
                at += 1
            out[m[1]] = [re.sub(r"\s+", " ", p).strip() for p in src[m.end():at - 1].split(",")]
    return out


def test_restrict_is_not_promised_of_tensors_that_may_be_the_same():
    kernels = _kernels()
    assert len(kernels) > 40
    # add and dlogits of the balance losses' gradient; sum over x or residual
    # and dx over dsum (the norm's are members of one argument)
    for name, may_be_same in (("balance_bwd_kernel", ("add", "dlogits")), ("norm_kernel", ()), ("norm_bwd_kernel", ())):
        named = {re.split(r"[ *]", p)[-1]: p for p in kernels[name]}
        assert all(n in named for n in may_be_same)
        for n in may_be_same:
            assert "__restrict__" not in named[n], (name, named[n])
    assert kernels["norm_kernel"] == kernels["norm_bwd_kernel"] == ["NormArgs a"]
    fields = re.search(r"struct NormArgs \{(.*?)\n\};", open(os.path.join(CSRC, "norm.hpp")).read(), re.S)[1]
    assert "void* sum" in fields and "__restrict__" not in fields

"""When kernels let the next one on the stream start.

Every kernel is launched as a programmatic dependent.  One that releases its
dependents before its own wait lets the next kernel run beside the kernels before
itself, and a decode under KVQ_CACHE_READY then reads its early inputs while any of
those may still write them.  Only kvq_write does so, as kvq.h says (a decode
step's chain of write and decode gains by it), and the first two kernels of
kvq_calibrate_scales, whose last one waits."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_quantized_paged_gb300", "csrc")
EARLY = {("kvq_write.cu", "write_kernel"), ("kvq_calib.cu", "calib_kernel"), ("kvq_calib.cu", "calib_zero")}


def kernels():
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith((".cu", ".cuh")):
            continue
        text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
        at = [m.start() for m in re.finditer(r"__global__", text)] + [len(text)]
        for a, z in zip(at, at[1:]):
            body = text[a:z]
            yield name, re.search(r"(\w+)\s*\(\s*(?:const|uint32_t|__grid)", body).group(1), body


def test_release_comes_after_the_wait():
    early, seen = set(), 0
    for file, kernel, body in kernels():
        allow, wait = body.find("pdl_allow_next()"), body.find("pdl_wait()")
        if allow < 0:
            continue
        seen += 1
        assert wait >= 0, (file, kernel)
        if allow < wait:
            early.add((file, kernel))
    assert seen >= 12 and early == EARLY

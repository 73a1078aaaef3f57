"""Which kernels may release the next launch before they end (no GPU needed: the sources are read).  qmv streams its weights before
griddepcontrol.wait, so a kernel that writes weights must end first."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_fp4_fp_gb300", "csrc")


def kernels(name):
    """kernel name -> its source text."""
    text = open(os.path.join(CSRC, name)).read()
    starts = [(m.start(), m.group(1)) for m in re.finditer(r"__global__[^;{]*?\b(\w+_kernel)\s*\(", text)]
    return {n: text[at:text.index("\n}\n", at)] for at, n in starts}


def test_the_quantizers_end_before_what_is_behind_them_starts():
    found = kernels("quant.cu")
    assert {"quantize_kernel", "quantize_tiled_kernel", "quantize_nvfp4_tiled_kernel"} <= set(found)
    for name, body in found.items():
        if name.startswith("quantize"):
            assert "griddepcontrol.wait" in body and "launch_dependents" not in body, name


def test_what_releases_early_waits_first_or_writes_no_weights():
    """Elsewhere a kernel that releases early either waits before it does (so that whatever came before it is complete), or reads
    weights or a cache and writes none."""
    readers = {"qmv_tc_kernel", "qmv_kernel", "qmv_affine_kernel", "weight_stream_kernel", "kv_decode_kernel", "kv_prefill_kernel"}
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith(".cu"):
            continue
        for kernel, body in kernels(name).items():
            at = body.find("griddepcontrol.launch_dependents")
            waits = body.find("griddepcontrol.wait")
            if at >= 0 and not 0 <= waits < at:
                assert kernel in readers, (name, kernel)

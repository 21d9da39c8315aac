"""The build's check of spills covers the kernels: every one in csrc but the measurement probes."""
import glob
import os
import re

from varlen_top_select_amd import build


def kernels():
    found = {}
    for path in glob.glob(os.path.join(build.CSRC, "*.h*")):
        if os.path.basename(path) in build.PROBE_SOURCES:
            continue
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"__global__", text):
            # the name before the parameter list, behind __launch_bounds__(...)
            rest = re.sub(r"__launch_bounds__\((?:[^()]|\([^()]*\))*\)", "", text[m.end():m.end() + 400])
            found[re.search(r"(\w+)\s*\(", rest).group(1)] = os.path.basename(path)
    return found


def test_every_kernel_is_checked_for_spills():
    names = kernels()
    assert {"attend_kernel", "write_kernel", "prompt_kernel", "prompt_join_kernel", "topk_kernel"} <= set(names)
    missing = {n: f for n, f in names.items() if not any(k in n for k in build.NO_SCRATCH)}
    assert not missing

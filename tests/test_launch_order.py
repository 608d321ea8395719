"""CPU checks, on the sources, of the rules that kernels launched programmatically
behind another one keep: such a kernel is on the device while the one before it still
writes, and the wait (griddepcontrol.wait) is what makes those writes visible to it.
A kernel that breaks a rule may still give the right result for years, so no run shows it."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_paged_kv_q8_gb300", "csrc")
WAIT = 'asm volatile("griddepcontrol.wait;"'


def _kernels():
    """(file:name, parameter list, body) of every kernel that waits for the grid before it."""
    found = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__ void[^;{]*?\b(\w+_kernel)\(", text):
            depth, end = 1, m.end()
            while depth:                                    # the parameter list
                depth += {"(": 1, ")": -1}.get(text[end], 0)
                end += 1
            params, begin = text[m.end():end - 1], text.index("{", end)
            depth, end = 1, begin + 1
            while depth:                                    # the body
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
            if WAIT in text[begin:end]:
                found.append((f"{os.path.basename(path)}:{m.group(1)}", params, text[begin:end]))
    return found


KERNELS = _kernels()
each = pytest.mark.parametrize("name,params,body", KERNELS, ids=[k[0] for k in KERNELS])


def test_the_kernels_are_found():
    names = {k[0].split(":")[1] for k in KERNELS}
    assert {"decode_kernel", "combine_kernel", "combine_rows_kernel", "norm_rope_kernel", "append_rope_kernel",
            "append_rope_bf16_kernel", "accept_kernel", "shared_prefix_kernel", "dequant_kernel", "attend_splitk_kernel",
            "verify_ws_kernel"} <= names


@each
def test_nothing_is_read_ahead_of_the_wait(name, params, body):
    """No load, copy or prefetch of device memory stands ahead of the wait (tensor maps are kernel parameters)."""
    assert body.count(WAIT) == 1
    ahead = body[:body.index(WAIT)]
    reads = re.findall(r"__ld\w+\(|\bld\.\w*\.?global|tma_load\w*\(|bulk_load\(|load_tile\(|cp_async\w*\(|cp\.async|"
                       r"prefetch\.global|load\w*8\w*\(|\b(?:p|a|C)\.(?:pt|lens|pos|steps|q|k|v|pages|table)\b", ahead)
    assert not reads, reads


@each
def test_nothing_goes_through_the_read_only_path(name, params, body):
    """The read-only path may keep what it read before the writes of the grid before it: neither const __restrict__
    parameters nor its load instructions in such a kernel."""
    for p in params.split(","):
        assert not ("const" in p.split("*")[0] and "*" in p and "__restrict__" in p), p
    assert not re.findall(r"__ldg\(|\.nc\b", body)

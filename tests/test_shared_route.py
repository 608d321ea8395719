"""CPU check of attn_k8v4_decode_shared's choice of route, on a fake of the CUDA runtime
(fake_cudart.c, preloaded into a child process): which kernels a call launches where the
pair kernel's set-up works, fails, and works again."""
import ctypes
import json
import os
import shutil
import subprocess
import sys

import pytest

import quantized_paged_kv_q8_gb300 as k8
from quantized_paged_kv_q8_gb300 import buildlib

HERE = os.path.dirname(os.path.abspath(__file__))

CHILD = r"""
import ctypes, json, sys
lib, fake = ctypes.CDLL(sys.argv[1]), ctypes.CDLL(sys.argv[2])
fake.fake_launched.restype = ctypes.c_char_p
P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
class Cache(ctypes.Structure):
    _fields_ = [("pages", P), ("n_pages", I64), ("page_size", I32), ("n_kv_heads", I32), ("head_dim", I32), ("format", I32)]
cache = ctypes.byref(Cache(0x10000, 1 << 16, 64, 2, 256, 3))
size, call = lib.attn_k8v4_shared_workspace_bytes, lib.attn_k8v4_decode_shared
size.argtypes, size.restype = [P, I32, I32, I32], SZ
call.argtypes = [P, P, I32, P, I64, P, I32, I32, I32, ctypes.c_float, P, P, SZ, P]
def shared(ws):
    fake.fake_forget()
    rc = call(cache, 0x20000, 1, 0x30000, 1000, 0x40000, 32, 33000, 32768, 0.0625, 0x50000, 0x60000, ws, None)
    return [rc, [fake.fake_launched(i).decode() for i in range(fake.fake_launches())]]
out = []
for fails in json.loads(sys.argv[3]):
    fake.fake_fail_occupancy(fails)
    ws = size(cache, 32, 32768, 33000)
    out.append([ws, shared(ws), shared(out[0][0] if out else ws)])
print(json.dumps(out))
"""


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    k8.build()
    so = str(tmp_path_factory.mktemp("fake") / "libfake.so")
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(buildlib.nvcc()))), "include")
    cc = shutil.which("gcc") or "gcc"
    r = subprocess.run([cc, "-shared", "-fPIC", "-O1", f"-I{inc}", os.path.join(HERE, "fake_cudart.c"), "-o", so, "-ldl"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return so


def routes(fake, states):
    """Per state (0: set-up works, 1: it fails): workspace bytes, and status and kernels of a call with that
    workspace, and of one with the first state's."""
    r = subprocess.run([sys.executable, "-c", CHILD, buildlib.LIB, fake, json.dumps(states)], capture_output=True,
                       text=True, env={**os.environ, "LD_PRELOAD": fake})
    assert r.returncode == 0, r.stderr
    return json.loads(r.stdout)


def names(kernels):
    known = ("shared_prefix_kernel", "combine_rows_kernel", "combine_kernel", "decode_kernel")
    return [next(k for k in known if k in n) for n in kernels]


PAIR = ["decode_kernel", "shared_prefix_kernel", "combine_rows_kernel"]
ALONE = ["decode_kernel", "combine_kernel"]


def test_pair_route(fake):
    (ws, mine, _), = routes(fake, [0])
    assert mine[0] == k8.OK and names(mine[1]) == PAIR and ws > 0


@pytest.mark.parametrize("states", [[1], [1, 0], [0, 1], [0, 1, 0], [1, 1, 0, 0]])
def test_a_failed_set_up_takes_the_per_sequence_route_and_is_tried_again(fake, states):
    """Any workspace that the library asked for, before or after a failure, serves any later call."""
    for i, (_, mine, first) in enumerate(routes(fake, states)):
        worked = 0 in states[:i + 1]                        # that lasts
        for rc, kernels in (mine, first):
            assert rc == k8.OK
            assert names(kernels) == (PAIR if worked else ALONE)

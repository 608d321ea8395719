"""CPU checks: sizes near the ends of their types are refused on the host.  A sum or
product that wraps would pass as a small one."""
import ctypes

import pytest

import quantized_paged_kv_q8_gb300 as k8

FAKE = ctypes.c_void_p(0x20000)
MAX32, MAX64 = (1 << 31) - 1, (1 << 63) - 1


@pytest.fixture(scope="module")
def L():
    k8.build()
    return k8.lib()


def _desc(fmt=k8.FORMAT_K8V4, heads=2):
    return ctypes.byref(k8.k8v4_cache(ctypes.c_void_p(0x10000), 4, 16, heads, 256, fmt))


@pytest.mark.parametrize("fmt", [k8.FORMAT_K8V4, k8.FORMAT_INT8, k8.FORMAT_Q4])
@pytest.mark.parametrize("start,n", [(MAX64, 1), (1, MAX64), (MAX64, MAX64), (MAX64 - 15, 16), (65, 0), (64, 1), (0, 65), (1, 64)])
def test_dequant_refuses_cells_behind_the_table(L, fmt, start, n):
    """A table of four 16-cell pages has 64 cells."""
    assert L.kv_dequant_k8v4(_desc(fmt), FAKE, 4, start, n, FAKE, FAKE, None, None) == k8.EINVAL


def test_dequant_takes_the_end_of_the_table(L):
    assert L.kv_dequant_k8v4(_desc(), FAKE, 4, 64, 0, FAKE, FAKE, None, None) == k8.OK


@pytest.mark.parametrize("heads", [1, 2, 4, 8])
@pytest.mark.parametrize("n,t", [(MAX32, MAX32), (1 << 30, MAX32), (1 << 30, 1 << 30), (1 << 15, 1 << 16), (MAX32, 2)])
def test_appends_refuse_more_tokens_than_they_index(L, n, t, heads):
    """n_seqs * n_tok * heads of 2^64 and more; the mirrored append takes the same sizes."""
    d, rope = _desc(heads=heads), ctypes.byref(k8.k8v4_rope(FAKE, 64, 64, 0))
    assert L.kv_append_k8v4(d, FAKE, 4, n, FAKE, t, FAKE, FAKE, k8.BF16, None) == k8.EINVAL
    assert L.kv_append_k8v4_mirrored(d, d, FAKE, FAKE, 4, n, FAKE, t, FAKE, FAKE, k8.BF16, None) == k8.EINVAL
    assert L.kv_append_k8v4_rope(d, FAKE, 4, n, FAKE, t, FAKE, 256 * heads, FAKE, 256 * heads, k8.BF16, None, 0.0, rope,
                                 None) == k8.EINVAL
    assert L.qk_norm_rope_k8v4(FAKE, 256 * heads, heads, None, 0, 0, k8.BF16, None, None, 0.0, FAKE, n, t, rope,
                               ctypes.c_void_p(0x90000), None, None) == k8.EINVAL

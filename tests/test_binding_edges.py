"""CPU checks of the binding's handling of unusual Python arguments (CPU tensors: a
call that gets past its checks ends at "CUDA tensors expected")."""
import ctypes

import pytest
import torch

import quantized_paged_kv_q8_gb300 as k8


@pytest.fixture(scope="module", autouse=True)
def built():
    k8.build()


class NoTruth:
    def __bool__(self):
        raise KeyError("no truth value")


def test_an_argument_without_a_truth_value_raises():
    """`interleaved` as an array of two values, or as an object that raises: its own error, and no call made as if it
    were False."""
    q, pos, tab = torch.zeros(2, 3, 16, 256), torch.zeros(2, dtype=torch.int64), torch.zeros(8, 64)
    cache, kv, pt = k8.PagedCache(4, 16, device="cpu"), torch.zeros(2, 3, 2, 256), torch.zeros(2, 4, dtype=torch.int32)
    for bad, error, match in ((torch.zeros(2), RuntimeError, "[Bb]ool"), (NoTruth(), KeyError, "no truth")):
        with pytest.raises(error, match=match):
            k8.qk_norm_rope_k8v4(q, None, pos, tab, torch.empty_like(q), None, interleaved=bad)
        with pytest.raises(error, match=match):
            k8.kv_append_k8v4_rope(cache, pt, pos, kv, kv, tab, interleaved=bad)
    for fine in (0, 1, True, torch.ones(1), [1]):
        with pytest.raises(ValueError, match="CUDA tensors"):
            k8.qk_norm_rope_k8v4(q, None, pos, tab, torch.empty_like(q), None, interleaved=fine)


def test_the_descriptor_in_use_is_the_caches_own():
    """A cache whose descriptor was replaced: the calls of the extension module take the new one, as all others do (the
    old one may be gone)."""
    cache = k8.PagedCache(4, 16, device="cpu")
    old = cache.desc
    cache.desc = k8.k8v4_cache(old.pages, 4, 16, 1, 256, k8.FORMAT_INT8)
    assert cache.address == ctypes.addressof(cache.desc)
    pos, tab, pt = torch.zeros(2, dtype=torch.int64), torch.zeros(8, 64), torch.zeros(2, 4, dtype=torch.int32)
    one, two = torch.zeros(2, 3, 1, 256), torch.zeros(2, 3, 2, 256)
    with pytest.raises(ValueError, match=r"\[n_seqs, n_tok, 1, 256\]"):
        k8.kv_append_k8v4_rope(cache, pt, pos, two, two, tab)
    with pytest.raises(ValueError, match="CUDA tensors"):
        k8.kv_append_k8v4_rope(cache, pt, pos, one, one, tab)

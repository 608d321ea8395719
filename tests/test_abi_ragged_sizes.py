"""CPU checks of what the workspaces of a ragged batch's step promise: one that was made for the largest batch serves
every smaller one."""
import ctypes
import itertools

import pytest

import quantized_paged_kv_q8_gb300 as k8
from test_abi_ragged import L, _desc  # noqa: F401


@pytest.mark.parametrize("H", [1, 2, 8])
def test_a_smaller_batch_needs_no_larger_workspace(L, H):  # noqa: F811
    d = _desc(n_pages=1 << 20, page_size=64, n_kv_heads=H)
    seqs = [0, 1, 2, 7, 8, 9, 60, 63, 64, 65, 600, 65535]
    toks = [0, 1, 8, 9, 31, 32, 33, 56, 63, 64, 65, 480, 504, 512, 513, 4096, 5000, 21429, (1 << 24) - 1]
    cells = [0, 1, 127, 128, 129, 4000, 32768, 1 << 24, 2 ** 31 - 257, 2 ** 31 - 256, 2 ** 31 - 129, 2 ** 31 - 1]
    need = {a: L.attn_k8v4_diff_workspace_bytes(d, *a) for a in itertools.product(seqs, toks, cells)}
    for (s, t, c), n in need.items():
        assert n > 0
        for smaller in ((seqs[max(seqs.index(s) - 1, 0)], t, c), (s, toks[max(toks.index(t) - 1, 0)], c),
                        (s, t, cells[max(cells.index(c) - 1, 0)])):
            assert need[smaller] <= n, (smaller, (s, t, c))
    one = {a: L.attn_k8v4_diff_decode_workspace_bytes(d, *a) for a in itertools.product(seqs, cells)}
    for (s, c), n in one.items():
        assert one[seqs[max(seqs.index(s) - 1, 0)], c] <= n and one[s, cells[max(cells.index(c) - 1, 0)]] <= n

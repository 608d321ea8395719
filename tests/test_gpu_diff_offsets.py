"""attn_k8v4_diff with offsets that claim far more tokens than there are."""
import pytest
import torch

import quantized_paged_kv_q8_gb300 as k8

pytestmark = pytest.mark.gpu


def test_offsets_that_claim_more_than_32_bits_of_tiles():
    """Offsets that name the same tokens 32,768 times: their token tiles, 2^32 and 100, are counted in full, refused and
    recorded; nothing outside the call's arrays is written."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 170 << 30:
        pytest.skip("150 GB of rows and partial rows")
    n_seqs, N = 65535, 1 << 22
    T = N + 3200
    cache = k8.PagedCache(1, 16, 1)
    i32 = dict(dtype=torch.int32, device="cuda")
    off = torch.zeros(n_seqs + 1, **i32)
    off[1::2] = N
    off[-1] = T
    assert 32767 * (N // 32) + T // 32 == 2 ** 32 + 100
    q = torch.zeros(T, 8, 256, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 77.0)
    size = k8.attn_k8v4_diff_workspace_bytes(cache, n_seqs, T, 16)
    room = torch.empty(size + 4096, dtype=torch.uint8, device="cuda")
    room[size:] = 0x5a
    k8.attn_k8v4_diff(cache, q, off, torch.zeros(n_seqs, 1, **i32), torch.full((n_seqs,), 16, **i32), 16, k8.DifferentialHeads(), out,
                      room[:size])
    assert k8.k8v4_last_device_status() == k8.ERANGE
    assert (room[size:] == 0x5a).all() and all((part == 77.0).all() for part in out.split(1 << 19))
    del q, out, room
    torch.cuda.empty_cache()

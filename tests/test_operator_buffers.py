"""Scratch and error words that the caller passes to the operators around a draft block:
of the call's device, packed, large enough; anything else is refused on the host, before
a kernel could follow a pointer that is not the device's."""

from __future__ import annotations

import pytest
import torch

from block_diffusion_speculative_propose_b200 import DFlash, DFlashError, sample_tokens, \
    verify_sampled

BF = torch.bfloat16


def test_prefix_scratch_is_checked_on_the_host():
    """On CPU tensors, with a handle that has no library object: what passes the binding's
    checks ends in the library's own (no handle, nothing launched)."""
    h = DFlash.__new__(DFlash)
    h.h, h.device, h._heads, h._prefix_bytes = None, torch.device("cpu"), (4, 2, 64, 16, -1), {}
    q, o = torch.zeros(2, 4, 64, dtype=BF), torch.zeros(2, 256, dtype=torch.float16)
    seq, table = torch.zeros(1, dtype=torch.int32), torch.zeros(1, 4, dtype=torch.int32)
    kc = torch.zeros(4, 2, 16, 64, dtype=BF)
    args = (q, seq, table, 0, kc, kc)
    whole = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(DFlashError):
        h.prefix_attention(*args, o=o, workspace=whole, stream=0)
    with pytest.raises(ValueError, match="workspace"):
        h.prefix_attention(*args, o=o, workspace=whole[::2], stream=0)


@pytest.mark.gpu
def test_buffers_of_the_host_are_refused():
    dev = "cuda:0"
    x, u = torch.randn(3, 50, device=dev), torch.rand(3, device=dev)
    word = torch.zeros(1, dtype=torch.int32)
    for bad in (word, word.to(dev)[:0], torch.zeros(8, dtype=torch.uint8, device=dev)):
        with pytest.raises(ValueError, match="device_error"):
            sample_tokens(x, u, device_error=bad)
    drafts, ua = torch.zeros(1, 2, dtype=torch.int32, device=dev), torch.rand(1, 2, device=dev)
    args = (drafts, x.view(1, 3, 50), ua, u[:1])
    with pytest.raises(ValueError, match="device_error"):
        verify_sampled(*args, device_error=word)
    with pytest.raises(ValueError, match="workspace"):
        verify_sampled(*args, workspace=torch.zeros(4096, dtype=torch.uint8))
    want = verify_sampled(*args)
    # any type, counted in bytes
    got = verify_sampled(*args, workspace=torch.zeros(64, device=dev),
                         device_error=torch.zeros(1, dtype=torch.int64, device=dev))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_prefix_scratch_of_the_host_is_refused():
    from tests.test_gpu_prefix_attention import case, check, handle
    h = handle(4, 2, 64)
    q, seq, table, kc, vc = case(4, 2, 64, 1, [40, 45], 2, seed=13)
    n = h.prefix_attention_workspace_bytes(2, 1, table.shape[1], 2)
    with pytest.raises(ValueError, match="workspace"):
        h.prefix_attention(q, seq, table, 2, kc, vc, workspace=torch.zeros(n, dtype=torch.uint8))
    check(h, q, seq, table, 2, kc, vc, workspace=torch.zeros(-(-n // 4), device="cuda:0"))

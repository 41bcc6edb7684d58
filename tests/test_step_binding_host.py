"""What the binding of the expert layer holds and refuses before any CUDA call (no GPU needed)."""
import gc
import weakref

import pytest
import torch

import block_quantized_weight_matmulnbits_gb300 as mnb


def _weights(monkeypatch):
    """A descriptor of CPU tensors, as if they were on the GPU."""
    monkeypatch.setattr(mnb, "_here", lambda what, t, dev: t.data_ptr())
    packed = torch.empty(2 * mnb.mnb_packed_size(16, 32, 4, 32), dtype=torch.uint8)
    scales = torch.ones((2, 16, 1), dtype=torch.float16)
    return mnb.expert_weights(packed, scales, None, 2, 16, 32, 4, 32), weakref.ref(packed)


def test_weights_go_with_their_descriptor(monkeypatch):
    """No cycle keeps gigabytes of weights until the collector runs."""
    w, packed = _weights(monkeypatch)
    again = w
    gc.collect()
    gc.disable()
    try:
        del w
        assert packed() is not None and again.tensors[0] is packed()
        del again
        assert packed() is None
    finally:
        gc.enable()


def test_descriptor_points_to_itself(monkeypatch):
    w, _ = _weights(monkeypatch)
    assert (w.ref.contents.E, w.ref.contents.N, w.ref.contents.K) == (2, 16, 32) and w.ref.contents.packed_b == w.packed_b


def test_workspace_is_checked():
    x, logits, y = torch.ones((1, 32), dtype=torch.bfloat16), torch.ones((1, 2)), torch.ones((1, 32))
    w = mnb.ExpertWeights()
    for workspace in (torch.empty(1 << 20, dtype=torch.uint8), torch.empty((1 << 12, 512), dtype=torch.uint8)[:, :256], torch.empty(0)):
        with pytest.raises(ValueError, match="workspace"):
            mnb.mnb_moe(x, logits, w, w, w, y, 1, workspace=workspace, stream=0)

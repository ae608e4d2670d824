"""The decoder example's timed region: the host waits for nothing between the layer and its output head."""
import pytest
import torch

from int4_grouped_expert_router_gb300 import run_decoder

pytestmark = pytest.mark.gpu


def test_nothing_waits_between_the_layer_and_the_head(monkeypatch, capsys):
    layer, head = run_decoder.DecoderLayer.forward, run_decoder.Head.forward
    steps = []

    def layer_forward(self, h, new):
        out = layer(self, h, new)
        torch.cuda.set_sync_debug_mode("error")  # a copy from pageable memory or a read of a value raises from here on
        return out

    def head_forward(self, n, top=1):
        out = head(self, n, top)
        torch.cuda.set_sync_debug_mode("default")
        steps.append(n.shape[0])
        return out

    monkeypatch.setattr(run_decoder.DecoderLayer, "forward", layer_forward)
    monkeypatch.setattr(run_decoder.Head, "forward", head_forward)
    try:
        assert run_decoder.main(["--prompt", "40", "--steps", "2", "--batch", "3", "--rotary", "--vocab", "500"]) == 0
        assert run_decoder.main(["--prompt", "1", "--steps", "1", "--batch", "2", "--vocab", "500"]) == 0
    finally:
        torch.cuda.set_sync_debug_mode("default")
    assert steps == [3, 3, 3, 2, 2]

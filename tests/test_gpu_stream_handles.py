"""Streams given as handles: a call's buffers belong to the stream it runs on."""
import pytest
import torch

from transformer_xl_relative_attn_gb300 import train

pytestmark = pytest.mark.gpu


def test_buffers_belong_to_the_stream_of_a_handle():
    device = torch.device("cuda", torch.cuda.current_device())
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    for current in (torch.cuda.default_stream(), side):
        with torch.cuda.stream(current):
            for given, handle in ((0, 0), (side.cuda_stream, side.cuda_stream), (other, other.cuda_stream),
                                  (torch.cuda.default_stream(), 0), (None, current.cuda_stream)):
                with train._on(given, device):
                    assert torch.cuda.current_stream().cuda_stream == handle
            assert torch.cuda.current_stream() == current

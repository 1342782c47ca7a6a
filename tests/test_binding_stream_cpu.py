"""Which stream a call of the binding takes (no device here)."""
from types import SimpleNamespace

import pytest
import torch

import mxfp4_quantised_mixture_b200 as moe


def test_the_callers_stream_passes_through():
    assert moe._s(7) == 7 and moe._s(SimpleNamespace(cuda_stream=9)) == 9


@pytest.mark.parametrize("quick", [True, False])
def test_the_current_stream_is_found_with_and_without_the_quick_lookup(monkeypatch, quick):
    # the lookup without a Stream object is not a documented function of torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: SimpleNamespace(cuda_stream=42))
    if quick:
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 100 + dev, raising=False)
    else:
        monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    assert moe._s(None) == (103 if quick else 42)

"""Edges of the language-model operators' C entries that need no GPU."""
import pytest

import sampling_threshold_filtering_amd as stf


@pytest.mark.parametrize("B", [0, 1, 61, 1 << 22, (1 << 31) - 1])
@pytest.mark.parametrize("V", [1, 50257, 1 << 17, 1 << 24])
def test_sampling_uses_no_scratch(B, V):
    assert stf.load_library().profk_sample_tokens_scratch(B, V) == 0


def test_stream_and_device_without_torchs_fast_functions(monkeypatch):
    """Where torch lacks the private fast ones, the operators use its public ones."""
    torch = pytest.importorskip("torch")
    from sampling_threshold_filtering_amd import operators

    class Stream:
        cuda_stream = 12345

    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.delattr(torch._C, "_cuda_getDevice", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream if device == 3 else None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    for name in ("_module", "_torch", "_stream", "_device"):
        monkeypatch.setattr(operators, name, None)
    operators._native()
    assert operators._device() == 3 and operators._stream(3) == 12345

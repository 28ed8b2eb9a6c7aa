"""The device and stream that a call takes when it names none, by torch's public names too."""
import pytest
import torch

import gated_delta_rule_153_b200 as gdn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("public", [False, True])
def test_runs_on_the_current_stream(dev, monkeypatch, public):
    if public:
        monkeypatch.setattr(gdn, "_current_device", torch.cuda.current_device)
        monkeypatch.setattr(gdn, "_stream_handle", lambda index: torch.cuda.current_stream(index).cuda_stream)
    x, z = (torch.randn(64, 4, 128, device=dev) for _ in range(2))
    w = torch.ones(128, device=dev)
    want = gdn.gdn_gated_norm_fwd(x, z, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert gdn._stream_handle(dev.index) == side.cuda_stream
        got = gdn.gdn_gated_norm_fwd(x, z, w)
    torch.cuda.synchronize()
    assert gdn._current_device() == dev.index and torch.equal(got, want)

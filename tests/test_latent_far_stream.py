"""A stream of another device than the tensors' is refused by the latent attention's
entry points, before anything else is looked at.  No GPU is needed."""
import types

import pytest
import torch

import gated_delta_rule_21_gb300 as kda


class Far:
    """A tensor on device 1, as far as the checks in front look."""
    is_cuda = True

    def get_device(self):
        return 1


def test_a_stream_of_another_device_is_refused(monkeypatch):
    monkeypatch.setattr(kda, "_elsewhere", lambda s: True)
    monkeypatch.setattr(kda, "_device_now", lambda: 1)
    other = types.SimpleNamespace(device=torch.device("cuda", 0), cuda_stream=0)
    x = Far()
    for call in (lambda: kda.rotate(x, x, stream=other),
                 lambda: kda.latent_append(x, x, x, x, x, stream=other),
                 lambda: kda.latent_step(x, x, x, x, x, scale=1.0, stream=other),
                 lambda: kda.latent_fwd(x, x, x, stream=other),
                 lambda: kda.latent_bwd(x, x, x, x, x, x, stream=other)):
        with pytest.raises(ValueError, match="stream"):
            call()
    same = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    assert kda._away(x, same)
    # the current stream of another device too
    monkeypatch.setattr(kda, "_elsewhere", lambda s: False)
    with pytest.raises(ValueError, match="stream"):
        kda.rotate(x, x, stream=other)
    assert not kda._away(x, same)

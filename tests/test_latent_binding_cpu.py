"""What the binding of the latent cache's calls hands to the C call, and what it refuses: a recording library stands in
for libdsa.so, host tensors for device tensors."""
import pytest
import torch

import sparse_attention_decode_lightning_b200 as dsa

INT_MAX = 2 ** 31 - 1


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def calls(monkeypatch):
    rec = Recorder()
    monkeypatch.setattr(dsa, "_lib", rec)
    monkeypatch.setattr(dsa, "_device_of", lambda t: t.get_device())       # -1 for all of them
    monkeypatch.setattr(dsa, "_raw_stream", lambda stream, dev: 0)
    return rec.calls


def sinks_args(**over):
    t = torch.zeros
    a = dict(q=t(2, 128, 576, dtype=torch.bfloat16), kv_pool=t(4, 64, 576, dtype=torch.uint8),
             page_table=t(1, 4, dtype=torch.int32), q_offsets=t(2, dtype=torch.int32), q_vis=t(2, dtype=torch.int32), B=1,
             sinks=0, window=5, scale=1.0, out=t(2, 128, 512, dtype=torch.bfloat16), lse=t(2, 128),
             ws=t(256, dtype=torch.uint8), kv_scales=t(4, 4))
    a.update(over)
    return a


@pytest.mark.parametrize("given,handed", [(0, 0), (5, 5), (INT_MAX, INT_MAX), (INT_MAX + 1, INT_MAX), (1 << 32, INT_MAX),
                                          (1 << 40, INT_MAX), ((1 << 63) - 1, INT_MAX), (10 ** 30, INT_MAX)])
@pytest.mark.parametrize("name", ["sinks", "window"])
def test_counts_beyond_the_c_int_stay_large(calls, name, given, handed):
    """A window of 2^40 asks for dense attention; its lower 32 bits would ask for none."""
    dsa.dsa_mla_decode_sinks(**sinks_args(**{name: given}))
    (fn, args), = calls
    assert fn == "dsa_mla_decode_sinks"
    assert args[13 if name == "sinks" else 14] == handed


@pytest.mark.parametrize("name", ["sinks", "window"])
@pytest.mark.parametrize("bad,error", [(-1, ValueError), (-(1 << 32), ValueError), (-(1 << 63), ValueError),
                                       (3.0, TypeError), (None, TypeError)])
def test_negative_and_fractional_counts_are_refused(calls, name, bad, error):
    with pytest.raises(error):
        dsa.dsa_mla_decode_sinks(**sinks_args(**{name: bad}))
    assert not calls

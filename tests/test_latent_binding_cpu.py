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


def block_args(**over):
    a = sinks_args(idx=torch.zeros(2, 9, dtype=torch.int32))
    del a["sinks"], a["window"]
    a.update(over)
    return a


def append_args(**over):
    t = torch.zeros
    x = t(3, 576, dtype=torch.bfloat16)
    a = dict(kv=x[:, :512], k_pe=x[:, 512:], inv_freq=t(32), kv_pool=t(4, 64, 576, dtype=torch.uint8),
             page_table=t(1, 4, dtype=torch.int32), q_offsets=t(2, dtype=torch.int32), q_vis=t(3, dtype=torch.int32), B=1,
             ws=t(256, dtype=torch.uint8), kv_scales=t(4, 4))
    a.update(over)
    return a


CALLS = {"dsa_mla_decode_sinks": sinks_args, "dsa_sparse_mla_decode_fp8_block": block_args, "dsa_latent_append": append_args}


@pytest.mark.parametrize("name", CALLS)
def test_right_arguments_reach_the_call(calls, name):
    """Of each type that the cache may have."""
    getattr(dsa, name)(**CALLS[name]())
    getattr(dsa, name)(**CALLS[name](kv_pool=torch.zeros(4, 64, 576, dtype=torch.uint8).view(torch.float8_e4m3fn)))
    if name != "dsa_sparse_mla_decode_fp8_block":
        getattr(dsa, name)(**CALLS[name](kv_pool=torch.zeros(4, 64, 576, dtype=torch.bfloat16), kv_scales=None))
    assert {n for n, _ in calls} == {name} and len(calls) == (2 if name == "dsa_sparse_mla_decode_fp8_block" else 3)


def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


I32, BF16, U8 = torch.int32, torch.bfloat16, torch.uint8
CACHE = [("kv_pool", z(4, 64, 576, dtype=BF16)), ("kv_pool", z(4, 576, dtype=U8)), ("kv_pool", z(4, 64, 512, dtype=U8)),
         ("kv_pool", z(4, 64, 1152, dtype=U8)[:, :, ::2]), ("kv_scales", z(4, 5)), ("kv_scales", z(3, 4)), ("kv_scales", z(4)),
         ("kv_scales", z(4, 4, dtype=torch.float64)), ("kv_scales", z(4, 8)[:, ::2]), ("page_table", z(2, 4, dtype=I32)),
         ("page_table", z(1, 4, dtype=torch.int64)), ("page_table", z(4, dtype=I32)), ("q_offsets", z(3, dtype=I32)),
         ("q_offsets", z(2, dtype=torch.int64)), ("q_vis", z(1, dtype=I32)), ("q_vis", z(9, dtype=torch.int64))]
ATTEND = CACHE + [("q", z(2, 128, 576)), ("q", z(2, 128, 512, dtype=BF16)), ("q", z(2, 73728, dtype=BF16)),
                  ("q", z(2, 576, 128, dtype=BF16).transpose(1, 2)), ("out", z(2, 128, 512)),
                  ("out", z(2, 64, 512, dtype=BF16)), ("lse", z(2, 64)), ("lse", z(2, 128, dtype=BF16)),
                  ("ws", z(16, 16, dtype=U8).t())]
WRONG = {
    "dsa_mla_decode_sinks": ATTEND,
    "dsa_sparse_mla_decode_fp8_block": ATTEND + [("idx", z(2, 9)), ("idx", z(3, 9, dtype=I32)), ("idx", z(2, dtype=I32)),
                                                 ("kv_scales", None)],
    "dsa_latent_append": CACHE + [("kv", z(3, 512)), ("kv", z(3, 500, dtype=BF16)), ("kv", z(512, 3, dtype=BF16).t()),
                                  ("kv", z(1536, dtype=BF16)), ("k_pe", z(2, 64, dtype=BF16)), ("k_pe", z(3, 64)),
                                  ("k_pe", z(3, 32, dtype=BF16)), ("inv_freq", z(64)), ("inv_freq", z(32, dtype=BF16)),
                                  ("ws", z(16, 16, dtype=U8).t())],
}


@pytest.mark.parametrize("name,arg,value", [(n, a, v) for n, l in WRONG.items() for a, v in l])
def test_a_wrong_argument_is_refused_by_its_name(calls, name, arg, value):
    with pytest.raises(ValueError, match=rf"\b{arg}:"):
        getattr(dsa, name)(**CALLS[name](**{arg: value}))
    assert not calls

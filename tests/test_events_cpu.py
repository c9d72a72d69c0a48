"""Calls that are timed with events, without a GPU: the library gets the events'
handles, so a prepared call has to keep the events alive."""
import gc
import weakref

import torch

import offloaded_kv_decode_gb300 as clo
from offloaded_kv_decode_gb300 import kv4


class Event:
    def __init__(self, handle):
        self.cuda_event = handle


class Tensor(torch.Tensor):
    """A host tensor that says it is on the GPU: nothing is launched here."""

    @property
    def is_cuda(self):
        return True


def gpu(*shape, dtype=torch.float16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Tensor)


def test_options_hold_their_events():
    events = [Event(16), Event(32)]
    refs = [weakref.ref(e) for e in events]
    opts = clo._opts(0, events)
    assert (opts.ev_begin, opts.ev_end) == (16, 32)
    del events
    gc.collect()
    assert all(r() is not None for r in refs)
    del opts
    gc.collect()
    assert all(r() is None for r in refs)


def test_marshalled_calls_hold_their_events(monkeypatch):
    """What a prepared call keeps: its arguments (a reference into the options, or
    a struct with their address) and the tuple of what is behind them."""
    monkeypatch.setattr(kv4, "_device_of", lambda *tensors: 0)
    i32 = torch.int32
    q, pool = gpu(2, 1, 8, 128), gpu(4, 2, 2304, dtype=torch.uint8)
    events = [Event(16), Event(32)]
    refs = [weakref.ref(e) for e in events]
    call, _ = kv4._attn_call(q, pool, gpu(2, 3, dtype=i32), gpu(2, dtype=i32), gpu(2, 1, 8, 128),
                             gpu(64, dtype=torch.uint8), None, None, None, 0, events)
    del events
    gc.collect()
    assert all(r() is not None for r in refs)
    del call
    gc.collect()
    assert all(r() is None for r in refs)

"""What a call allocates itself comes from the pool of the stream that the call runs on.  No GPU is needed: the library,
the pointers and torch's stream context are stand-ins that record which stream was current at each allocation."""
import contextlib
import types

import pytest
import torch

HANDLE = 0x5000


class Recorder:
    def __init__(self):
        self.current, self.allocated = None, []

    @contextlib.contextmanager
    def stream(self, s):
        before, self.current = self.current, s
        yield
        self.current = before


class Stream:
    cuda_stream = HANDLE


MINE = Stream()  # stands for a torch stream, which is entered as it is


class Host:
    """A pinned host tensor, as far as the binding looks."""
    is_cuda = False

    def is_pinned(self):
        return True

    def data_ptr(self):
        return 0


class Library:
    def __getattr__(self, name):
        def call(*args):
            return 0
        call.__name__ = name
        return call


@pytest.fixture
def rec(xkv, monkeypatch):
    r = Recorder()

    def empty(*args, **kw):
        r.allocated.append(r.current)
        return torch.zeros(64, dtype=torch.uint8)

    monkeypatch.setattr(xkv, "lib", Library())
    monkeypatch.setattr(xkv, "torch", types.SimpleNamespace(**{**vars(torch), "empty": empty}))
    monkeypatch.setattr(xkv, "_ptr", lambda t: None)
    monkeypatch.setattr(xkv, "_addr", lambda t: None)
    monkeypatch.setattr(torch.cuda, "stream", r.stream)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=0))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    return r


def _calls(xkv):
    t, bf = torch.zeros((4, 4)), torch.zeros((4, 4), dtype=torch.bfloat16)
    sr = xkv.sr_params(1, 1, 1, 4, 4, 4, 4, 1, 1, 0, 0, 1.0, torch.bfloat16)
    app = xkv.append_params(1, 1, 1, 4, 1, 0, 0, 1.0, torch.bfloat16, 4, 4, 4, 0, 0, 0, 0, 0, 0)
    kv8 = types.SimpleNamespace(sizes=(1, 1, 16, 16, 8), index=-1, pointers=None)
    q, lens = torch.zeros((1, 2, 16)), torch.zeros(1, dtype=torch.int32)
    return {
        "gram": lambda s: xkv.xkv_gram_accumulate([bf], t, stream=s),
        "compress": lambda s: xkv.xkv_compress_group([bf], 4, bf, bf, stream=s),
        "factor": lambda s: xkv.xkv_factor_gram(t, 1, 4, 4, 4, bf, stream=s),
        "project": lambda s: xkv.xkv_project([bf], t, types.SimpleNamespace(
            shape=(4, 4), stride=lambda i: 1, is_cuda=True, data_ptr=lambda: 0), stream=s),
        "sr": lambda s: xkv.xkv_sr_attention_decode(sr, t, t, t, t, t, t, t, t, t, stream=s),
        "xk_sr": lambda s: xkv.xkv_xk_sr_attention_decode(sr, t, t, t, t, t, t, t, t, stream=s),
        "xk_sr_host": lambda s: xkv.xkv_xk_sr_attention_decode_host_values(sr, t, t, t, Host(), t, t, t, t, stream=s),
        "partial": lambda s: xkv.xkv_sr_attention_partial(sr, xkv.ShardParams(), t, t, t, t, t, t, t, t, t, t, stream=s),
        "dense": lambda s: xkv.xkv_dense_attention_decode(xkv.dense_params(1, 1, 1, 4, 4, torch.bfloat16), t, t, t, t, stream=s),
        "append": lambda s: xkv.xkv_sr_append(app, [t], [t], [t], [t], t, t, t, t, [t], stream=s),
        "kv8": lambda s: xkv.xkv_kv8_attention_decode(xkv.kv8_params(1, 1, 16, 8, 16), kv8, lens, q, q, stream=s),
        "ner": lambda s: xkv.xkv_ner(t, 2, t, stream=s),
        "energy_rank": lambda s: xkv.xkv_energy_rank(t, 2, stream=s),
    }


NAMES = ("gram", "compress", "factor", "project", "sr", "xk_sr", "xk_sr_host", "partial", "dense", "append", "kv8", "ner",
         "energy_rank")


@pytest.mark.parametrize("name", NAMES)
def test_own_allocations_belong_to_the_launch_stream(xkv, rec, name):
    call = _calls(xkv)[name]
    for given, pool in ((None, None), (HANDLE, ("external", HANDLE)), (0, "default"), (1, "default"),
                        (types.SimpleNamespace(cuda_stream=HANDLE), ("external", HANDLE)), (MINE, MINE)):
        rec.allocated.clear()
        call(given)
        assert rec.allocated and all(p == pool for p in rec.allocated), (given, rec.allocated)

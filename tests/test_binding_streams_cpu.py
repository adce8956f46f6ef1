"""What a call on another stream allocates itself is that stream's memory: the
workspace it zeroes and frees, and the outputs it returns."""
import contextlib
import types

import pytest
import torch

from mla_latent_kv_05_gb300 import binding
from tests.test_binding_cpu import FakeLib, FakeTensor
from tests.test_operators_cpu import Rows

SIDE, CURRENT = 0x77, 0x11


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Made(FakeTensor):
    users = ()

    def record_stream(self, s):
        self.users += (s.cuda_stream,)


@pytest.fixture
def made(monkeypatch):
    """The tensors that calls allocate, each with the stream it was made on."""
    now, out = [Stream(CURRENT)], []

    @contextlib.contextmanager
    def on(s):
        now.append(s)
        yield
        now.pop()

    def make(shape, **kw):
        t = Made(shape if isinstance(shape, tuple) else (shape,))
        t.made_on = now[-1].cuda_stream
        out.append(t)
        return t

    monkeypatch.setattr(binding, "load", lambda *a, **k: FakeLib())
    monkeypatch.setattr(binding, "_check", lambda *a, **k: None)
    monkeypatch.setattr(binding, "_check_rows", lambda *a, **k: None)
    fake = types.SimpleNamespace(**{n: getattr(torch, n) for n in ("bfloat16", "float32", "int32", "uint8", "Tensor")},
                                 empty=make, zeros=make,
                                 cuda=types.SimpleNamespace(current_device=lambda: 0, current_stream=lambda: now[-1],
                                                            stream=on, Stream=Stream, ExternalStream=Stream))
    monkeypatch.setattr(binding, "torch", fake)
    monkeypatch.setattr(binding, "_raw_stream", lambda d: now[-1].cuda_stream)
    return out


def calls():
    B, T, H = 3, 2, 128
    q, qr = FakeTensor((B, T, H, 512)), FakeTensor((B, T, H, 64))
    table, lens, cu, par = FakeTensor((B, 5)), FakeTensor((B,)), FakeTensor((B + 1,)), FakeTensor((B, T))

    def cache(width):
        return FakeTensor((9, 64, width))

    x, kr, w = Rows((7, 512)), Rows((7, 64)), FakeTensor((128, 128, 512))
    pq, pqr, pk = Rows((7, 128, 128)), Rows((7, 128, 64)), Rows((7, 128, 128))
    yield "decode", 3, lambda **k: binding.mla_decode_bf16(q, qr, cache(576), table, lens, 0.1, **k)
    yield "noalloc", 2, lambda **k: binding.mla_decode_bf16_noalloc(q, qr, cache(576), table, lens, 0.1, **k)
    yield "sparse", 3, lambda **k: binding.mla_decode_sparse_bf16(q, qr, cache(576), FakeTensor((B, T, 4)), 0.1, **k)
    yield "wuv", 2, lambda **k: binding.mla_up_project_wuv(FakeTensor((6, 128, 512)), w, **k)
    yield "append", 1, lambda **k: binding.mla_cache_append_fp8(x, kr, cache(594), table, lens, cu, **k)
    yield "gather", 2, lambda **k: binding.mla_cache_gather_fp8(cache(594), table, lens, cu, 7, **k)
    yield "tree", 3, lambda **k: binding.mla_decode_tree_fp8(q, qr, cache(594), table, lens, par, 0.1, **k)
    yield "expand", 3, lambda **k: binding.mla_expand_kv(x, w, w, **k)
    yield "prefill", 3, lambda **k: binding.mla_prefill_bf16(pq, pqr, pk, kr, pk, cu, cu, 0.1, **k)
    yield "merge", 2, lambda **k: binding.mla_combine_splits(FakeTensor((7, 128, 512)), FakeTensor((7, 128)), cu, **k)


@pytest.mark.parametrize("name,count,call", list(calls()), ids=[c[0] for c in calls()])
def test_a_call_allocates_on_its_own_stream(made, name, count, call):
    call(stream=Stream(SIDE))
    assert len(made) == count
    assert [t.made_on for t in made] == [SIDE] * count
    assert [t.users for t in made] == [(CURRENT,)] * count     # who may use an output after the call
    made.clear()
    call()
    call(stream=Stream(CURRENT))
    assert [t.made_on for t in made] == [CURRENT] * 2 * count and not any(t.users for t in made)

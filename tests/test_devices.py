"""Calls on tensors of a device that is not the current one enqueue with that
device current and on its stream.  On the CPU: host tensors that say they are
on device 1, a library that records where it was called; nothing is launched."""
import contextlib

import pytest
import torch

import ternary_weight_only_amd as tq
from ternary_weight_only_amd import binding
from tests import ffn_reference as ref


class OnOne(torch.Tensor):
    device = property(lambda self: torch.device("cuda", 1))
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 1


def one(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnOne)


@pytest.fixture
def calls(monkeypatch):
    """(function, current device, stream) of every call of the library; the
    default streams of the devices are 100 and 101 here."""
    made, current = [], [0]

    class Library:
        def __getattr__(self, name):
            if "bytes" in name or "workspace" in name:
                return getattr(real, name)

            def call(*args):
                made.append((name, current[0], args[-1]))
                return 0
            return call

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], torch.device(d).index
        yield
        current[0] = before

    real = binding.lib()
    monkeypatch.setattr(binding, "lib", lambda: library)
    monkeypatch.setattr(binding, "_current_device", lambda: current[0], raising=False)
    monkeypatch.setattr(binding, "_stream", lambda: 100 + current[0])
    monkeypatch.setattr(binding, "_stream_of", lambda d: 100 + d.index)
    monkeypatch.setattr(torch.cuda, "device", device)
    library = Library()
    return made


M, N, K, G, R = 4, 8, 128, 64, 8


def _packed():
    p, s = ref.packed_weight(1, N, K, G)
    return p.as_subclass(OnOne), s.as_subclass(OnOne)


def test_new_calls(calls):
    x, w, mn, pair = one(M, K), one(N, K), one(M, N), _packed()
    ws = one(tq.glu_backward_workspace(M, N, K) + (1 << 20), dtype=torch.uint8)
    tq.glu(x, pair, pair, N, K, G, out=one(M, N), workspace=ws)
    tq.lora_matmul(x, *pair, one(M, dtype=torch.int32), one(2, R, K), one(2, N, R), one(2, dtype=torch.float32),
                   N, K, G, out=one(M, N, dtype=torch.float32), workspace=ws)
    tq.glu_forward(x, w, w, out=(mn, mn, mn))
    tq.glu_backward(mn, x, w, w, mn, mn, out=(one(M, K), one(N, K), one(N, K)), workspace=ws)
    assert calls == [(f, 1, 101) for f in ("tq_glu", "tq_lora_matmul", "tq_glu_forward", "tq_glu_backward")]


def test_calls_of_one_and_of_many(calls):
    x, pair = one(M, K), _packed()
    y = one(M, N, dtype=torch.float32)
    tq.quantize_pack(one(N, K), G, out=pair)
    tq.gemv(x, *pair, N, K, G, out=y)
    tq.gemm(x=x, packed=pair[0], scales=pair[1], N=N, K=K, G=G, out=y)
    tq.gemm_batched([x], [pair[0]], [pair[1]], N, K, G, outs=[y])
    tq.dequantize(*pair, N, K, G, out=one(N, K))
    assert [c[1:] for c in calls] == [(1, 101)] * 5


def test_lists_of_none(calls):
    assert tq.gemm_batched([], [], [], N, K, G) == [] and tq.unpack_batched([], N, K, G) == [] and calls == []

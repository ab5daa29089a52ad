"""Buffers that a call makes for itself belong to the stream that its kernels run on, whichever stream is
current; results are known to the current one too.  On the CPU: tensors that say they are on the GPU, streams that
are numbers, and calls into the library that only note their arguments."""

import contextlib

import pytest
import torch

from ternary_bit_quantized_amd import q2_0 as B

CURRENT, OTHER = 7, 99


class OnGpu(torch.Tensor):
    made, known = [], []       # (address, the stream that was current when it was made); (address, stream)
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0

    def new_empty(self, *a, **kw):
        t = super().new_empty(*a, **kw)
        OnGpu.made.append((t.data_ptr(), torch.cuda.current_stream().cuda_stream))
        return t

    def record_stream(self, stream):
        OnGpu.known.append((self.data_ptr(), stream.cuda_stream))


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream, self.device_index = handle, 0


def gpu(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


@pytest.fixture
def fakes(monkeypatch):
    now = [CURRENT]
    empty = torch.empty

    @contextlib.contextmanager
    def on(stream):
        now[0], before = stream.cuda_stream, now[0]
        yield
        now[0] = before

    def logged_empty(*a, **kw):
        t = empty(*a, **kw).as_subclass(OnGpu)
        OnGpu.made.append((t.data_ptr(), now[0]))
        return t

    monkeypatch.setattr(torch, "empty", logged_empty)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: FakeStream(now[0]))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", FakeStream)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: now[0], raising=False)
    launched = []
    for name in [n for n in dir(B) if n.endswith("_raw")]:
        monkeypatch.setattr(B, name, lambda *a, **kw: launched.append(a) or 0)
    OnGpu.made.clear()
    OnGpu.known.clear()
    return launched


def w(rows, k):
    return gpu(rows, k // 64 * 18, dtype=torch.uint8)


def int32(*shape):
    return gpu(*shape, dtype=torch.int32)


def cache():
    return gpu(40, 2, 16, 64, dtype=torch.float16)


CALLS = {
    "get_rows": lambda s: B.q2_0_get_rows(w(4, 64), 4, 64, int32(3), stream=s),
    "quantize": lambda s: B.q2_0_quantize(gpu(4, 64), stream=s),
    "repack": lambda s: B.q2_0_repack_g128(gpu(4, 34, dtype=torch.uint8), 4, 128, stream=s),
    "mat_vec": lambda s: B.q2_0_mul_mat_vec(w(16, 64), 16, 64, gpu(2, 64), stream=s),
    "mat_vec_group": lambda s: B.q2_0_mul_mat_vec_group([(w(16, 64), 16), (w(8, 64), 8)], 64, gpu(2, 64), stream=s),
    "mat_vec_batch": lambda s: B.q2_0_mul_mat_vec_batch([(w(16, 64), 16, 64, gpu(2, 64))], stream=s),
    "mul_mat": lambda s: B.q2_0_mul_mat(w(128, 256), 128, 256, gpu(64, 256), stream=s),
    "mul_mat_group": lambda s: B.q2_0_mul_mat_group([(w(128, 256), 128)], 256, gpu(64, 256), stream=s),
    "mul_mat_id": lambda s: B.q2_0_mul_mat_id(w(256, 64), 2, 128, 64, gpu(6, 64), int32(6, 2), stream=s),
    "kv_append": lambda s: B.q2_0_kv_append(cache(), cache(), int32(2, 20), int32(3), int32(3), gpu(3, 128), gpu(3, 128),
                                            q=gpu(3, 256), stream=s),
    "attn_shared": lambda s: B.q2_0_attn_shared(gpu(2, 256, dtype=torch.float16), cache(), cache(), int32(2, 200), int32(2),
                                                0.125, prefix_len=2000, stream=s),
    "moe_route": lambda s: B.q2_0_moe_route(gpu(5, 16), 2, stream=s),
    "moe_layer": lambda s: B.q2_0_moe_layer(w(4 * 128, 192), w(4 * 128, 192), w(4 * 192, 128), 4, 128, 192, gpu(3, 192),
                                            int32(3, 2), gpu(3, 2), stream=s),
}


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("stream", [FakeStream(OTHER), OTHER])
def test_buffers_are_the_given_streams(name, stream, fakes):
    result = CALLS[name](stream)
    assert OnGpu.made and all(at == OTHER for _, at in OnGpu.made), OnGpu.made
    assert len(fakes) == 1 and OTHER in fakes[0]                    # the launch goes there
    for t in result if isinstance(result, (list, tuple)) else [result]:
        assert (t.data_ptr(), CURRENT) in OnGpu.known


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("stream", [None, FakeStream(CURRENT), CURRENT])
def test_buffers_of_the_current_stream(name, stream, fakes):
    CALLS[name](stream)
    assert OnGpu.made and all(at == CURRENT for _, at in OnGpu.made)
    assert CURRENT in fakes[0] and not OnGpu.known


def test_what_these_calls_reach():
    """The attention, the expert layer and the GEMM of the calls above do need a workspace."""
    assert B.attn_shared_workspace_bytes(2, 4, 2, 64, 1, 2000, 3200) > 0
    assert B.moe_layer_workspace_bytes(128, 192, 2, 3) > 0
    assert B.mul_mat_workspace_bytes(128, 256, 64, B.Q2_0_PREC_F16_MFMA) > 0

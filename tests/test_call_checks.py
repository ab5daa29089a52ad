"""What the decoder operators' Python calls refuse: tensors that are not on the current device (those of another GPU
too), workspaces that are not or are not memory of their own length, tensors of the wrong rank.  On the CPU,
with tensors that say where they are and calls into the library that only note their arguments."""

import pytest
import torch
from test_call_streams import FakeStream, OnGpu, cache, fakes, gpu, int32, w  # noqa: F401

from ternary_bit_quantized_amd import q2_0 as B


class OnSecondGpu(OnGpu):
    def get_device(self):
        return 1


def arguments(name):
    """(call, its tensor arguments by name, the others)"""
    half = dict(dtype=torch.float16)
    if name == "kv_append":
        return B.q2_0_kv_append, dict(k_cache=cache(), v_cache=cache(), table=int32(2, 20), seq=int32(3), pos=int32(3),
                                      k=gpu(3, 128), v=gpu(3, 128), rope=gpu(50, 64), q=gpu(3, 256), q_out=gpu(3, 256, **half)), {}
    if name == "attn_shared":
        return B.q2_0_attn_shared, dict(q=gpu(2, 256, **half), k_cache=cache(), v_cache=cache(), table=int32(2, 200),
                                        lens=int32(2), out=gpu(2, 256, **half), workspace=gpu(1 << 22)), \
            dict(scale=0.125, prefix_len=2000)
    if name == "moe_route":
        return B.q2_0_moe_route, dict(logits=gpu(5, 16), ids=int32(5, 2), weights=gpu(5, 2)), dict(n_used=2)
    return B.q2_0_moe_layer, dict(w_gate=w(4 * 128, 192), w_up=w(4 * 128, 192), w_down=w(4 * 192, 128), x=gpu(3, 192),
                                  ids=int32(3, 2), weights=gpu(3, 2), y=gpu(3, 192), workspace=gpu(1 << 20)), \
        dict(n_expert=4, n_ff=128, K=192)


@pytest.mark.parametrize("name", ["kv_append", "attn_shared", "moe_route", "moe_layer"])
def test_tensors_elsewhere_are_refused(name, fakes):  # noqa: F811
    call, tensors, others = arguments(name)
    call(**tensors, **others)
    assert len(fakes) == 1
    for arg, t in tensors.items():
        for there in (t.as_subclass(OnSecondGpu), t.as_subclass(torch.Tensor)):
            with pytest.raises(ValueError):
                call(**dict(tensors, **{arg: there}), **others)
    with pytest.raises(ValueError):
        stream = FakeStream(5)
        stream.device_index = 1
        call(**tensors, **others, stream=stream)
    assert len(fakes) == 1


@pytest.mark.parametrize("name", ["kv_append", "attn_shared", "moe_route", "moe_layer"])
def test_ranks_and_workspaces(name, fakes):  # noqa: F811
    call, tensors, others = arguments(name)
    for arg, t in tensors.items():
        if arg == "workspace":
            with pytest.raises(ValueError):     # as many elements, but not as much memory
                call(**dict(tensors, workspace=gpu(1).expand(t.numel())), **others)
        elif arg[:2] != "w_":                   # (weights are counted in bytes, of any shape)
            with pytest.raises(ValueError):
                call(**dict(tensors, **{arg: t.reshape(1, *t.shape)}), **others)
            with pytest.raises(ValueError):
                call(**dict(tensors, **{arg: t.reshape(-1)[:1].reshape(())}), **others)
    if "k_cache" in tensors:
        empty = gpu(40, 2, 16, 0, dtype=torch.float16)
        with pytest.raises(ValueError):
            call(**dict(tensors, k_cache=empty, v_cache=empty), **others)
    assert not fakes

"""The Python calls of the operators between two decoder steps: buffers that they make belong to the stream they launch
on, and tensors elsewhere, of other types, ranks or shapes are refused.  On the CPU, with tensors that say where they are
and calls into the library that only note their arguments."""

import pytest
import torch
from test_call_checks import OnSecondGpu
from test_call_streams import CURRENT, OTHER, FakeStream, OnGpu, cache, fakes, gpu, int32  # noqa: F401

from ternary_bit_quantized_amd import q2_0 as B


def arguments(name):
    """(call, its tensor arguments by name, the others)"""
    pools = dict(k_cache=cache(), v_cache=cache(), ref=int32(40), free=int32(2))
    if name == "route":
        return B.q2_0_moe_route_groups, dict(logits=gpu(5, 16), bias=gpu(16), ids=int32(5, 2), weights=gpu(5, 2)), \
            dict(n_used=2, n_group=4, n_group_used=2)
    if name == "verify":
        return B.q2_0_draft_verify, dict(target=gpu(6, 50), draft=gpu(4, 50), tokens=int32(2, 2), n_draft=int32(2), u=gpu(2, 3),
                                         temperature=gpu(2), out=int32(2, 3), n_accepted=int32(2), workspace=gpu(1 << 16)), {}
    if name == "copy":
        return B.q2_0_kv_copy, dict(k_to=cache(), v_to=cache(), k_from=cache(), v_from=cache(), src=int32(3), dst=int32(3)), {}
    if name == "fork":
        return B.q2_0_kv_fork, dict(ref=int32(40), table=int32(3, 6), lens=int32(3), src=int32(2), dst=int32(2),
                                    workspace=gpu(1 << 10)), dict(page_size=16)
    if name == "resize":
        return B.q2_0_kv_resize, dict(**pools, table=int32(3, 6), lens=int32(3), new_lens=int32(3), missing=int32(1),
                                      workspace=gpu(1 << 10)), {}
    return B.q2_0_kv_compact, dict(k_to=cache(), v_to=cache(), ref_to=int32(40), free_to=int32(2), table_to=int32(3, 6),
                                   k_from=cache(), v_from=cache(), ref=int32(40), free=int32(2), table=int32(3, 6),
                                   lens=int32(3), n_used=int32(1), workspace=gpu(1 << 10)), {}


NAMES = ["route", "verify", "copy", "fork", "resize", "compact"]
MADE = {"route": ("ids", "weights"), "verify": ("out", "n_accepted"), "resize": ("missing",), "compact": ("n_used",)}


@pytest.mark.parametrize("name", NAMES)
def test_what_is_refused(name, fakes):  # noqa: F811
    call, tensors, others = arguments(name)
    call(**tensors, **others)
    assert len(fakes) == 1
    with pytest.raises(ValueError):
        stream = FakeStream(5)
        stream.device_index = 1
        call(**tensors, **others, stream=stream)
    for arg, t in tensors.items():
        bad = [t.as_subclass(OnSecondGpu), t.as_subclass(torch.Tensor)]
        if arg == "workspace":
            bad.append(gpu(1).expand(t.numel()))        # as many elements, but not as much memory
        else:
            bad += [t.reshape(1, *t.shape), t.reshape(-1)[:1].reshape(()), t.double() if t.is_floating_point() else t.long()]
            if t.shape[-1] > 1:                         # every other element of a larger tensor
                bad.append(t.repeat_interleave(2, dim=-1)[..., ::2])
            if arg not in ("target", "logits", "tokens", "table", "src", "ref", "k_from", "v_from", "k_to", "v_to",
                           "k_cache", "v_cache"):       # (sizes that others go by)
                bad.append(torch.cat([t, t]).as_subclass(OnGpu))
        for there in bad:
            with pytest.raises(ValueError):
                call(**dict(tensors, **{arg: there}), **others)
    assert len(fakes) == 1


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("stream", [None, FakeStream(CURRENT), FakeStream(OTHER), OTHER])
def test_own_buffers(name, stream, fakes):  # noqa: F811
    call, tensors, others = arguments(name)
    made = MADE.get(name, ())
    given = {k: t for k, t in tensors.items() if k not in made and k != "workspace"}
    OnGpu.made.clear()
    result = call(**given, **others, stream=stream)
    on = OTHER if stream == OTHER or getattr(stream, "cuda_stream", None) == OTHER else CURRENT
    assert len(OnGpu.made) == len(made) + (name not in ("route", "copy"))     # (those have no workspace)
    assert all(at == on for _, at in OnGpu.made) and len(fakes) == 1 and on in fakes[0]
    for t in result if isinstance(result, tuple) else [result] if result is not None else []:
        assert on == CURRENT or (t.data_ptr(), CURRENT) in OnGpu.known


def test_types_that_differ(fakes):  # noqa: F811
    call, t, others = arguments("verify")
    with pytest.raises(ValueError):
        call(**dict(t, draft=t["draft"].half()))
    with pytest.raises(ValueError):
        call(**dict(t, draft=gpu(4, 51)))
    call, t, _ = arguments("copy")
    with pytest.raises(ValueError):
        call(**dict(t, v_to=t["v_to"].bfloat16()))
    call, t, _ = arguments("compact")
    with pytest.raises(ValueError):
        call(**dict(t, table_to=int32(3, 7)))
    assert not fakes


def test_no_sequences(fakes):  # noqa: F811
    """Nothing is missing where there is nothing to grow, though no kernel writes it."""
    call, t, _ = arguments("resize")
    assert call(**dict(t, table=int32(0, 6), lens=int32(0), new_lens=int32(0), missing=None)).item() == 0


def test_a_new_pool():
    ref, free = B.q2_0_kv_pages(70, device="cpu")
    assert ref.dtype == free.dtype == torch.int32 and ref.tolist() == [0] * 70 and free.tolist() == [-1] * 3


@pytest.mark.parametrize("stream", [None, FakeStream(CURRENT), FakeStream(OTHER), OTHER])
@pytest.mark.parametrize("given", [False, True])
def test_no_sequences_on_a_stream(stream, given, fakes, monkeypatch):  # noqa: F811
    """What is missing is written on the call's stream, where its reader waits for it."""
    written = []
    zero = torch.Tensor.zero_

    def noted(t):
        written.append(torch.cuda.current_stream().cuda_stream)
        return zero(t)

    monkeypatch.setattr(OnGpu, "zero_", noted, raising=False)
    call, t, _ = arguments("resize")
    missing = torch.ones_like(t["missing"]).as_subclass(OnGpu) if given else None
    got = call(**dict(t, table=int32(0, 6), lens=int32(0), new_lens=int32(0), missing=missing), stream=stream)
    assert got.item() == 0 and (got is missing or not given) and not fakes
    assert written == [OTHER if stream == OTHER or getattr(stream, "cuda_stream", None) == OTHER else CURRENT]
    with pytest.raises(ValueError):
        other = FakeStream(5)
        other.device_index = 1
        call(**dict(t, table=int32(0, 6), lens=int32(0), new_lens=int32(0), missing=missing), stream=other)

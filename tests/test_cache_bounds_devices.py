"""Host tensors, and tensors of another device, are refused by the calls that bound a cache,
whichever argument they are.  The C calls are stand-ins that only count: nothing is launched, and
a tensor's device is what its class says, so that this runs without a GPU."""
from types import SimpleNamespace

import pytest
import torch


class OnDevice(torch.Tensor):
    def get_device(self):
        return 0


class OnAnother(torch.Tensor):
    def get_device(self):
        return 1


def _i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def _calls(pa):
    """name -> (call, its tensors, its other arguments)"""
    cache, q, kv = torch.zeros(4, 2, 16, 64), torch.zeros(5, 4, 64), torch.zeros(5, 2, 64)
    mass, ws = torch.zeros(3, 2, 32), torch.zeros(1 << 12, dtype=torch.uint8)
    caches = dict(k_cache=cache, v_cache=cache)
    batch = dict(block_tables=_i32(2, 2), context_lens=_i32(2))
    attention = dict(mass=mass, workspace=ws, mass_rows=_i32(2), **caches, **batch)
    plain = dict(max_ctx=32, scale=0.1)
    return {
        "rotary_append": (dict(q_out=q, q=q, k_new=kv, v_new=kv, cu_q_lens=_i32(3),
                               positions=_i32(1, 5), slots=torch.zeros(5, dtype=torch.int64),
                               **caches, **batch), dict(rotary=pa.Rotary([1.0] * 32))),
        "decode_mass": (dict(out=q[:2], q=q[:2], **attention), plain),
        "prefill_mass": (dict(out=q, q=q, cu_q_lens=_i32(3), observe=_i32(2), **attention),
                         dict(max_q=4, **plain)),
        "evict": (dict(mass=mass, new_mass=mass, new_block_tables=_i32(2, 2), keep_lens=_i32(2),
                       new_context_lens=_i32(2), kept=_i32(2, 2, 8), workspace=ws,
                       mass_rows=_i32(2), **caches, **batch), dict(max_ctx=32)),
    }


@pytest.mark.parametrize("name", ["rotary_append", "decode_mass", "prefill_mass", "evict"])
def test_every_tensor_has_to_be_on_the_current_device(name, monkeypatch):
    import paged_kv_cache_53_gb300 as pa
    reached = []
    monkeypatch.setattr(pa, "_lib", SimpleNamespace(**{
        "pa_" + name: lambda *a: reached.append(a) or 0}))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    tensors, others = _calls(pa)[name]
    here = {k: t.as_subclass(OnDevice) for k, t in tensors.items()}
    others["stream"] = SimpleNamespace(cuda_stream=0)
    call = getattr(pa, name)
    call(**here, **others)
    assert len(reached) == 1
    for k, t in tensors.items():
        for elsewhere in (t, t.as_subclass(OnAnother)):
            with pytest.raises(ValueError, match="current device"):
                call(**{**here, k: elsewhere}, **others)
            assert len(reached) == 1, k


@pytest.mark.parametrize("name", ["rotary_append", "decode_mass", "prefill_mass", "evict"])
def test_a_type_that_is_not_built_is_a_type_error(name, monkeypatch):
    import paged_kv_cache_53_gb300 as pa
    reached = []
    monkeypatch.setattr(pa, "_lib", SimpleNamespace(**{
        "pa_" + name: lambda *a: reached.append(a) or 0}))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    tensors, others = _calls(pa)[name]
    others["stream"] = SimpleNamespace(cuda_stream=0)
    wide = {k: (t.double() if k in ("out", "q", "q_out", "k_new", "v_new", "k_cache", "v_cache")
                else t).as_subclass(OnDevice) for k, t in tensors.items()}
    with pytest.raises(TypeError, match="unsupported dtype"):
        getattr(pa, name)(**wide, **others)
    assert not reached

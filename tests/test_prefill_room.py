"""Chunks that a prefill call has no room for (a work list made for a smaller max_q, rows past
num_tokens): the sequence is flagged and left alone, and the others come out as without it."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
HQ, HKV, BS = 8, 2, 16


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_53_gb300 as pa
    pa.get_status()
    return pa


def _run(pa, d, cu, ctx, max_q, tokens, weights):
    n, w = len(ctx), -(-max(ctx) // BS)
    g = torch.Generator(device="cuda").manual_seed(7)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    kc, vc, q = randn(n * w, HKV, BS, d), randn(n * w, HKV, BS, d), randn(2000, HQ, d)[:tokens]
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    tab = torch.arange(n * w, dtype=torch.int32, device="cuda").view(n, w)
    # rows and workspace end on guards, which stay as they are
    out = torch.full((tokens + 700, HQ, d), -7.0, dtype=torch.bfloat16, device="cuda")
    size = pa.prefill_mass_workspace_bytes if weights else pa.prefill_workspace_bytes
    need = size(n, tokens, max_q, HQ, HKV, d, max(ctx), BS)
    ws = torch.full((need + 65536,), 0x5a, dtype=torch.uint8, device="cuda")
    mass = torch.ones(n, HKV, max(ctx), device="cuda")
    args = out[:tokens], q, kc, vc, tab, i32(cu), i32(ctx), max_q, max(ctx), d ** -0.5
    if weights:
        pa.prefill_mass(*args, mass, ws[:need], decay=0.5)
    else:
        pa.prefill_chunk(*args, ws[:need])
    torch.cuda.synchronize()
    assert (out[tokens:] == -7).all() and (ws[need:] == 0x5a).all()
    return out[:tokens], mass


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("cu,tokens,max_q", [
    ([0, 40, 640], 640, 40),   # 600 tokens where the list has room for 64 or 128
    ([0, 40, 640], 300, 600),  # rows past the 300 there are
])
def test_a_chunk_without_room_is_flagged_and_left_alone(pa, d, weights, cu, tokens, max_q):
    ctx = [90, 700]
    out, mass = _run(pa, d, cu, ctx, max_q, tokens, weights)
    assert pa.get_status() == pa.STATUS_BAD_CONTEXT
    ref, ref_mass = _run(pa, d, [0, 40, 640], ctx, 600, 640, weights)
    assert pa.get_status() == 0
    assert torch.equal(out[:40], ref[:40]) and (out[40:] == -7).all()
    assert torch.equal(mass[0], ref_mass[0]) and (mass[1] == 1).all()


@pytest.mark.parametrize("weights", [False, True])
def test_chunks_that_fit_all_the_same(pa, weights):
    """A max_q that is too small by less than an item's tokens still has its room."""
    cu = np.cumsum([0, 60, 33, 0, 64]).tolist()
    ctx = [60, 100, 20, 400]
    out, mass = _run(pa, 64, cu, ctx, 1, cu[-1], weights)
    ref, ref_mass = _run(pa, 64, cu, ctx, 64, cu[-1], weights)
    assert pa.get_status() == 0
    assert torch.equal(out, ref) and torch.equal(mass, ref_mass)


@pytest.mark.parametrize("weights", [False, True])
def test_starts_that_fall_back_to_zero_are_no_chunks(pa, weights):
    """Entries behind the batch's own sequences, left at zero."""
    out, mass = _run(pa, 64, [0, 30, 0, 0], [50, 0, 0], 30, 30, weights)
    ref, ref_mass = _run(pa, 64, [0, 30], [50], 30, 30, weights)
    assert pa.get_status() == 0
    assert torch.equal(mass[0], ref_mass[0]) and (mass[1:] == 1).all()
    assert torch.isfinite(out.float()).all() and out.shape == ref.shape

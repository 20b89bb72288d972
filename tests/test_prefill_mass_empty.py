"""pa_prefill_mass where no chunk has a query: decay is applied to every context all the same.

A position's new mass is decay * old rounded to fp32 once, in a call without tokens as in one where
another sequence has some: bit for bit.
"""

import numpy as np
import pytest
import torch

FAKE = 0x10000
HQ, HKV, D, BS = 8, 2, 64, 16


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_53_gb300 import build
    path = build.build()
    import paged_kv_cache_53_gb300 as pa
    pa.lib(path)
    return pa


def _c_call(lib, **kw):
    a = dict(out=None, odt=2, q=None, k=FAKE, v=FAKE, bt=FAKE, maxblk=8, cu=FAKE, ctx=FAKE,
             observe=None, max_q=0, max_ctx=128, mass=FAKE, stride=128, rows=None, nrows=4,
             decay=0.5, B=4, T=0, Hq=HQ, Hkv=HKV, D=D, BS=BS, NB=64, scale=0.1, dt=2, ws=None,
             wsb=0)
    a.update(kw)
    return lib.pa_prefill_mass(*a.values(), None)


@pytest.mark.parametrize("kw,code,needle", [
    (dict(mass=None), 1, "null mass"), (dict(mass=FAKE + 2), 1, "4-byte"),
    (dict(stride=127), 1, "mass_stride"), (dict(nrows=3), 1, "rows of mass"),
    (dict(decay=-0.1), 1, "decay"), (dict(decay=float("nan")), 1, "decay"),
    (dict(ctx=None), 1, "null"), (dict(maxblk=0), 1, "max_blocks"), (dict(dt=0, odt=0), 2, "fp32"),
    (dict(B=70000, nrows=70000), 2, "65535"), (dict(D=96), 2, "head_dim"),
])
def test_refusals_without_tokens(pa, kw, code, needle):
    lib = pa.lib()
    assert _c_call(lib, **kw) == code
    msg = lib.pa_last_error_string().decode()
    assert "pa_prefill_mass" in msg and needle in msg


def test_nothing_to_do(pa):
    lib = pa.lib()
    assert _c_call(lib, decay=1.0) == 0          # no query, nothing fades
    assert _c_call(lib, B=0, mass=None, ctx=None) == 0


def _dev(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()


def _run(pa, ctx, new, mass, rows, decay, max_ctx, width=None, run=None):
    """One call over `ctx` with `new` queries each; `run` wraps the call itself."""
    n, t = len(ctx), int(sum(new))
    w = width or -(-max_ctx // BS)
    g = torch.Generator(device="cuda").manual_seed(3)
    kc, vc = (torch.randn(n * w, HKV, BS, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    tab = torch.arange(n * w, dtype=torch.int32, device="cuda").view(n, w)
    q = torch.randn(t, HQ, D, generator=g, device="cuda").bfloat16()
    out, cu, mq = torch.empty_like(q), _dev(np.concatenate([[0], np.cumsum(new)])), max(new)
    cl, mr = _dev(ctx), None if rows is None else _dev(rows)
    ws = torch.empty(pa.prefill_mass_workspace_bytes(n, t, mq, HQ, HKV, D, max_ctx, BS),
                     dtype=torch.uint8, device="cuda")
    call = lambda: pa.prefill_mass(out, q, kc, vc, tab, cu, cl, mq, max_ctx, 0.125, mass, ws,  # noqa: E731
                                   mass_rows=mr, decay=decay)
    call() if run is None else run(call)
    torch.cuda.synchronize()
    return mass


CTX = [40, 0, 700, 1, 33, 1500]


@pytest.mark.gpu
@pytest.mark.parametrize("decay", [1.0, 0.75, 0.3, 0.0])
@pytest.mark.parametrize("in_order", [False, True])
def test_decay_without_any_token(pa, decay, in_order):
    pa.get_status()
    n = len(CTX)
    rows = None if in_order else np.random.default_rng(1).permutation(n + 3)[:n]
    g = torch.Generator(device="cuda").manual_seed(2)
    old = torch.rand(n + 3, HKV, 1507, generator=g, device="cuda")
    if decay == 0.0:
        old.fill_(float("nan"))  # not read
    got = _run(pa, CTX, [0] * n, old.clone(), rows, decay, 1500)
    assert pa.get_status() == 0
    want = old.clone()
    for b, c in enumerate(CTX):
        r = b if rows is None else int(rows[b])
        want[r, :, :c] = old[r, :, :c] * decay if decay else 0.0
    assert torch.equal(got.view(torch.int32), want.view(torch.int32))
    # a batch in which one more sequence has queries leaves the others the same
    more = _run(pa, CTX + [20], [0] * n + [20], old.clone(),
                list(range(n + 1)) if rows is None else list(rows) + [sorted(set(range(n + 3)) - set(rows))[0]],
                decay, 1500)
    for b in range(n):
        r = b if rows is None else int(rows[b])
        assert torch.equal(more[r].view(torch.int32), got[r].view(torch.int32))


@pytest.mark.gpu
def test_bad_rows_and_contexts_without_tokens(pa):
    """Flagged and left alone; the table bounds a context as max_ctx does."""
    pa.get_status()
    g = torch.Generator(device="cuda").manual_seed(5)
    for ctx, rows, kw in (([40, 30], [9, 1], {}), ([40, 30], [-1, 1], {}),
                          ([-3, 30], [0, 1], {}), ([101, 30], [0, 1], {}),
                          ([40, 30], [0, 1], dict(width=2))):
        old = torch.rand(3, HKV, 112, generator=g, device="cuda")
        got = _run(pa, ctx, [0, 0], old.clone(), rows, 0.5, 100, **kw)
        assert pa.get_status() == pa.STATUS_BAD_CONTEXT
        want = old.clone()
        want[1, :, :30] *= 0.5
        assert torch.equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("ctx", [-3, 101])
def test_bad_contexts_of_empty_chunks_beside_a_query(pa, ctx):
    pa.get_status()
    old = torch.rand(3, HKV, 112, device="cuda")
    got = _run(pa, [ctx, 30], [0, 7], old.clone(), None, 0.5, 100)
    assert pa.get_status() == pa.STATUS_BAD_CONTEXT
    assert torch.equal(got[[0, 2]], old[[0, 2]]) and not torch.equal(got[1], old[1])


@pytest.mark.gpu
def test_captured_and_replayed(pa):
    pa.get_status()
    old = torch.rand(2, HKV, 100, device="cuda")
    mass = old.clone()

    def capture(call):
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()

    _run(pa, [90, 17], [0, 0], mass, None, 0.5, 100, run=capture)
    want = old.clone()
    want[0, :, :90] *= 0.125
    want[1, :, :17] *= 0.125
    assert pa.get_status() == 0 and torch.equal(mass, want)

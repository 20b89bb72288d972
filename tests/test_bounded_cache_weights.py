"""The weights of every step of a bounded cache's run (prefill, decode, cut, decode on), each
position's increment on its own, against softmax sums in 64 bits over the device's stored rows.

The bound on a position's new mass is the one of the single calls: the relative error of its weight
that cache_bounds_ref.attention derives from the fp32 scores, and fp32's rounding of the old mass
plus the weight (2^-23 of both).  It is a small part of a step's own weights, which the test asserts:
a step that added nothing, or another step's weights, would not pass.
"""
import numpy as np
import pytest
import torch

import workloads as W
from cache_bounds_ref import attention, dev, select

pytestmark = pytest.mark.gpu

HQ, HKV, D, BS, NB, WIDTH = 8, 2, 64, 16, 80, 24
SCALE = D ** -0.5


class Server:
    def __init__(self, pa, prompts, seed):
        from paged_kv_cache_53_gb300.block_manager import BlockManager
        self.pa, self.gen = pa, torch.Generator(device="cuda").manual_seed(seed)
        self.n = len(prompts)
        self.bm = BlockManager(NB, BS)
        for b, p in enumerate(prompts):
            self.bm.add_sequence(b, list(range(p)))
        self.kc, self.vc = (torch.zeros(NB, HKV, BS, D, dtype=torch.bfloat16, device="cuda")
                            for _ in range(2))
        self.mass = torch.zeros(self.n, HKV, WIDTH * BS, device="cuda")
        self.rotary = pa.Rotary([10000.0 ** (-2.0 * i / D) for i in range(D // 2)],
                                [i % 3 for i in range(D // 2)])
        self.pos = [0] * self.n  # the next token's place in the text

    def step(self, counts, decay):
        pa, n = self.pa, self.n
        tab, ctx = self.bm.block_tables(range(n), WIDTH)
        cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        t, m = int(cu[-1]), int(ctx.max())
        q, k, v = (W.randn((t, h, D), "bf16", "cuda", self.gen) for h in (HQ, HKV, HKV))
        at = np.concatenate([np.arange(p, p + c) for p, c in zip(self.pos, counts)])
        self.pos = [p + c for p, c in zip(self.pos, counts)]
        qo, out = torch.empty_like(q), torch.empty(q.shape, device="cuda")
        bt, cl, cq = dev(tab), dev(ctx), dev(cu)
        pa.rotary_append(qo, q, k, v, self.kc, self.vc, bt, cq, cl,
                         dev(np.stack([at // f for f in (1, 3, 5)])), self.rotary)
        old = self.mass.clone()
        if max(counts) == 1:
            ws = torch.empty(pa.decode_mass_workspace_bytes(n, HQ, HKV, D, m, BS),
                             dtype=torch.uint8, device="cuda")
            pa.decode_mass(out, qo, self.kc, self.vc, bt, cl, m, SCALE, self.mass, ws, decay=decay)
        else:
            ws = torch.empty(pa.prefill_mass_workspace_bytes(n, t, max(counts), HQ, HKV, D, m, BS),
                             dtype=torch.uint8, device="cuda")
            pa.prefill_mass(out, qo, self.kc, self.vc, bt, cq, cl, max(counts), m, SCALE,
                            self.mass, ws, decay=decay)
        ref_out, ref, w, rel = attention(qo, self.kc, self.vc, bt, cu, ctx, SCALE, old, None, decay)
        assert rel < 2e-3
        tol = rel * w + 2.0 ** -23 * (old.double() + w)
        assert ((self.mass.double() - ref).abs() <= tol).all()
        added = (self.mass.double() - decay * old.double()).sum(-1)
        want = torch.tensor(counts, device="cuda", dtype=torch.float64)[:, None] * (HQ // HKV)
        assert ((added - want).abs() <= tol.sum(-1)).all()
        assert (want >= 100 * tol.sum(-1)).all()  # what a step adds is far above the bound
        assert (out.double() - ref_out).abs().max().item() < 2e-3

    def cut(self, budget, sinks, recent):
        pa, n = self.pa, self.n
        before, ctx = self.bm.block_tables(range(n), WIDTH)
        keep = [min(budget, int(c)) for c in ctx]
        self.bm.evict(range(n), keep)
        after, _ = self.bm.block_tables(range(n), WIDTH)
        k0, v0, m0 = self.kc.clone(), self.vc.clone(), self.mass.clone()
        kept = torch.empty(n, HKV, budget, dtype=torch.int32, device="cuda")
        new_ctx = torch.empty(n, dtype=torch.int32, device="cuda")
        ws = torch.empty(pa.evict_workspace_bytes(n, HKV, int(ctx.max()), budget),
                         dtype=torch.uint8, device="cuda")
        pa.evict(self.kc, self.vc, self.mass, self.mass, dev(before), dev(after), dev(ctx),
                 dev(keep), int(ctx.max()), new_ctx, kept, ws, sinks=sinks, recent=recent)
        assert new_ctx.tolist() == keep
        for b in range(n):
            for h in range(HKV):
                sel = select(m0[b, h, :int(ctx[b])].cpu().numpy(), keep[b], sinks, recent)
                assert np.array_equal(kept[b, h, :keep[b]].cpu().numpy(), sel)
                assert torch.equal(self.mass[b, h, :keep[b]], m0[b, h, dev(sel, np.int64)])
                assert not self.mass[b, h, keep[b]:].any()
                to = np.arange(keep[b])
                src, dst = (dev(x, np.int64) for x in (before[b, sel // BS], after[b, to // BS]))
                so, do = dev(sel % BS, np.int64), dev(to % BS, np.int64)
                assert torch.equal(self.kc[dst, h, do], k0[src, h, so])
                assert torch.equal(self.vc[dst, h, do], v0[src, h, so])


@pytest.mark.parametrize("decay", [1.0, 0.9, 0.0])
def test_every_step_adds_its_own_weights(decay):
    import paged_kv_cache_53_gb300 as pa
    pa.get_status()
    s = Server(pa, [300, 171], seed=int(10 * decay))
    s.step([300, 171], decay)
    for _ in range(2):
        for _ in range(6):
            s.bm.append_tokens_batch([0, 1], [7, 8])
            s.step([1, 1], decay)
        s.cut(100, sinks=2, recent=16)
    s.bm.append_tokens_batch([0, 1], list(range(30)), [21, 9])  # a chunk over the cut cache
    s.step([21, 9], decay)
    assert pa.get_status() == 0

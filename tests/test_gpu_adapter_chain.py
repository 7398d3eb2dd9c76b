"""Adapters, their gradients and their orthogonalised updates together, as
fine-tuning beside frozen NVFP4 weights and serving use them."""
import numpy as np
import pytest
import torch

import adapter_ref as A
import operator_ref as R
from gpu_util import say

pytestmark = pytest.mark.gpu
USUAL = (3.4445, -4.7750, 2.0315)


class Tuned:
    """A frozen NVFP4 projection with trainable adapters."""

    def __init__(self, K, N, rank, S, dtype, seed):
        from nvfp4_w4a4_quantized_amd.ops import NvFp4Weights
        self.gen = torch.Generator().manual_seed(seed)
        parts = R.make_weights(np.random.default_rng(seed), 1, N, K, std=0.1)
        self.matrix = R.decode(*parts)[0]
        self.w = NvFp4Weights(*(t.cuda() for t in parts)).packed()
        self.K, self.N, self.dtype, self.S = K, N, dtype, S
        self.a = self.normal(S, rank, K, std=K ** -0.5)
        self.b = self.normal(S, N, rank, std=0.1)
        self.scale = (torch.rand(S, generator=self.gen) + 0.5).cuda()

    def normal(self, *shape, std=1.0):
        return (torch.randn(*shape, generator=self.gen) * std).to(self.dtype).cuda()

    def inputs(self, T, kind):
        return [self.normal(T, self.K), self.normal(T, self.N), A.make_ids(self.gen, T, self.S, kind).cuda()]

    def step(self, x, target, ids):
        """Forward, the gradient of |y - target|^2 / 2 and the updates."""
        from nvfp4_w4a4_quantized_amd import ops
        base = ops.nvfp4_matvec(x, self.w)
        y, h = ops.lora_forward(x, self.a, self.b, ids, scale=self.scale, base=base, return_h=True)
        dy = y - target
        dx, da, db = ops.lora_backward(dy, x, self.a, self.b, ids, scale=self.scale, h=h)
        return [y, dx, da, db, ops.newton_schulz(da, out_dtype=self.dtype),
                ops.newton_schulz(db, out_dtype=self.dtype, scale=0.2),
                ops.newton_schulz(db.view(-1, db.shape[-1]), out_dtype=torch.bfloat16),
                ops.newton_schulz(torch.mm(db[0], da[0])),
                ops.nvfp4_lora_matvec(x, self.w, self.a, self.b, ids, scale=self.scale)]


@pytest.mark.parametrize("T,kind", [(6, "random"), (500, "runs")])
def test_one_step_against_binary64(T, kind):
    """Every result of a step against the definitions chained in binary64.
    Sums of at most 512 binary32 terms through four products: 1e-4 of each norm
    leaves a factor of ten; the updates repeat newton_schulz's own tolerance, 4e-3
    of bf16 results, on the gradients that the step itself gave."""
    t = Tuned(256, 128, 8, 3, torch.float32, 1)
    x, target, ids = t.inputs(T, kind)
    say("step", T, kind)
    y, dx, da, db, ua, ub, uf, um, served = (v.cpu() for v in t.step(x, target, ids))
    a, b, i = t.a.cpu(), t.b.cpu(), ids.cpu()
    ref, _, h, _ = A.forward(x.cpu(), a, b, i, t.scale.cpu(), None, t.matrix)
    (rdx, _), (rda, _), (rdb, _) = A.backward(ref - target.cpu().double(), x.cpu(), a, b, i,
                                              t.scale.cpu(), h, None)
    for got, want in ((y, ref), (served, ref), (dx, rdx), (da, rda), (db, rdb)):
        assert float((got.double() - want).norm()) <= 1e-4 * float(want.norm())
    for got, g, c, tol in ((ua, da, 1.0, 1e-4), (ub, db, 0.2, 1e-4), (uf, db.view(-1, 8), 1.0, 8e-3),
                           (um, db[0] @ da[0], 1.0, None)):
        want = A.newton_schulz(g, 5, USUAL, 1e-7, c)
        if tol is None:        # of rank 8: X's 22 bits grow by a^5 in the other directions
            tol = 1e-4 + USUAL[0] ** 5 * 2.0 ** -22 / float(want.norm()) + 1e-2
        assert float((got.double() - want).norm()) <= tol * float(want.norm())


def test_updates_of_the_expert_layers_gradients():
    """moe_expert_backward's binary32 weight gradients go straight into the
    update, every expert's matrix by itself (an expert without tokens: zeros)."""
    from nvfp4_w4a4_quantized_amd import ops
    T, E, k, H, I = 96, 6, 2, 256, 128
    gen = torch.Generator().manual_seed(2)
    x = torch.randn(T, H, generator=gen).bfloat16().cuda()
    w1 = (torch.randn(E, 2 * I, H, generator=gen) * 0.1).bfloat16().cuda()
    w2 = (torch.randn(E, H, I, generator=gen) * 0.1).bfloat16().cuda()
    logits = torch.randn(T, E, generator=gen)
    logits[:, 4] = -float("inf")
    ids, w = ops.moe_router(logits.cuda(), k)
    y, it = ops.moe_expert_forward(x, ids, w, E, I, ops.NvFp4Weights.quantize(w1),
                                   ops.NvFp4Weights.quantize(w2), debug=True, fc1_out=True)
    g = ops.moe_expert_backward(y, x, it["fc1_out"], it["d"], it["expert_offsets"], it["row_src"],
                                it["row_prob"], it["dst_row"], w1, w2)
    for name in ("dw1", "dw2"):
        say("expert update", name)
        for dtype, tol in ((torch.float32, 1e-3), (torch.bfloat16, 8e-3)):
            u = ops.newton_schulz(g[name], out_dtype=dtype)
            ref = A.newton_schulz(g[name], 5, USUAL, 1e-7)
            assert not bool(u[4].any())
            # (a batch of 96 tokens leaves directions that only X's last bits fill:
            # a^5 2^-22 of |X0| = 1 each way)
            for e in range(E):
                lim = tol * float(ref[e].norm()) + USUAL[0] ** 5 * 2.0 ** -22
                assert float((u[e].double() - ref[e]).norm()) <= lim


def test_served_rows_are_the_projection_with_the_adapters():
    """nvfp4_lora_matvec against nvfp4_matvec in binary32 with lora_forward on
    top: the same sums in another order, (K + rank + 40) 2^-24 of the magnitudes."""
    from nvfp4_w4a4_quantized_amd import ops
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        t = Tuned(384, 160, 16, 4, dtype, 3)
        for T in (1, 9, 300):
            x, _, ids = t.inputs(T, "random")
            got = ops.nvfp4_lora_matvec(x, t.w, t.a, t.b, ids, scale=t.scale, out_dtype=torch.float32)
            base = ops.nvfp4_matvec(x, t.w, out_dtype=torch.float32)
            two = ops.lora_forward(x, t.a, t.b, ids, scale=t.scale, base=base, out_dtype=torch.float32)
            mag = A.forward(x.cpu(), t.a.cpu(), t.b.cpu(), ids.cpu(), t.scale.cpu(), None, t.matrix)[1]
            assert bool(((got - two).cpu().double().abs() <= 2 * (384 + 16 + 40) * A.ULP * mag).all())


@pytest.mark.parametrize("T,kind", [(5, "random"), (300, "runs")])
def test_captured_and_replayed(T, kind):
    """Two graphs of the same step, each with its own workspaces, replayed in
    turn on changed inputs with eager work between, give the eager bits."""
    t = Tuned(256, 192, 16, 3, torch.bfloat16, 4)
    held = t.inputs(T, kind)
    t.step(*held)                                   # loads the kernels
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = t.step(*held)
        graphs.append((g, out))
    for turn in range(4):
        new = t.inputs(T, ("runs", "random", "none", "wild")[turn])
        for old, v in zip(held, new):
            old.copy_(v)
        want = [v.clone() for v in t.step(*new)]
        for g, out in graphs:
            for v in out:
                v.fill_(0)
            g.replay()
            torch.cuda.synchronize()
            for p, q in zip(out, want):
                assert torch.equal(p.nan_to_num(7.0), q.nan_to_num(7.0))


def test_two_streams_at_once():
    """Calls in flight together on two side streams do not disturb each other."""
    a, b = Tuned(256, 128, 8, 3, torch.bfloat16, 5), Tuned(512, 384, 40, 2, torch.bfloat16, 6)
    ia, ib = a.inputs(7, "random"), b.inputs(400, "runs")
    want_a, want_b = a.step(*ia), b.step(*ib)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got_a, got_b = [], []
    for _ in range(5):
        with torch.cuda.stream(sa):
            got_a.append(a.step(*ia))
        with torch.cuda.stream(sb):
            got_b.append(b.step(*ib))
    torch.cuda.synchronize()
    for got, want in ((got_a, want_a), (got_b, want_b)):
        for out in got:
            for p, q in zip(out, want):
                assert torch.equal(p, q)

"""The operators together, as training and decoding use them: under graph
capture, on other streams, and beside the quantized layer's own calls."""
import numpy as np
import pytest
import torch

import operator_ref as R
from gpu_util import say

pytestmark = pytest.mark.gpu


def held(codes, scales, gs):
    from nvfp4_w4a4_quantized_amd.ops import NvFp4Weights
    return NvFp4Weights(codes.cuda(), scales.cuda(), gs.cuda()).packed()


def test_training_chain_against_autograd():
    """router -> metadata -> sort -> a linear map per expert -> weighted unsort
    and all their gradients, against binary64 autograd of the same formulas.
    Tolerance: binary32 sums of at most 96 terms of size O(1) through three
    stages, far below 1e-4 of each result's norm."""
    from nvfp4_w4a4_quantized_amd import ops
    rng = np.random.default_rng(1)
    T, E, k, H = 90, 12, 3, 96
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32))
    wr = torch.from_numpy(rng.standard_normal((H, E)).astype(np.float32) * 0.1)
    we = torch.from_numpy(rng.standard_normal((E, H, H)).astype(np.float32) * 0.1)
    dy = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32))

    xd, wed = x.double().requires_grad_(), we.double().requires_grad_()
    z = (x @ wr).double().requires_grad_()
    ids = R.router_ids((x @ wr), k)
    w = torch.softmax(z.gather(1, ids.long()), dim=1)
    y = torch.zeros(T, H, dtype=torch.float64)
    for j in range(k):
        y = y + w[:, j:j + 1] * torch.einsum("th,thg->tg", xd, wed[ids[:, j].long()])
    y.backward(dy.double())

    logits = (x @ wr).cuda()
    say("training chain")
    gi, gw = ops.moe_router(logits, k)
    assert torch.equal(gi.cpu(), ids)
    m = ops.moe_permute(None, gi, gw, E, align=8)
    maps = (m["dst_row"], m["row_src"], m["offsets"])
    o = m["offsets"].cpu().tolist()
    rows = ops.moe_sort_tokens(x.cuda(), *maps)
    out = torch.zeros_like(rows)
    for e in range(E):
        out[o[e]:o[e + 1]] = rows[o[e]:o[e + 1]] @ we[e].cuda()
    got = ops.moe_unsort_tokens(out, m["dst_row"], prob=gw)
    d_out, d_w = ops.moe_unsort_tokens_backward(dy.cuda(), *maps, rows=out, prob=gw)
    d_we = torch.zeros_like(we)
    d_rows = torch.zeros_like(rows)
    for e in range(E):
        seg = slice(o[e], o[e + 1])
        d_rows[seg] = d_out[seg] @ we[e].cuda().t().contiguous()
        d_we[e] = (rows[seg].t().contiguous() @ d_out[seg]).cpu()
    dx, _ = ops.moe_sort_tokens_backward(d_rows, m["dst_row"])
    dz = ops.moe_router_backward(d_w, logits, gi)
    for a, b in ((got, y.detach()), (dx, xd.grad), (dz, z.grad), (d_we, wed.grad)):
        a = a.cpu().double()
        assert float((a - b).norm() / b.norm()) < 1e-4


def test_router_gradient_from_the_expert_backward():
    """moe_expert_backward's dprob goes straight into moe_router_backward."""
    from nvfp4_w4a4_quantized_amd import ops
    rng = np.random.default_rng(2)
    T, E, k, H, I = 64, 8, 2, 128, 128
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).bfloat16().cuda()
    w1 = (torch.randn(E, 2 * I, H, device="cuda") * 0.1).bfloat16()
    w2 = (torch.randn(E, H, I, device="cuda") * 0.1).bfloat16()
    logits = torch.randn(T, E, device="cuda")
    ids, w = ops.moe_router(logits, k)
    q1, q2 = ops.NvFp4Weights.quantize(w1), ops.NvFp4Weights.quantize(w2)
    y, it = ops.moe_expert_forward(x, ids, w, E, I, q1, q2, debug=True, fc1_out=True)
    g = ops.moe_expert_backward(torch.ones_like(y), x, it["fc1_out"], it["d"],
                                it["expert_offsets"], it["row_src"], it["row_prob"],
                                it["dst_row"], w1, w2)
    dz = ops.moe_router_backward(g["dprob"], logits, ids).cpu()
    ref = R.router_gradient(logits.cpu(), ids.cpu(), g["dprob"].cpu(), 0, True)
    assert float((dz.double() - ref).norm() / ref.norm()) < 1e-5


class Decoder:
    """One decoding step: logits -> picks -> the expert layer, plus a projection."""

    def __init__(self, T, seed):
        rng = np.random.default_rng(seed)
        self.T, self.E, self.k, self.H, self.I = T, 16, 4, 256, 128
        self.w1 = held(*R.make_weights(rng, self.E, 2 * self.I, self.H, std=0.1))
        self.w2 = held(*R.make_weights(rng, self.E, self.H, self.I, std=0.1))
        self.wp = held(*R.make_weights(rng, 1, 96, self.H, std=0.1))
        self.rng = rng

    def inputs(self):
        x = torch.from_numpy(self.rng.standard_normal((self.T, self.H)).astype(np.float32))
        z = torch.from_numpy(self.rng.standard_normal((self.T, self.E)).astype(np.float32))
        return x.bfloat16().cuda(), z.cuda()

    def step(self, x, z):
        from nvfp4_w4a4_quantized_amd import ops
        ids, w = ops.moe_router(z, self.k)
        y = ops.moe_expert_decode(x, ids, w, self.E, self.I, self.w1, self.w2)
        m = ops.moe_permute(None, ids, w, self.E, align=4)
        rows = torch.zeros((m["row_src"].numel(), self.H), dtype=x.dtype, device=x.device)
        ops.moe_sort_tokens(x, m["dst_row"], m["row_src"], m["offsets"], out=rows)
        back = ops.moe_unsort_tokens(rows, m["dst_row"], prob=w)
        dz = ops.moe_router_backward(w, z, ids)
        return [y, ids, w, back, dz, ops.nvfp4_matvec(x, self.wp),
                ops.nvfp4_expert_matvec(x, ids, self.w1)]


def test_decoding_against_the_definition():
    d = Decoder(5, 3)
    x, z = d.inputs()
    y, ids, w, back, *_ = d.step(x, z)
    assert torch.equal(ids.cpu(), R.router_ids(z.cpu(), d.k))
    # sum of the weights is one, so sorted and weighted back x is x, up to k
    # binary32 roundings and the type's half step
    err = (back.double() - x.double()).abs()
    assert bool((err <= (2.0 ** -8 + 2.0 ** -18) * x.double().abs()).all())


@pytest.mark.parametrize("T", [1, 20])
def test_captured_and_replayed(T):
    """Two graphs of the same step (each with its own workspace), replayed in
    turn on changed inputs with eager work between, give the eager bits."""
    d = Decoder(T, 4)
    x, z = d.inputs()
    d.step(x, z)                                   # loads the kernels
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = d.step(x, z)
        graphs.append((g, out))
    for _ in range(4):
        nx, nz = d.inputs()
        x.copy_(nx)
        z.copy_(nz)
        want = [t.clone() for t in d.step(nx, nz)]
        for g, out in graphs:
            for t in out:
                t.fill_(0)
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(out, want):
                assert torch.equal(a, b)


def test_two_streams_at_once():
    """Calls in flight together on two side streams do not disturb each other."""
    a, b = Decoder(7, 5), Decoder(33, 6)
    ia, ib = a.inputs(), b.inputs()
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

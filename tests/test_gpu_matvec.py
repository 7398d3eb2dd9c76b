"""nvfp4_matvec, nvfp4_expert_matvec and moe_expert_decode against binary64.

Tolerances: the documented (k + 16) 2^-24 sum |w x| of a binary32 sum of
exact products, plus the output type's half step.  The layer: errors of h
carried through D = silu(g) u p (|silu'| <= 1.1, |silu| <= |g|), D's own
roundings (2^-17 of its two parts with 16-bit x, (|g| + 16) 2^-24 of the
exponential) and FC2's sum."""
import numpy as np
import pytest
import torch

import operator_ref as R
from gpu_util import say

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def held(codes, scales, gs, tiled):
    from nvfp4_w4a4_quantized_amd.ops import NvFp4Weights
    w = NvFp4Weights(codes.cuda(), scales.cuda(), gs.cuda())
    if tiled:
        w = w.packed()
        c, s = R.tile_weights(codes, scales)
        assert torch.equal(w.codes.cpu(), c) and torch.equal(w.scales.cpu(), s)
    return w


def check(got, ref, mag, k, what):
    bad = R.outside(got, ref, (k + 16) * 2.0 ** -24 * mag)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} outside"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,n,k,tiled", [
    (1, 1, 16, False), (1, 5, 48, False), (3, 33, 112, False), (17, 100, 144, False),
    (1, 32, 128, True), (2, 96, 256, True), (16, 64, 1024, True), (33, 160, 640, True),
    (5, 1001, 2064, False), (64, 257, 1040, False), (65, 48, 16384, False), (1, 64, 16384, True),
    (130, 64, 384, True), (1, 5120, 2048, True),
    # more weight rows: the kernel that shares x through LDS, at every number of
    # columns, with rows and stages that end inside a tile
    (1, 32771, 272, False), (2, 32768, 128, True), (7, 24581, 144, False), (8, 24576, 384, True),
    (16, 10247, 400, False), (15, 10240, 1024, True), (30, 8193, 112, False), (32, 8192, 640, True),
    (64, 6145, 1040, False), (70, 6176, 384, True), (64, 32800, 256, True), (40, 32771, 48, False),
    (33, 6150, 32, False), (64, 6200, 16, False),
    # columns over workgroups, four groups of waves with 16, 32 and 64 columns
    (40, 4100, 2064, False), (64, 4096, 1152, True), (50, 8170, 1040, False),
    (64, 8192, 1280, True), (61, 16380, 1040, False), (70, 16390, 528, False),
    (12, 16400, 1200, False), (100, 4101, 80, False)])
def test_matvec(T, n, k, tiled, dtype):
    from nvfp4_w4a4_quantized_amd import ops
    rng = np.random.default_rng(T + n + k)
    codes, scales, gs = R.make_weights(rng, 1, n, k)
    w = held(codes, scales, gs, tiled)
    x = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).to(dtype)
    m = R.decode(codes, scales, gs)[0]
    ref, mag = x.double() @ m.t(), x.double().abs() @ m.abs().t()
    for out in {dtype, torch.float32}:
        say("matvec", T, n, k, tiled, dtype, out)
        check(ops.nvfp4_matvec(x.cuda(), w, out_dtype=out), ref, mag, k, f"{dtype} -> {out}")


def test_matvec_every_code_and_scale_is_exact():
    """x = one-hot rows: out is the weight itself, every code with every
    finite E4M3 byte (outer scale 1, binary32 out)."""
    from nvfp4_w4a4_quantized_amd import ops
    from nvfp4_w4a4_quantized_amd.ops import NvFp4Weights
    n, k = 127, 16
    codes = np.zeros((1, n, k // 2), np.uint8)
    codes[:] = [(2 * j) | ((2 * j + 1) << 4) for j in range(8)]
    scales = np.arange(127, dtype=np.uint8).reshape(1, n, 1)
    gs = torch.ones(1)
    codes, scales = torch.from_numpy(codes), torch.from_numpy(scales)
    w = held(codes, scales, gs, False)
    ref = R.decode(codes, scales, gs)[0].t()
    for dtype in DTYPES:
        y = ops.nvfp4_matvec(torch.eye(k, dtype=dtype, device="cuda"), w, out_dtype=torch.float32)
        assert torch.equal(y.cpu().double(), ref)


def test_matvec_binary32_keeps_all_bits():
    """A binary32 x is used whole: one-hot rows with 24-bit values."""
    from nvfp4_w4a4_quantized_amd import ops
    rng = np.random.default_rng(3)
    codes, scales, _ = R.make_weights(rng, 1, 40, 64)
    gs = torch.ones(1)
    w = held(codes, scales, gs, False)
    v = torch.from_numpy(rng.standard_normal(64).astype(np.float32))
    y = ops.nvfp4_matvec(torch.diag(v).cuda(), w)
    ref = (R.decode(codes, scales, gs)[0] * v.double()).t()
    assert bool(((y.cpu().double() - ref).abs() <= 2.0 ** -24 * 1.0001 * 3 * ref.abs()).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_matvec_strided_x(dtype):
    from nvfp4_w4a4_quantized_amd import ops
    rng = np.random.default_rng(5)
    codes, scales, gs = R.make_weights(rng, 1, 70, 208)
    w = held(codes, scales, gs, False)
    big = torch.full((9, 240), float("nan"), dtype=dtype, device="cuda")
    xs = big[:, 5:213]
    xs.copy_(torch.from_numpy(rng.standard_normal((9, 208)).astype(np.float32)))
    out = torch.empty((9, 70), dtype=torch.float32, device="cuda")
    y = ops.nvfp4_matvec(xs, w, out_dtype=torch.float32, out=out)
    assert y is out and torch.equal(y, ops.nvfp4_matvec(xs.contiguous(), w, out_dtype=torch.float32))


def make_ids(rng, T, k, E, kind):
    if kind == "one":
        ids = np.full((T, k), -1, np.int32)
        ids[:, 0] = E - 1                   # one expert holds every entry
    else:
        ids = np.stack([rng.choice(E, k, replace=False) for _ in range(T)]).astype(np.int32)
        if kind == "dropped":
            gone = rng.random((T, k)) < 0.3
            ids[gone] = rng.choice([-1, E, -1000, 1 << 30], int(gone.sum()))
            ids[T // 2] = -1
    return torch.from_numpy(ids.reshape(T, k))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,E,n,K,tiled,kind", [
    (1, 1, 1, 16, 16, False, "plain"), (1, 8, 128, 64, 256, True, "plain"),
    (4, 3, 5, 50, 80, False, "dropped"), (37, 4, 60, 101, 336, False, "dropped"),
    (40, 1, 7, 32, 128, True, "one"), (64, 8, 16, 96, 384, True, "dropped"),
    (512, 8, 8, 32, 128, True, "plain"), (4096, 1, 3, 17, 32, False, "plain"),
    (2, 2, 1024, 16, 48, False, "plain"),
    (64, 2, 64, 1500, 208, False, "dropped"), (300, 4, 12, 1101, 336, False, "dropped"),
    (100, 1, 1, 400, 144, False, "one"), (60, 6, 50, 1024, 512, True, "plain"),
    # workgroups that share an expert's columns, one expert with many more than
    # the others; two groups of waves with 16 and 32 columns
    (300, 4, 12, 500, 272, False, "one"), (1000, 4, 12, 1100, 80, False, "one"),
    (60, 6, 50, 600, 528, False, "dropped"), (128, 4, 16, 512, 384, True, "plain")])
def test_expert_matvec(T, k, E, n, K, tiled, kind, dtype):
    from nvfp4_w4a4_quantized_amd import ops
    rng = np.random.default_rng(T + n + K)
    codes, scales, gs = R.make_weights(rng, E, n, K)
    w = held(codes, scales, gs, tiled)
    m = R.decode(codes, scales, gs)
    ids = make_ids(rng, T, k, E, kind)
    for by_entry in (False, True):
        shape = (T, k, K) if by_entry else (T, K)
        x = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dtype)
        ref, mag = R.expert_products(x, ids, m, by_entry)
        say("expert_matvec", T, k, E, n, K, tiled, kind, dtype, by_entry)
        out = torch.full((T, k, n), 3.0, dtype=dtype, device="cuda")
        y = ops.nvfp4_expert_matvec(x.cuda(), ids.cuda(), w, out=out)
        assert y is out
        check(y, ref, mag, K, f"by_entry={by_entry}")
        assert bool((y.cpu()[(ids < 0) | (ids >= E)] == 0).all())


def decode_ref(x, ids, prob, m1, m2):
    """y, and how far a result may be from it before its rounding."""
    I = m2.shape[2]
    H = m1.shape[2]
    h, hm = R.expert_products(x, ids, m1)
    g, u = h[..., :I], h[..., I:]
    p = prob.double().unsqueeze(-1)
    sig = torch.exp(R.log_sigmoid(g))
    ok = ((ids >= 0) & (ids < m1.shape[0])).unsqueeze(-1)
    d = torch.where(ok, g * sig * u * p, torch.zeros_like(h[..., :I]))
    eg, eu = ((H + 16) * 2.0 ** -24 * hm[..., :I], (H + 16) * 2.0 ** -24 * hm[..., I:])
    ed = torch.where(ok, (1.1 * eg * (u.abs() + eu) + (g * sig).abs() * eu) * p.abs()
                     + d.abs() * ((0.0 if x.dtype == torch.float32 else 2.0 ** -17)
                                  + (g.abs() + 16) * 2.0 ** -24), torch.zeros_like(d))
    y, ym = R.expert_products(d, ids, m2, True)
    _, ey = R.expert_products(ed, ids, m2, True)
    lim = ey.sum(1) + (I + 32 + ids.shape[1]) * 2.0 ** -24 * ym.sum(1)
    return y.sum(1), lim


DECODE = [(1, 1, 1, 16, 16, False, "plain"), (1, 8, 128, 256, 128, True, "plain"),
          (3, 2, 4, 48, 80, False, "dropped"), (16, 4, 8, 256, 128, True, "dropped"),
          (37, 4, 20, 272, 112, False, "dropped"), (40, 1, 7, 128, 128, True, "one"),
          (128, 8, 16, 256, 256, True, "plain"), (512, 8, 12, 64, 48, False, "plain"),
          (3, 20, 24, 48, 80, False, "dropped"), (4, 16, 16, 128, 1040, False, "plain"),
          (200, 4, 40, 336, 208, False, "dropped"), (100, 2, 60, 512, 384, True, "plain"),
          (200, 4, 40, 336, 512, False, "dropped"), (100, 2, 60, 512, 256, True, "plain"),
          (300, 3, 12, 256, 144, False, "one")]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,E,H,I,tiled,kind", DECODE)
def test_expert_decode(T, k, E, H, I, tiled, kind, dtype):
    from nvfp4_w4a4_quantized_amd import ops
    rng = np.random.default_rng(T + H + I)
    w1, w2 = R.make_weights(rng, E, 2 * I, H, std=0.1), R.make_weights(rng, E, H, I, std=0.1)
    ids = make_ids(rng, T, k, E, kind)
    prob = torch.from_numpy(rng.random((T, k)).astype(np.float32))
    prob[(ids < 0) | (ids >= E)] = float("nan")       # of no entry: must not matter
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(dtype)
    ref, lim = decode_ref(x, ids, torch.nan_to_num(prob), R.decode(*w1), R.decode(*w2))
    say("expert_decode", T, k, E, H, I, tiled, kind, dtype)
    a, b = held(*w1, tiled), held(*w2, tiled)
    # the workspace's old contents must not matter
    ws = torch.full((ops.moe_expert_decode_workspace_size(T, H, I, k),), 255, dtype=torch.uint8,
                    device="cuda")
    y = ops.moe_expert_decode(x.cuda(), ids.cuda(), prob.cuda(), E, I, a, b, workspace=ws)
    assert y.dtype == dtype
    bad = R.outside(y, ref, lim)
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} outside"
    assert torch.equal(y, ops.moe_expert_decode(x.cuda(), ids.cuda(), prob.cuda(), E, I, a, b))


def test_infinite_activations_stay_in_their_row():
    from nvfp4_w4a4_quantized_amd import ops
    rng = np.random.default_rng(10)
    w = held(*R.make_weights(rng, 1, 64, 256), True)
    x = torch.from_numpy(rng.standard_normal((6, 256)).astype(np.float32)).bfloat16().cuda()
    clean = ops.nvfp4_matvec(x, w)
    x[2, 5] = float("inf")
    x[4, 100] = float("nan")
    y = ops.nvfp4_matvec(x, w)
    for t in (0, 1, 3, 5):
        assert torch.equal(y[t], clean[t])
    assert not bool(torch.isfinite(y[2]).any()) and bool(torch.isnan(y[4]).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,n,k", [(3, 40, 272), (64, 6160, 272)])
def test_infinite_activations_give_the_formula(T, n, k, dtype):
    """An infinite x gives the infinities (and, against a zero weight or an
    infinity of the other sign, the NaN) of its formula, in both kernels."""
    from nvfp4_w4a4_quantized_amd import ops
    rng = np.random.default_rng(14)
    codes, scales, gs = R.make_weights(rng, 1, n, k)
    w = held(codes, scales, gs, False)
    x = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).to(dtype)
    x[0, k - 1] = float("inf")
    x[1, 7] = float("-inf")
    x[2, [3, 200]] = float("inf")
    m = R.decode(codes, scales, gs)[0]
    terms = x[:3].double().unsqueeze(1) * m.unsqueeze(0)
    y = ops.nvfp4_matvec(x.cuda(), w).cpu()[:3].double()
    ref = terms.sum(2)
    assert bool(torch.isinf(ref).any()) and bool(torch.isnan(ref).any())
    assert torch.equal(torch.nan_to_num(y, nan=7.0), torch.nan_to_num(ref, nan=7.0))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [2, 64])
def test_decode_of_an_infinite_intermediate(T, dtype):
    """One element of D overflows: y is infinite with its sign, NaN against a
    zero weight, and the other tokens are as they were."""
    from nvfp4_w4a4_quantized_amd import ops
    E, H, I, c = 8, 2048, 384, 77
    rng = np.random.default_rng(15)
    w1, w2 = R.make_weights(rng, E, 2 * I, H, std=0.1), R.make_weights(rng, E, H, I, std=0.1)
    ids = torch.full((T, 2), 3, dtype=torch.int32)
    ids[0] = torch.tensor([5, 6])
    keep = w1[0][5, [c, I + c]].clone()
    w1[0][5] = 0                                # expert 5: D is zero but at c
    w1[0][5, [c, I + c]] = keep
    prob = torch.full((T, 2), 0.5)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32) * 4).to(dtype)
    h, _ = R.expert_products(x[:1], ids[:1, :1], R.decode(*w1))
    if h[0, 0, c] < 0:                          # a positive gate, so silu(g) is g
        x[0] = -x[0]
        h = -h
    d = float(h[0, 0, c] * h[0, 0, I + c])
    assert h[0, 0, c] > 20 and abs(d) > 2
    a, b = held(*w1, True), held(*w2, True)
    clean = ops.moe_expert_decode(x.cuda(), ids.cuda(), prob.cuda(), E, I, a, b).cpu()
    prob[0, 0] = 3e38
    y = ops.moe_expert_decode(x.cuda(), ids.cuda(), prob.cuda(), E, I, a, b).cpu()
    col = R.decode(*w2)[5][:, c]
    want = torch.where(col == 0, float("nan"), np.sign(d) * col.sign() * np.inf)
    assert bool(torch.isnan(want).any()) and bool(torch.isinf(want).any())
    assert torch.equal(torch.nan_to_num(y[0].double(), nan=7.0), torch.nan_to_num(want, nan=7.0))
    assert torch.equal(y[1:], clean[1:])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,n,k", [(5, 70, 208), (16, 10247, 400), (64, 6145, 144)])
def test_any_alignment(T, n, k, dtype):
    """x at an odd element, its rows an odd distance apart, row-major weights
    and the output at odd addresses: the aligned call's bits, in both kernels."""
    from nvfp4_w4a4_quantized_amd import ops
    from nvfp4_w4a4_quantized_amd.ops import NvFp4Weights
    rng = np.random.default_rng(16)
    codes, scales, gs = R.make_weights(rng, 1, n, k)

    def shifted(t, by):
        t = t.cuda()
        flat = torch.zeros(t.numel() + 16, dtype=t.dtype, device="cuda")
        flat[by:by + t.numel()] = t.reshape(-1)
        return flat[by:by + t.numel()].view(t.shape)
    x = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).to(dtype).cuda()
    wide = torch.full((T, k + 21), float("nan"), dtype=dtype, device="cuda")
    wide[:, 5:5 + k] = x
    want = ops.nvfp4_matvec(x, held(codes, scales, gs, False))
    odd = NvFp4Weights(shifted(codes, 3), shifted(scales, 1), shifted(gs, 1))
    out = shifted(torch.zeros((T, n), dtype=dtype), 1)
    say("alignment", T, n, k, dtype)
    assert torch.equal(ops.nvfp4_matvec(wide[:, 5:5 + k], odd, out=out), want)


def test_no_tokens():
    from nvfp4_w4a4_quantized_amd import ops
    rng = np.random.default_rng(11)
    w1, w2 = held(*R.make_weights(rng, 4, 256, 128), True), held(*R.make_weights(rng, 4, 128, 128), True)
    x = torch.empty((0, 128), dtype=torch.bfloat16, device="cuda")
    ids = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    prob = torch.empty((0, 2), dtype=torch.float32, device="cuda")
    assert ops.moe_expert_decode(x, ids, prob, 4, 128, w1, w2).shape == (0, 128)
    assert ops.nvfp4_expert_matvec(x, ids, w1).shape == (0, 2, 256)


@pytest.mark.parametrize("T,n", [(3, 40), (64, 6160)])
def test_smallest_values(T, n):
    """Subnormal fp16 activations count in full, in both kernels."""
    from nvfp4_w4a4_quantized_amd import ops
    rng = np.random.default_rng(12)
    codes, scales, gs = R.make_weights(rng, 1, n, 256)
    gs[:] = 1.0
    w = held(codes, scales, gs, False)
    x = torch.from_numpy(rng.integers(-63, 64, (T, 256)).astype(np.float32) * 2.0 ** -24).half()
    m = R.decode(codes, scales, gs)[0]
    y = ops.nvfp4_matvec(x.cuda(), w, out_dtype=torch.float32)
    check(y, x.double() @ m.t(), x.double().abs() @ m.abs().t(), 256, "subnormal")


def test_rows_far_apart():
    """Rows of x more than 2^31 bytes apart in all."""
    from nvfp4_w4a4_quantized_amd import ops
    rng = np.random.default_rng(13)
    w = held(*R.make_weights(rng, 1, 6208, 64), False)
    big = torch.empty((64, 20_000_000), dtype=torch.bfloat16, device="cuda")
    x = big[:, 19_999_000:19_999_064]
    x.copy_(torch.from_numpy(rng.standard_normal((64, 64)).astype(np.float32)))
    near = ops.nvfp4_matvec(x.contiguous(), w, out_dtype=torch.float32).double()
    far = ops.nvfp4_matvec(x, w, out_dtype=torch.float32).double()
    # two kernels: 80 * 2^-23 of the terms' magnitudes, themselves below 30 in sum
    assert float((near - far).abs().max()) < 80 * 2.0 ** -23 * 30


def test_weights_beyond_four_gigabytes():
    """The last of 40 experts of 134 MB each, against it alone."""
    from nvfp4_w4a4_quantized_amd import ops
    from nvfp4_w4a4_quantized_amd.ops import NvFp4Weights
    E, n, k = 40, 16384, 16384
    codes = torch.randint(0, 256, (E, n, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.randint(40, 60, (E, n, k // 16), dtype=torch.uint8, device="cuda")
    gs = torch.full((E,), 0.01, device="cuda")
    w, last = NvFp4Weights(codes, scales, gs), NvFp4Weights(codes[E - 1:], scales[E - 1:], gs[E - 1:])
    x = torch.randn((2, k), device="cuda").bfloat16()
    ids = torch.full((2, 1), E - 1, dtype=torch.int32, device="cuda")
    y = ops.nvfp4_expert_matvec(x, ids, w, out_dtype=torch.float32)
    z = ops.nvfp4_matvec(x, last, out_dtype=torch.float32)
    assert float((y[:, 0] - z).norm() / z.norm()) < 1e-5


def empty_weights(groups, n, k):
    """All-zero codes with block scales of one, outer scales of one."""
    return (torch.zeros((groups, n, k // 2), dtype=torch.uint8),
            torch.full((groups, n, k // 16), 0x38, dtype=torch.uint8), torch.ones(groups))


def put(w, row, col, code, scale=0x38):
    """Element [:, row, col] = code (E2M1), its block's scale byte."""
    assert int(w[0][:, row, col // 2].max()) == 0
    w[0][:, row, col // 2] = code << (4 * (col % 2))
    w[1][:, row, col // 16] = scale


# sizes of the layer that reach, for FC2: the kernel with the sum (up to four
# tokens, up to eight), the direct kernel, and the kernel that shares D through LDS
REACH = [(1, 2, 8, 512, 128), (4, 2, 8, 512, 384), (8, 2, 8, 512, 128), (20, 2, 8, 512, 128),
         (100, 2, 8, 512, 128)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,E,H,I", REACH)
def test_decode_keeps_d_in_binary32(T, k, E, H, I, dtype):
    """Two elements of D that differ in their 21st significant bit and cancel
    in FC2: every value up to y is a binary32 one, so y is exact."""
    from nvfp4_w4a4_quantized_amd import ops
    w1, w2 = empty_weights(E, 2 * I, H), empty_weights(E, H, I)
    for c in (0, 1):
        put(w1, c, 0, 6, 0x50)              # gate: 4 * 8 = 32, so silu(32) = 32
        put(w1, I + c, 0, 2)                # up: 1
        put(w1, I + c, 16, 2, 2)            #   + 2^-8
    put(w1, I, 32, 1, 1)                    #   + 2^-10 * x, the first element alone
    for n in range(H):
        w2[0][:, n, 0] = 2 | (10 << 4)      # 8 D[0] - 8 D[1]
        w2[1][:, n, 0] = 0x50
    x = torch.zeros((T, H))
    x[:, [0, 16]] = 1.0
    x[:, 32] = 2.0 ** -10
    ids = torch.arange(T * k, dtype=torch.int32).view(T, k) % E
    prob = torch.full((T, k), 0.5)
    say("decode, D in binary32", T, k, E, H, I, dtype)
    y = ops.moe_expert_decode(x.to(dtype).cuda(), ids.cuda(), prob.cuda(), E, I, held(*w1, True),
                              held(*w2, True))
    # k entries of 8 * (32 * 2^-20) * 0.5
    assert torch.equal(y.cpu().double(), torch.full((T, H), k * 2.0 ** -13, dtype=torch.float64))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,E,H,I", REACH)
def test_decode_of_far_negative_gates(T, k, E, H, I, dtype):
    """Gates of -85 to -100, where binary32 exp(-g) overflows while silu(g) u p
    is a normal number.  Tolerance: D, the outer scale and the sum of k = 2
    equal terms round once each (2^-24), and D's two lower parts may count as
    zero below 2^-126, times the weights' 2^100 in each entry."""
    from nvfp4_w4a4_quantized_amd import ops
    w1, w2 = empty_weights(E, 2 * I, H), empty_weights(E, H, I)
    x = torch.zeros((T, H))
    for j in range(16):
        put(w1, j, j, 2)                    # gate j: x[j]
        put(w1, I + j, 16 + j, 7, 0x7E)     # up j: 6 * 448 * x[16 + j]
        x[:, j] = -85.0 - j
        x[:, 16 + j] = 2.0 ** 15
    for n in range(H):
        put(w2, n, n % 16, 2)
    w2[2][:] = 2.0 ** 100
    ids = torch.arange(T * k, dtype=torch.int32).view(T, k) % E
    prob = torch.full((T, k), 0.75)
    g, u = x[0, :16].double(), 2688.0 * x[0, 16:32].double()
    d = g * torch.exp(g) / (1.0 + torch.exp(g)) * u * 0.75
    assert bool((d.abs() > 2.0 ** -126).all())
    ref = (k * 2.0 ** 100 * d).repeat(H // 16).expand(T, H)
    say("decode, far negative gates", T, k, E, H, I, dtype)
    y = ops.moe_expert_decode(x.to(dtype).cuda(), ids.cuda(), prob.cuda(), E, I, held(*w1, True),
                              held(*w2, True))
    bad = R.outside(y, ref, 4 * 2.0 ** -24 * ref.abs() + k * 2 * 2.0 ** -26)
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} outside"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,k,E,H,I", REACH)
def test_decode_of_far_negative_gates_and_infinite_up(T, k, E, H, I, dtype):
    """silu(g) is below zero however far g is, so an up value past binary32's
    range makes D an infinity and no NaN."""
    from nvfp4_w4a4_quantized_amd import ops
    w1 = empty_weights(E, 2 * I, H)
    w1[2][:] = 2.0 ** 100
    gates = [-90.0, -100.0, -500.0, -800.0, -2.0 ** 40]
    x = torch.zeros((T, H))
    for j, g in enumerate(gates):
        put(w1, j, j, 2)
        put(w1, I + j, 16 + j, 7 if j % 2 else 15, 0x7E)   # +-2688 x[16 + j]
        x[:, j] = g * 2.0 ** -100
    for j in range(len(gates)):
        w2 = empty_weights(E, H, I)
        w2[0][:, :, j // 2] = 2 << (4 * (j % 2))
        xs = x.clone()
        xs[:, 16 + j] = 2.0 ** 20           # up: 2688 * 2^120, past the range
        say("decode, infinite up", T, k, E, H, I, dtype, gates[j])
        y = ops.moe_expert_decode(xs.to(dtype).cuda(), (torch.arange(T * k).view(T, k) % E).int().cuda(),
                                  torch.full((T, k), 0.5).cuda(), E, I, held(*w1, True),
                                  held(*w2, True)).cpu()
        assert torch.equal(y.float(), torch.full((T, H), -np.inf if j % 2 else np.inf))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,E,H,I", REACH)
@pytest.mark.parametrize("large", [True, False])
def test_decode_whose_partial_products_leave_the_range(large, T, k, E, H, I, dtype):
    """silu(g) u overflows (g = u = 2^70, p = 2^-100) or falls below the normal
    range (g = -79, u = 2^-30, p = 2^60) while D = silu(g) u p does neither.
    Tolerance: the exponential's (|g| + 16) 2^-24, and 2^-24 for each of D, the
    outer scale and the sum."""
    from nvfp4_w4a4_quantized_amd import ops
    w1, w2 = empty_weights(E, 2 * I, H), empty_weights(E, H, I)
    x = torch.zeros((T, H))
    if large:
        w1[2][:], prob, d, tol = 2.0 ** 60, 2.0 ** -100, 2.0 ** 40, 3
        put(w1, 0, 0, 2)
        put(w1, I, 16, 2)
        x[:, 0] = x[:, 16] = 2.0 ** 10
    else:
        w1[2][:], prob, tol = 2.0 ** -10, 2.0 ** 60, 79 + 16 + 3
        put(w1, 0, 0, 2, 0x70)              # 2^7
        put(w1, I, 16, 1, 1)                # 2^-10
        x[:, 0], x[:, 16] = -79.0 * 8, 2.0 ** -10
        d = -79.0 / (1.0 + np.exp(79.0)) * 2.0 ** 30
    w2[0][:, :, 0] = 2
    w2[2][:] = 2.0 ** -round(np.log2(abs(d)))
    ids = torch.arange(T * k, dtype=torch.int32).view(T, k) % E
    say("decode, partial products", large, T, k, E, H, I, dtype)
    y = ops.moe_expert_decode(x.to(dtype).cuda(), ids.cuda(), torch.full((T, k), prob).cuda(), E, I,
                              held(*w1, True), held(*w2, True))
    ref = torch.full((T, H), k * d * float(w2[2][0]), dtype=torch.float64)
    bad = R.outside(y, ref, tol * 2.0 ** -24 * ref.abs())
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} outside"


# the kernel with the sum, the separate sum with either kernel for FC2, and
# entries past the sixteenth in each
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,E,H,I", [(1, 3, 8, 512, 128), (2, 3, 8, 512, 640), (5, 3, 8, 512, 384),
                                       (6, 3, 8, 512, 384), (20, 3, 8, 512, 384),
                                       (100, 3, 8, 512, 384), (1, 20, 24, 512, 128), (4, 40, 40, 128, 384),
                                       (6, 20, 24, 512, 128), (40, 20, 24, 512, 384),
                                       (1, 1024, 1024, 128, 128)])
def test_decode_adds_whole_entries_in_their_order(T, k, E, H, I, dtype):
    """y is the sum over j, ascending, of the binary32 results of the entries:
    with three entries 1, 2^30 - 2^30 (its halves a stage apart in k) and 0 it
    is 1, with 2^30, 1, ..., -2^30 (more than sixteen entries) it is 0 as 2^30 +
    1 rounds to 2^30; any other order or grouping gives another sum."""
    from nvfp4_w4a4_quantized_amd import ops
    w1, w2 = empty_weights(E, 2 * I, H), empty_weights(E, H, I)
    far = I - 1 if I > 128 else 1           # another stage of 128, or the same one
    for c in (0, 16, far):
        put(w1, c, 0, 6, 0x50)              # gate 32: silu(32) = 32
        put(w1, I + c, 0, 2)                # up 1
    x = torch.zeros((T, H))
    x[:, 0] = 1.0
    big = w2[2]
    if k == 3:
        w2[0][0, :, 0] = 2                                       # expert 0: D[0]
        w2[0][1, :, 0] = 2                                       # expert 1: D[0] - D[far]
        w2[0][1, :, far // 2] |= 10 << (4 * (far % 2))
        big[0], big[1] = 2.0 ** -4, 2.0 ** 26
        want = 1.0
    else:
        w2[0][0, :, 0] = 2                                       # 2^30 from entry 0
        w2[0][1, :, 0] = 2                                       # 1 from entry 1
        w2[0][16, :, 0] = 10                                     # -2^30 from entry 16
        big[0], big[1], big[16] = 2.0 ** 26, 2.0 ** -4, 2.0 ** 26
        want = 0.0
    ids = torch.arange(k, dtype=torch.int32).expand(T, k).contiguous()
    say("decode, order of the sum", T, k, E, H, I, dtype)
    y = ops.moe_expert_decode(x.to(dtype).cuda(), ids.cuda(), torch.full((T, k), 0.5).cuda(), E, I,
                              held(*w1, True), held(*w2, True))
    assert torch.equal(y.cpu().double(), torch.full((T, H), want, dtype=torch.float64))


def shifted(t, by):
    """t on the device, `by` elements behind an aligned address."""
    flat = torch.zeros(t.numel() + 16, dtype=t.dtype, device="cuda")
    flat[by:by + t.numel()] = t.reshape(-1).cuda()
    return flat[by:by + t.numel()].view(t.shape)


def strided(x, left, right):
    """The rows of x inside rows of NaN: odd addresses and row distances."""
    wide = torch.full((x.shape[0], left + x.shape[1] + right), float("nan"), dtype=x.dtype, device="cuda")
    wide[:, left:left + x.shape[1]] = x.cuda()
    return wide[:, left:left + x.shape[1]]


# the direct kernel (a slot per entry, a slot per expert) and the kernel that
# shares x through LDS in its four shapes (16 or 32 columns, one group or two)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,E,n,K", [(2, 3, 8, 70, 208), (20, 3, 8, 70, 208), (60, 6, 50, 2049, 144),
                                       (60, 6, 50, 600, 528), (300, 4, 12, 4100, 144), (128, 4, 16, 500, 400)])
def test_expert_matvec_of_strided_rows_and_odd_addresses(T, k, E, n, K, dtype):
    from nvfp4_w4a4_quantized_amd import ops
    from nvfp4_w4a4_quantized_amd.ops import NvFp4Weights
    rng = np.random.default_rng(T + n + K)
    codes, scales, gs = R.make_weights(rng, E, n, K)
    ids = make_ids(rng, T, k, E, "dropped").cuda()
    x = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).to(dtype)
    say("expert_matvec, strides", T, k, E, n, K, dtype)
    want = ops.nvfp4_expert_matvec(x.cuda(), ids, held(codes, scales, gs, False))
    odd = NvFp4Weights(shifted(codes, 3), shifted(scales, 1), shifted(gs, 1))
    out = shifted(torch.zeros((T, k, n), dtype=dtype), 1)
    assert torch.equal(ops.nvfp4_expert_matvec(strided(x, 5, 8), ids, odd, out=out), want)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,E,H,I", [(3, 2, 8, 512, 384), (20, 2, 8, 512, 384), (100, 2, 8, 512, 384),
                                       (200, 4, 40, 640, 512)])
def test_decode_of_strided_rows_and_either_layout(T, k, E, H, I, dtype):
    """Rows at odd addresses, each projection in either layout, row-major weights
    at odd addresses: the bits of the plain call."""
    from nvfp4_w4a4_quantized_amd import ops
    from nvfp4_w4a4_quantized_amd.ops import NvFp4Weights
    rng = np.random.default_rng(T + H + I)
    w1, w2 = R.make_weights(rng, E, 2 * I, H, std=0.1), R.make_weights(rng, E, H, I, std=0.1)
    ids = make_ids(rng, T, k, E, "dropped").cuda()
    prob = torch.from_numpy(rng.random((T, k)).astype(np.float32)).cuda()
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(dtype)
    say("decode, strides and layouts", T, k, E, H, I, dtype)
    want = ops.moe_expert_decode(x.cuda(), ids, prob, E, I, held(*w1, False), held(*w2, False))

    def odd(w):
        return NvFp4Weights(shifted(w[0], 3), shifted(w[1], 1), shifted(w[2], 1))
    for a, b in ((held(*w1, True), held(*w2, False)), (held(*w1, False), held(*w2, True)),
                 (odd(w1), odd(w2)), (held(*w1, True), odd(w2))):
        y = ops.moe_expert_decode(strided(x, 3, 8), ids, prob, E, I, a, b,
                                  y=shifted(torch.zeros((T, H), dtype=dtype), 1))
        assert torch.equal(y, want)


def test_weights_beyond_four_gigabytes_through_lds():
    """As many entries of the last of 40 experts of 134 MB as take the kernel
    that shares x through LDS, against that expert alone."""
    from nvfp4_w4a4_quantized_amd import ops
    from nvfp4_w4a4_quantized_amd.ops import NvFp4Weights
    E, n, k = 40, 16384, 16384
    codes = torch.randint(0, 256, (E, n, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.randint(40, 60, (E, n, k // 16), dtype=torch.uint8, device="cuda")
    gs = torch.full((E,), 0.01, device="cuda")
    w, last = NvFp4Weights(codes, scales, gs), NvFp4Weights(codes[E - 1:], scales[E - 1:], gs[E - 1:])
    x = torch.randn((8, k), device="cuda").bfloat16()
    ids = torch.full((8, 1), E - 1, dtype=torch.int32, device="cuda")
    say("weights beyond 4 GB, LDS kernel")
    y = ops.nvfp4_expert_matvec(x, ids, w, out_dtype=torch.float32)
    z = ops.nvfp4_matvec(x, last, out_dtype=torch.float32)
    assert float((y[:, 0] - z).norm() / z.norm()) < 1e-5

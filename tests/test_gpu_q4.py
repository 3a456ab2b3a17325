"""4-bit weights with group scales (dfw_q4_*) against plain 64-bit arithmetic.

Tolerances, derived for the kernels' documented arithmetic (include/dfw.h):

* products (q - z) x of whole numbers below 16 and bf16 are exact in fp32.  A
  matrix instruction adds 16 of them to its accumulator; its terms are
  aligned to the largest and may be cut there instead of rounded, so each of
  the 17 terms loses at most 2^-23 of the largest one: 17 2^-23 times the sum
  of magnitudes so far.  At most 8 follow each other in a group (128 / 16), so
  a group's sum is off by at most 136 2^-23 of its sum of magnitudes S_g.
* the fp32 sum over groups adds one rounding per group and one per partial
  sum that is joined (at most 64 of them): (groups + 64) 2^-24 of S = sum s S_g.
* a bf16 result is rounded once: 2^-8 of its value.

Whole-number inputs whose sums stay below 2^24 leave nothing to round, so
there the result must be exact, whatever the order.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import lossless_entropy_coded_canonical_b200 as dfw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    dfw.lib()
    dfw.check()


def make(rows, cols, group, zeros, seed=0, whole=False):
    """Row-major codes [rows, cols] and bf16 scales / zero points per group."""
    rng = np.random.default_rng(seed)
    q = rng.integers(0, 16, (rows, cols)).astype(np.uint8)
    s = (2.0 ** rng.integers(-2, 3, (rows, cols // group)) if whole
         else torch.from_numpy(rng.uniform(0.001, 0.05, (rows, cols // group))).to(torch.bfloat16).double().numpy())
    z = rng.integers(0, 16, (rows, cols // group)).astype(np.uint8) if zeros else None
    return q, s, z


def to_gpu(q, s, z, group):
    codes = torch.from_numpy(q[:, 0::2] | (q[:, 1::2] << 4)).cuda().contiguous()
    return dfw.q4_pack(codes, torch.from_numpy(s).to(torch.bfloat16).cuda(), None if z is None else torch.from_numpy(z).cuda(),
                       group=group)


def weights(q, s, z, group):
    zz = 8.0 if z is None else np.repeat(z.astype(np.float64), group, 1)
    return np.repeat(s, group, 1) * (q.astype(np.float64) - zz)


def vectors(tokens, cols, seed=1, whole=False):
    rng = np.random.default_rng(seed)
    x = rng.integers(-3, 4, (tokens, cols)).astype(np.float64) if whole else rng.standard_normal((tokens, cols))
    return torch.from_numpy(x).to(torch.bfloat16)


def product_bound(w, x, group, dtype, y):
    groups = w.shape[1] // group
    mags = np.abs(x) @ np.abs(w).T
    b = (136 * 2.0 ** -23 + (groups + 64) * 2.0 ** -24) * mags
    return b + (2.0 ** -8 * (np.abs(y) + b) if dtype == torch.bfloat16 else 0.0) + 1e-35


SHAPES = [  # rows, cols, group: one group, ragged tiles, odd rows, more groups than a tile, long rows
    (1, 32, 32), (1, 128, 128), (16, 128, 64), (17, 160, 32), (15, 192, 64), (333, 96, 32), (64, 4096, 128), (257, 2080, 32),
    (48, 14336, 128), (1003, 11008, 64), (5, 65536, 128), (4100, 512, 32)]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("rows,cols,group", SHAPES)
def test_products(rows, cols, group, zeros):
    q, s, z = make(rows, cols, group, zeros, rows + cols)
    qw = to_gpu(q, s, z, group)
    w = weights(q, s, z, group)
    for tokens in (1, 2, 7, 8, 9, 16):
        x = vectors(tokens, cols, tokens)
        want = x.double().numpy() @ w.T
        for dtype in (torch.float32, torch.bfloat16):
            y = dfw.q4_gemv(qw, x.cuda(), out_dtype=dtype)
            assert y.dtype == dtype and y.shape == (tokens, rows)
            err = np.abs(y.double().cpu().numpy() - want)
            assert (err <= product_bound(w, x.double().numpy(), group, dtype, want)).all(), (tokens, dtype, err.max())


@pytest.mark.parametrize("rows,cols,group,zeros,tokens", [
    (70, 1024, 128, False, 1), (33, 416, 32, True, 3), (130, 4096, 64, True, 16), (16, 128, 128, False, 17), (50, 256, 64, True, 33),
    (40, 384, 128, True, 64), (2000, 64, 32, False, 5), (21, 32768, 32, True, 2), (19, 40960, 128, False, 16)])
def test_whole_numbers_are_exact(rows, cols, group, zeros, tokens):
    q, s, z = make(rows, cols, group, zeros, 7, whole=True)
    x = vectors(tokens, cols, 8, whole=True)
    want = x.double().numpy() @ weights(q, s, z, group).T
    assert np.abs(want).max() < 2 ** 22
    y = dfw.q4_gemv(to_gpu(q, s, z, group), x.cuda())
    assert np.array_equal(y.double().cpu().numpy(), want)


def test_each_code_and_column_lands_where_it_should():
    """Unit vectors read single weights back, exactly."""
    rows, cols, group = 37, 288, 32
    q, s, z = make(rows, cols, group, True, 3)
    qw, w = to_gpu(q, s, z, group), weights(q, s, z, group)
    for k0 in range(0, cols, 64):
        k = np.arange(k0, min(k0 + 64, cols))
        x = torch.zeros(len(k), cols, dtype=torch.bfloat16)
        x[np.arange(len(k)), k] = 1.0
        assert np.array_equal(dfw.q4_gemv(qw, x.cuda()).double().cpu().numpy(), w[:, k].T)


def test_dequantise():
    for rows, cols, group, zeros in ((1, 32, 32, True), (35, 352, 32, True), (64, 512, 128, False), (18, 192, 64, True)):
        q, s, z = make(rows, cols, group, zeros, 5)
        got = dfw.q4_dequantise(to_gpu(q, s, z, group))
        want = torch.from_numpy(weights(q, s, z, group)).float().to(torch.bfloat16)  # 12 bits: fp32 is exact
        assert torch.equal(got.cpu(), want)


def quantised(w, group, zeros):
    """The formula of include/dfw.h in 64 bits (the bf16 scale rounded from fp32)."""
    rows, cols = w.shape
    g = w.reshape(rows, cols // group, group)
    lo, hi = np.minimum(g.min(-1), 0), np.maximum(g.max(-1), 0)
    bad = ~np.isfinite(g).all(-1)
    with np.errstate(all="ignore"):
        rng = (hi.astype(np.float32) / np.float32(15) - lo.astype(np.float32) / np.float32(15)) if zeros else \
            np.abs(g).max(-1).astype(np.float32) / np.float32(7)
        s = torch.from_numpy(np.where(bad, np.float32(np.nan), rng)).to(torch.bfloat16).double().numpy()
        live = s > 0
        z = np.where(live, np.clip(np.rint(-lo / s), 0, 15), 0) if zeros else np.full(s.shape, 8.0)
        q = np.where(live[..., None], np.clip(np.rint(g / s[..., None]) + z[..., None], 0, 15), z[..., None])
    return q.reshape(rows, cols).astype(np.uint8), s, z.astype(np.uint8) if zeros else None


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("rows,cols,group,kind", [
    (1, 32, 32, "normal"), (40, 4096, 128, "normal"), (77, 352, 32, "positive"), (23, 704, 64, "special"), (16, 128, 128, "tiny"),
    (31, 640, 128, "ties")])
def test_quantise_is_the_formula(rows, cols, group, kind, zeros):
    rng = np.random.default_rng(rows)
    w = rng.standard_normal((rows, cols)) * 0.02
    if kind == "positive":
        w = np.abs(w) + 0.01
    if kind == "tiny":
        w *= 1e-38
    if kind == "ties":  # multiples of a quarter of the scale: half steps among them
        w = rng.integers(-28, 29, (rows, cols)) / 4.0
        w[:, ::group] = 7.0
    w = torch.from_numpy(w).to(torch.bfloat16)
    if kind == "special":
        w[0, :group] = 0.0
        w[1, 3] = float("inf")
        w[2, 5] = float("-inf")
        w[3, group] = float("nan")
        w[4, :] = 3.3895e38
        w[5, 0], w[5, 1] = 3.3895e38, -3.3895e38
    q, s, z = quantised(w.double().numpy(), group, zeros)
    got = dfw.q4_quantise(w.cuda(), group=group, zeros=zeros)
    want = to_gpu(q, s, z, group)
    assert got.packed.numel() == want.packed.numel()
    if kind == "special":  # NaN scales: compare the values they stand for
        a, b = dfw.q4_dequantise(got).cpu(), dfw.q4_dequantise(want).cpu()
        assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))
        assert a[1, :group].isnan().all() and not a[1, group:].isnan().any()
    else:
        assert torch.equal(got.packed, want.packed)


def test_quantise_takes_row_strides_and_any_alignment():
    w = (torch.randn(40, 1000, device="cuda") * 0.1).to(torch.bfloat16)
    for view in (w[:, 4:4 + 128], w[:, 1:1 + 128], w[::3, 64:64 + 256]):
        a, b = dfw.q4_quantise(view, group=64, zeros=True), dfw.q4_quantise(view.contiguous(), group=64, zeros=True)
        assert torch.equal(a.packed, b.packed)


def test_vector_and_result_strides():
    rows, cols, group = 61, 512, 128
    q, s, z = make(rows, cols, group, False, 1)
    qw = to_gpu(q, s, z, group)
    base = torch.randn(9, cols + 25, device="cuda").to(torch.bfloat16)
    for off in (0, 1, 8, 25):  # odd offsets: only 2-byte aligned
        x = base[:, off:off + cols]
        want = dfw.q4_gemv(qw, x.contiguous())
        assert torch.equal(dfw.q4_gemv(qw, x), want)
        assert torch.equal(dfw.q4_gemv(qw, x[4]), want[4])
        wide = torch.full((9, rows + 7), 5.0, device="cuda")
        out = dfw.q4_gemv(qw, x, out=wide[:, 3:3 + rows])
        assert torch.equal(out, want) and (wide[:, :3] == 5).all() and (wide[:, 3 + rows:] == 5).all()
    odd = torch.full((rows + 2,), 7.0, device="cuda", dtype=torch.bfloat16)
    dfw.q4_gemv(qw, base[0, :cols], out=odd[1:1 + rows])
    assert torch.equal(odd[1:1 + rows], dfw.q4_gemv(qw, base[0, :cols], out_dtype=torch.bfloat16)) and odd[0] == 7 and odd[-1] == 7


def test_a_nan_stays_with_its_vector_and_its_row():
    rows, cols, group = 50, 384, 128
    q, s, z = make(rows, cols, group, True, 2)
    x = vectors(6, cols, 4).cuda()
    want = dfw.q4_gemv(to_gpu(q, s, z, group), x)
    x[2, 77] = float("nan")
    x[4, 5] = float("inf")
    got = dfw.q4_gemv(to_gpu(q, s, z, group), x)
    keep = [0, 1, 3, 5]
    assert got[2].isnan().all() and not got[4].isfinite().any() and torch.equal(got[keep], want[keep])
    s2 = s.copy()
    s2[9, 1] = np.nan
    got = dfw.q4_gemv(to_gpu(q, s2, z, group), vectors(6, cols, 4).cuda())
    rest = [r for r in range(rows) if r != 9]
    assert got[:, 9].isnan().all() and torch.equal(got[:, rest], want[:, rest])


def test_no_vectors_and_too_many():
    q, s, z = make(16, 128, 128, False)
    qw = to_gpu(q, s, z, 128)
    assert dfw.q4_gemv(qw, torch.zeros(0, 128, dtype=torch.bfloat16, device="cuda")).shape == (0, 16)
    with pytest.raises(dfw.DfwError) as ei:
        dfw.q4_gemv(qw, torch.zeros(65, 128, dtype=torch.bfloat16, device="cuda"))
    assert ei.value.status == dfw.EINVAL
    with pytest.raises(ValueError):
        dfw.q4_gemv(qw, torch.zeros(1, 256, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        dfw.q4_gemv(qw, torch.zeros(128, 4, dtype=torch.bfloat16, device="cuda").t())  # columns not contiguous
    with pytest.raises(dfw.DfwError):
        dfw.q4_gemv(qw, torch.zeros(1, 128, dtype=torch.bfloat16, device="cuda").expand(4, 128))  # rows on top of each other
    with pytest.raises(TypeError):
        dfw.q4_gemv(qw, torch.zeros(1, 128, device="cuda"))


def test_repeats_streams_and_graphs():
    """Two streams at once and a graph replayed on new inputs give the bits of
    plain calls (the kernels keep no state between calls)."""
    rows, cols, group = 2051, 4096, 128
    q, s, z = make(rows, cols, group, True, 11)
    qw = to_gpu(q, s, z, group)
    xs = [vectors(t, cols, t).cuda() for t in (1, 4, 16)]
    want = [dfw.q4_gemv(qw, x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[dfw.q4_gemv(qw, x, stream=st) for x in xs] for _ in range(5) for st in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
    x, y = torch.zeros_like(xs[1]), torch.empty(4, rows, device="cuda")
    dfw.q4_gemv(qw, x, out=y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dfw.q4_gemv(qw, x, out=y)
    for scale in (1.0, 2.0):
        x.copy_(xs[1] * scale)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[1] * scale)  # a power of two: exact


def test_quantise_rounds_every_pair_of_bf16_significands():
    """Every quotient a / b of 8-bit significands, at six powers of two: ties
    and the quotients next to them, with scales down to the smallest bf16."""
    a = torch.arange(128, 256, dtype=torch.float64)
    for shift in (-6, -3, -2, -1, 0, 1):
        for expo in (-9, 100, -132):  # of the scale: ordinary, large, below the normal range
            # column 0 of a row fixes the scale at b 2^expo: 7 times it, exactly a bf16 or not, is rounded back to it
            b = torch.arange(128, 256, dtype=torch.float64)
            w = torch.zeros(128, 160, dtype=torch.float64)
            w[:, 0] = 7 * b * 2.0 ** (expo - 7)
            w[:, 1:129] = a[None, :] * 2.0 ** (shift + expo - 7)
            w = w.clamp(max=3e38).to(torch.bfloat16)
            q, s, z = quantised(w.double().numpy(), 32, False)
            got = dfw.q4_quantise(w.cuda(), group=32)
            assert torch.equal(got.packed, to_gpu(q, s, z, 32).packed), (shift, expo)


def test_a_captured_call_behind_a_copy_a_fill_and_another_stream():
    """What precedes a call inside a graph need not be a kernel, nor one thing."""
    q, s, z = make(500, 1024, 64, True, seed=5, whole=True)
    qw = to_gpu(q, s, z, 64)
    src, ids = vectors(3, 1024, seed=6, whole=True).cuda(), torch.tensor([2, 0, 1], device="cuda")
    want = src.double().cpu() @ torch.from_numpy(weights(q, s, z, 64)).T
    x, y1, y2 = torch.empty_like(src), torch.empty(3, 500, device="cuda"), torch.empty(3, 500, device="cuda")
    picked, grad = torch.empty_like(src), torch.empty(3, 1024, device="cuda")
    side = torch.cuda.Stream()

    def calls():
        x.copy_(src)  # a copy, then a product
        dfw.q4_gemv(qw, x, out=y1)
        y2.zero_()  # a fill, then a product on each of two streams
        side.wait_stream(torch.cuda.current_stream())
        dfw.q4_gemv(qw, x, out=y2, stream=side)
        dfw.embed_rows(x, ids, out=picked)
        torch.cuda.current_stream().wait_stream(side)
        return dfw.embed_grad(ids, picked, 3, out=grad)  # behind both streams

    calls()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    for scale in (1.0, 2.0):
        src.mul_(scale)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y1.double().cpu(), want * scale) and torch.equal(y2, y1)
        assert torch.equal(picked, src[ids]) and torch.equal(grad, src.float())
    dfw.check()


def test_offsets_past_32_bits():
    """A matrix of 9.2e9 weights in 4.7 GB, all zero but for its ends."""
    rows, cols = 140001, 65536
    w = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    rng = torch.Generator(device="cuda").manual_seed(3)
    for part in (w[:5], w[-20:]):
        part.copy_(torch.randint(-7, 8, part.shape, generator=rng, device="cuda"))
        part[:, ::128] = 7  # scale 1: the codes are the weights
    q = dfw.q4_quantise(w)
    assert q.packed.numel() > 1 << 32
    x = torch.randint(-2, 3, (2, cols), generator=rng, device="cuda").to(torch.bfloat16)
    y = dfw.q4_gemv(q, x)
    for part in (slice(0, 5), slice(rows - 20, rows)):
        assert torch.equal(y[:, part].double(), x.double() @ w[part].double().T)
    assert not y[:, 5:-20].any()
    back = dfw.q4_dequantise(q)
    assert torch.equal(back[:5], w[:5]) and torch.equal(back[-20:], w[-20:]) and not back[5:-20].any()
    del back, w
    codes = torch.full((rows, cols // 2), 0x88, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(rows, cols // 128, dtype=torch.bfloat16, device="cuda")
    codes[-1, -1], scales[-1, -1] = 0xF8, 2.0
    y = dfw.q4_gemv(dfw.q4_pack(codes, scales), torch.ones(cols, dtype=torch.bfloat16, device="cuda"))
    assert y[-1] == 14.0 and not y[:-1].any()


@pytest.mark.parametrize("x_exp,s_exp", [(-130, 100), (-133, 120), (100, -110), (-60, -50), (0, -118), (120, 0), (-126, 127)])
def test_vectors_and_scales_far_from_one(x_exp, s_exp):
    """Whole numbers times powers of two, vectors below the normal range among
    them: exact as long as no result is below 2^-120 (the sums are kept over
    64), infinite where the result, not a sum on the way, is past fp32."""
    rows, cols, group = 70, 640, 64
    q, s, z = make(rows, cols, group, True, 31)
    s = np.full(s.shape, 2.0 ** s_exp)
    for tokens in (1, 12):
        x = vectors(tokens, cols, 5, whole=True)
        with np.errstate(over="ignore"):
            want = (x.double().numpy() @ weights(q, s, z, group).T * 2.0 ** x_exp).astype(np.float32)
        y = dfw.q4_gemv(to_gpu(q, s, z, group), (x.double() * 2.0 ** x_exp).to(torch.bfloat16).cuda())
        assert np.array_equal(y.cpu().numpy(), want)

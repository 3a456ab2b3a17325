"""Embedding rows from a coded scope and from a bf16 table, and the table's
gradient, against plain 64-bit arithmetic.

A row is one rounding of scale x weight, so it must be equal bit for bit: the
fp32 product of a scale of at most 16 bits and a bf16 weight is exact, that of
a scale of more bits is exact in 64 bits.
The gradient is a sum of k terms in fp32, in some order: off by at most
(k + 1) 2^-24 times the scaled sum of magnitudes (one rounding per addition
and one for the scale), plus 2^-8 of the value for a bf16 result, and exactly
rounded once where the sum itself is exact.  Whole numbers leave nothing to
round.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import lossless_entropy_coded_canonical_b200 as dfw
import workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    dfw.lib()
    dfw.check()


@pytest.fixture(autouse=True)
def _clean():
    yield
    dfw.check()  # no test leaves a status behind


def table(n, kind="normal", seed=0):
    """n bf16 patterns (uint16)."""
    rng = np.random.default_rng(seed)
    if kind == "single":  # one exponent: no stream
        return ((rng.integers(0, 2, n) << 15) | (119 << 7) | rng.integers(0, 128, n)).astype(np.uint16)
    if kind == "bitmap":  # two exponents: 1-bit codes
        return ((rng.integers(0, 2, n) << 15) | (rng.integers(119, 121, n) << 7) | rng.integers(0, 128, n)).astype(np.uint16)
    if kind == "uniform":  # every pattern: NaN and infinities among them, codes of 8 bits
        u = rng.integers(0, 1 << 16, n).astype(np.uint16)
        u[:256] = np.arange(256) << 7
        return u
    if kind == "long":  # exponent counts fall like Fibonacci numbers: codewords far longer than the fast table's key
        e = np.concatenate([np.full(f, 100 + i) for i, f in enumerate(fib_counts(n))])[:n]
        return ((rng.permutation(e).astype(np.int64) << 7) | rng.integers(0, 128, n)).astype(np.uint16)
    f = (rng.standard_normal(n) * 0.02).astype(np.float32)
    return workloads.as_u16_numpy(torch.from_numpy(f).to(torch.bfloat16))


def fib_counts(n):
    c = [1, 1]
    while sum(c) < n:
        c.append(c[-1] + c[-2])
    return c


def coded(u, fast_bits=0):
    enc = dfw.encode(u)
    return dfw.DeviceLanes.upload(enc, dfw.plan_lanes(enc, fast_bits=fast_bits))


def ids_for(rows, tokens, seed=0, dtype=torch.int64, pads=True):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, rows, tokens)
    ids[0], ids[-1] = 0, rows - 1
    if pads and tokens > 4:
        ids[1], ids[tokens // 2] = -1, -(1 << 30)
    return torch.from_numpy(ids).to(dtype)


def rows_of(u, first, rows, dim, ids, scale):
    """scale x row in 64 bits, rounded once to bf16; padding gives zeros."""
    w = torch.from_numpy(u.view(np.int16)).view(torch.bfloat16)[first: first + rows * dim].view(rows, dim)
    out = torch.zeros(*ids.shape, dim, dtype=torch.bfloat16)
    keep = (ids >= 0) & (ids < rows)
    sel = w[ids[keep].long()]
    out[keep] = sel if scale == 1.0 else (sel.double() * scale).float().to(torch.bfloat16)
    return out


def same(a, b):
    """Equal bits, but for the payload of a NaN that was multiplied."""
    a, b = a.cpu(), b.cpu()
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(torch.where(a.isnan(), 0, a.view(torch.int16)),
                                                             torch.where(b.isnan(), 0, b.view(torch.int16)))


SHAPES = [  # rows, dim, first: whole groups, shared groups, odd rows, rows that start anywhere, long and tiny rows
    (50, 4096, 0), (300, 1024, 0), (37, 2048, 0), (41, 6144, 2048), (90, 64, 0), (1000, 1, 0), (33, 1000, 0), (19, 2049, 3),
    (7, 5001, 77), (64, 192, 64), (5, 12345, 1), (3, 40000, 4096), (2000, 31, 5), (11, 4096, 1024), (9, 2080, 8)]


@pytest.mark.parametrize("rows,dim,first", SHAPES)
@pytest.mark.parametrize("tokens", [1, 70, 3000])
def test_coded_rows(rows, dim, first, tokens):
    u = table(first + rows * dim + 11, seed=dim)
    dl = coded(u)
    for scale, dtype in ((1.0, torch.int64), (-45.25, torch.int32)):
        ids = ids_for(rows, tokens, tokens, dtype)
        got = dfw.embed_lanes(dl, ids.cuda(), dim, scale=scale, first=first, rows=rows)
        assert torch.equal(got.cpu().view(torch.int16), rows_of(u, first, rows, dim, ids, scale).view(torch.int16)), scale


@pytest.mark.parametrize("kind", ["single", "bitmap", "uniform", "long"])
@pytest.mark.parametrize("rows,dim,tokens,fast_bits", [(40, 2048, 9, 0), (40, 2048, 4000, 8), (33, 1000, 700, 12), (500, 64, 3, 9)])
def test_coded_rows_of_other_codes(kind, rows, dim, tokens, fast_bits):
    u = table(rows * dim, kind, dim + tokens)
    dl = coded(u, fast_bits)
    ids = ids_for(rows, tokens, 5)
    assert torch.equal(dfw.embed_lanes(dl, ids.cuda(), dim).cpu().view(torch.int16), rows_of(u, 0, rows, dim, ids, 1.0).view(torch.int16))
    assert same(dfw.embed_lanes(dl, ids.cuda(), dim, scale=0.5), rows_of(u, 0, rows, dim, ids, 0.5))


@pytest.mark.parametrize("rows,dim,tokens,ld", [(50, 4096, 33, 0), (300, 129, 1000, 0), (7, 1, 5, 0), (64, 1024, 2000, 8), (20, 72, 77, 3),
                                                (10, 20000, 4, 0)])
def test_table_rows(rows, dim, tokens, ld):
    u = table(rows * (dim + ld), seed=dim)
    w = torch.from_numpy(u.view(np.int16)).view(torch.bfloat16).cuda().view(rows, dim + ld)[:, :dim]
    flat = workloads.as_u16_numpy(w.contiguous().cpu())
    for scale, dtype in ((1.0, torch.int32), (31.625, torch.int64)):
        ids = ids_for(rows, tokens, 3, dtype)
        assert torch.equal(dfw.embed_rows(w, ids.cuda(), scale=scale).cpu().view(torch.int16),
                           rows_of(flat, 0, rows, dim, ids, scale).view(torch.int16))


def test_a_scale_of_many_bits():
    u = table(100 * 512)
    ids = ids_for(100, 60, pads=False)
    w = torch.from_numpy(u.view(np.int16)).view(torch.bfloat16).view(100, 512)
    want = w[ids].double().numpy() * np.float64(np.float32(np.pi))
    for got in (dfw.embed_lanes(coded(u), ids.cuda(), 512, scale=np.pi), dfw.embed_rows(w.cuda(), ids.cuda(), scale=np.pi)):
        err = np.abs(got.cpu().double().numpy() - want)
        assert (err <= (2.0 ** -8 + 2.0 ** -23) * np.abs(want)).all()


@pytest.mark.parametrize("tokens", [6, 4000])
def test_ids_past_the_table_are_reported(tokens):
    u = table(50 * 256)
    ids = ids_for(50, tokens, 1)
    ids[2], ids[3] = 50, (1 << 40) + 3  # the second names row 3 to a 32-bit reader
    w = torch.from_numpy(u.view(np.int16)).view(torch.bfloat16).cuda().view(50, 256)
    want = rows_of(u, 0, 50, 256, ids, 1.0).view(torch.int16)
    dy = torch.ones(tokens, 8, device="cuda")
    for call in (lambda: dfw.embed_lanes(coded(u), ids.cuda(), 256), lambda: dfw.embed_rows(w, ids.cuda())):
        out = call()
        assert dfw.status_bits() == (dfw.ECORRUPT, dfw.ST_INDEX)
        assert torch.equal(out.cpu().view(torch.int16), want)
    grad = dfw.embed_grad(ids.cuda(), dy, 50)
    assert dfw.status_bits() == (dfw.ECORRUPT, dfw.ST_INDEX)
    keep = ids[(ids >= 0) & (ids < 50)]
    assert torch.equal(grad[:, 0].cpu(), torch.bincount(keep, minlength=50).float())


def test_rows_outside_are_left_alone():
    """Strided results, odd alignments, and the row behind the last token."""
    u = table(64 * 520)
    dl = coded(u)
    w = torch.from_numpy(u.view(np.int16)).view(torch.bfloat16).cuda().view(64, 520)
    ids = ids_for(64, 9)
    want = rows_of(u, 0, 64, 520, ids, 1.0).cuda()
    for off in (0, 1, 8, 16):
        for call in (lambda o: dfw.embed_lanes(dl, ids.cuda(), 520, out=o), lambda o: dfw.embed_rows(w, ids.cuda(), out=o)):
            buf = torch.full((10, 560), 3.0, dtype=torch.bfloat16, device="cuda")
            call(buf[:9, off: off + 520])
            assert torch.equal(buf[:9, off: off + 520], want)
            buf[:9, off: off + 520] = 3.0
            assert (buf == 3.0).all()


def test_shapes_and_empty():
    u = table(10 * 96)
    dl = coded(u)
    w = torch.from_numpy(u.view(np.int16)).view(torch.bfloat16).cuda().view(10, 96)
    ids = ids_for(10, 12).view(3, 4)
    want = rows_of(u, 0, 10, 96, ids, 1.0)
    assert torch.equal(dfw.embed_lanes(dl, ids.cuda(), 96).cpu(), want) and torch.equal(dfw.embed_rows(w, ids.cuda()).cpu(), want)
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    assert dfw.embed_lanes(dl, none, 96).shape == (0, 96) and dfw.embed_rows(w, none).shape == (0, 96)
    assert (dfw.embed_grad(none, torch.zeros(0, 96, device="cuda"), 4) == 0).all()
    with pytest.raises(dfw.DfwError):
        dfw.embed_lanes(dl, ids.cuda(), 96, rows=11)
    with pytest.raises(ValueError):
        dfw.embed_lanes(dl, ids.cuda().t(), 96)
    with pytest.raises(TypeError):
        dfw.embed_rows(w, ids.cuda().to(torch.int16))
    with pytest.raises(ValueError):
        dfw.embed_rows(w, ids.cuda(), out=torch.empty(3, 4, 95, dtype=torch.bfloat16, device="cuda"))


@pytest.mark.parametrize("tokens", [5, 3000])
def test_a_damaged_plan_is_reported(tokens):
    u = table(100 * 2048)
    for damage in ("chunk_bits", "group_start", "lut", "stream"):
        dl = coded(u)
        ids = torch.full((tokens,), 7, dtype=torch.int64, device="cuda")
        if damage == "chunk_bits":
            dl.chunk_bits[7 * 32 + 3] += 1
        elif damage == "group_start":
            dl.group_start[8] += 1
        elif damage == "stream":
            dl.stream.fill_(0xA7)
        else:
            dl.lut.fill_(-1)
        out = torch.full((tokens, 2048), 9.0, dtype=torch.bfloat16, device="cuda")
        dfw.embed_lanes(dl, ids, 2048, out=out)
        status, bits = dfw.status_bits()
        assert status == dfw.ECORRUPT and bits & (dfw.ST_COUNT | dfw.ST_RANGE | dfw.ST_LUT), damage
        assert (out == 9.0).all(), damage  # a damaged group writes nothing


def test_rows_of_a_decode_whose_last_scope_is_damaged():
    """The last launch of a sequence finds its table malformed and decodes
    nothing; what follows it must still wait for the launches before it."""
    u = table(20000 * 2048)
    scopes = [coded(u)] * 40 + [coded(table(2048))]  # a launch takes 40
    scopes[-1].lut.fill_(-1)
    assert dfw.decode_lanes_seq_launches(scopes) == 2
    ids = torch.arange(19999, 0, -7, dtype=torch.int64, device="cuda")
    want = rows_of(u, 0, 20000, 2048, ids.cpu(), 1.0)
    for _ in range(3):
        out = torch.zeros(20000, 2048, dtype=torch.bfloat16, device="cuda")
        dfw.decode_lanes_seq(scopes, out.view(-1))
        rows = dfw.embed_rows(out, ids)
        assert dfw.status_bits() == (dfw.ECORRUPT, dfw.ST_LUT)
        assert same(rows, want)


# ------------------------------------------------------------------ gradient

def grad_of(ids, dy, rows, scale):
    """(gradient, sum of magnitudes, tokens per row) in 64 bits."""
    keep = (ids >= 0) & (ids < rows)
    i, d = ids[keep].long(), dy.double().cpu()[keep]
    g = torch.zeros(rows, dy.shape[1], dtype=torch.float64).index_add_(0, i, d) * scale
    m = torch.zeros(rows, dy.shape[1], dtype=torch.float64).index_add_(0, i, d.abs()) * abs(scale)
    return g, m, torch.bincount(i, minlength=rows).double()[:, None]


def check_grad(got, ids, dy, rows, scale, base=None):
    g, m, k = grad_of(ids, dy, rows, scale)
    bound = (k + 1) * 2.0 ** -24 * m
    if base is not None:
        g = g + base.double().cpu()
        bound = bound + 2.0 ** -24 * (g.abs() + bound)
    if got.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (g.abs() + bound)
    err = (got.double().cpu() - g).abs()
    assert (err <= bound + 1e-40).all(), float((err - bound).max())
    if base is None:
        assert (got.cpu()[k[:, 0] == 0] == 0).all()


GRADS = [  # rows, dim, tokens, how the ids are spread
    (1000, 129, 33, "any"), (50, 64, 1, "any"), (1, 8, 500, "any"), (7, 1024, 5000, "any"), (5000, 72, 4000, "any"),
    (300, 1, 2000, "any"), (40, 5000, 100, "any"), (4097, 16, 9000, "zipf"), (100, 33, 20000, "one"), (257, 256, 70000, "zipf"),
    (64, 8, 200, "pads"), (100000, 8, 3000, "any"), (33, 2056, 1000, "sorted")]


def grad_ids(rows, tokens, spread, seed=0):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, rows, tokens)
    if spread == "zipf":
        ids = np.minimum((np.exp(rng.random(tokens) * np.log(rows + 1)) - 1).astype(np.int64), rows - 1)
    if spread == "one":
        ids[:] = rows // 2
    if spread == "sorted":
        ids = np.sort(ids)
    ids = torch.from_numpy(ids)
    if tokens > 10:
        ids[::17] = -1
    if spread == "pads":
        ids[:] = -1
    return ids


@pytest.mark.parametrize("rows,dim,tokens,spread", GRADS)
def test_gradient(rows, dim, tokens, spread):
    ids = grad_ids(rows, tokens, spread)
    dy = torch.randn(tokens, dim, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    for dy_dtype, out_dtype, id_dtype, scale in ((torch.float32, torch.float32, torch.int64, 1.0),
                                                 (torch.bfloat16, torch.bfloat16, torch.int32, -45.25),
                                                 (torch.bfloat16, torch.float32, torch.int64, 0.1),
                                                 (torch.float32, torch.bfloat16, torch.int32, 64.0)):
        d, i = dy.to(dy_dtype), ids.cuda().to(id_dtype)
        got = dfw.embed_grad(i, d, rows, scale=scale, out_dtype=out_dtype)
        check_grad(got, ids, d, rows, float(np.float32(scale)))
        assert torch.equal(got, dfw.embed_grad(i, d, rows, scale=scale, out_dtype=out_dtype)), "not reproducible"


@pytest.mark.parametrize("rows,dim,tokens,spread", [(97, 40, 3000, "any"), (97, 17, 40000, "zipf"), (3, 264, 9000, "any"), (5000, 8, 100, "any")])
def test_gradient_of_whole_numbers_is_exact(rows, dim, tokens, spread):
    ids = grad_ids(rows, tokens, spread, 3)
    dy = torch.randint(-8, 9, (tokens, dim), generator=torch.Generator("cuda").manual_seed(2), device="cuda").float()
    want, _, _ = grad_of(ids, dy, rows, 2.0)
    for d in (dy, dy.to(torch.bfloat16)):
        assert torch.equal(dfw.embed_grad(ids.cuda(), d, rows, scale=2.0).double().cpu(), want)


@pytest.mark.parametrize("tokens", [128, 129, 1024, 1025, 8192, 8193, 16385, 32768, 32769, 65536, 65537, 131073, 140000])
@pytest.mark.parametrize("rows", [90, 65535, 65536])
def test_gradient_at_every_change_of_its_cut(rows, tokens):
    """The sizes where the launches, blocks, windows and the width of a sorted
    token change, one token behind each, exact in whole numbers."""
    ids = grad_ids(rows, tokens, "zipf", tokens)
    ids[-1] = rows - 1
    dy = torch.randint(-3, 4, (tokens, 8), generator=torch.Generator("cuda").manual_seed(5), device="cuda").float()
    want, _, _ = grad_of(ids, dy, rows, 1.0)
    assert torch.equal(dfw.embed_grad(ids.cuda(), dy.to(torch.bfloat16), rows).double().cpu(), want)


def test_the_most_tokens_and_too_many():
    ids = torch.full((1 << 20,), 3, dtype=torch.int32, device="cuda")
    ids[: 1 << 19] = torch.arange(1 << 19, dtype=torch.int32, device="cuda") % 100000
    dy = torch.ones(1 << 20, 1, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(dfw.embed_grad(ids, dy, 100000)[:, 0].cpu(), torch.bincount(ids.long().cpu(), minlength=100000).float())
    with pytest.raises(dfw.DfwError):
        dfw.embed_grad(ids.new_zeros((1 << 20) + 1), dy.new_ones((1 << 20) + 1, 1), 10)


@pytest.mark.parametrize("rows,dim,tokens,spread", [(200, 48, 150, "any"), (50, 129, 5000, "zipf"), (300, 16, 1, "any"), (20, 8, 30, "pads")])
def test_gradient_accumulates(rows, dim, tokens, spread):
    ids = grad_ids(rows, tokens, spread, 4)
    dy = torch.randn(tokens, dim, device="cuda")
    hit = torch.zeros(rows, dtype=torch.bool)
    hit[ids[ids >= 0]] = True
    for dtype in (torch.float32, torch.bfloat16):
        base = torch.randn(rows, dim, device="cuda").to(dtype)
        base[~hit.cuda()] = float("nan")  # rows without tokens are not touched
        out = base.clone()
        dfw.embed_grad(ids.cuda(), dy, rows, scale=3.0, out=out, accumulate=True)
        assert torch.equal(out[~hit.cuda()].view(torch.int16), base[~hit.cuda()].view(torch.int16))
        if hit.any():
            check_grad(torch.where(hit.cuda()[:, None], out, 0.0).to(dtype), ids, dy, rows, 3.0, torch.where(hit.cuda()[:, None], base, 0.0))


@pytest.mark.parametrize("tokens", [40, 3000])
def test_what_padding_tokens_hold_is_not_read(tokens):
    ids = grad_ids(50, tokens, "any", 8)
    dy = torch.randn(tokens, 24, device="cuda")
    want = dfw.embed_grad(ids.cuda(), dy, 50)
    for bad in (float("nan"), float("inf"), torch.finfo(torch.float32).min):
        dy[(ids < 0).cuda()] = bad
        assert torch.equal(dfw.embed_grad(ids.cuda(), dy, 50), want)
    t = int(torch.nonzero(ids >= 0)[3])
    dy[t, 5] = float("nan")  # and a NaN that counts stays in its row and column
    got = dfw.embed_grad(ids.cuda(), dy, 50)
    assert got.isnan().sum() == 1 and got[int(ids[t]), 5].isnan()


def test_calls_that_follow_each_other_without_a_gap():
    """Each call reads what the one before wrote, or overwrites what it reads;
    the launches overlap, the results are those of calls with the GPU idle
    between them."""
    gen = torch.Generator("cuda").manual_seed(9)
    rows, dim, tokens = 3000, 2048, 5000
    emb = (torch.randn(rows, dim, generator=gen, device="cuda") * 0.02).to(torch.bfloat16)
    dl = dfw.encode_device(emb)
    w = dfw.q4_quantise((torch.randn(dim, dim, generator=gen, device="cuda") * 0.02).to(torch.bfloat16))
    ids = ids_for(rows, tokens).cuda()
    few = ids[:16].contiguous()

    def chain(wait):
        table = torch.empty(rows, dim, dtype=torch.bfloat16, device="cuda")
        kept, pause = [], (torch.cuda.synchronize if wait else lambda: None)
        for step in range(6):
            dfw.decode_lanes(dl, out=table.view(-1))
            pause()
            x = dfw.embed_rows(table, ids, scale=0.5 + step)
            pause()
            y = dfw.q4_gemv(w, dfw.embed_rows(table, few), out_dtype=torch.bfloat16)
            pause()
            for _ in range(3):
                y = dfw.q4_gemv(w, y, out_dtype=torch.bfloat16)
                pause()
            dfw.embed_grad(ids, x, rows, out=table)  # overwrites the table that the lookups read
            pause()
            z = dfw.embed_rows(table, few)
            pause()
            dfw.embed_grad(few, y, rows, out=table, accumulate=True)
            pause()
            kept += [x, y, z, table.clone()]
        torch.cuda.synchronize()
        return kept

    want = chain(True)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(chain(False), want))


def test_gradient_is_the_difference_quotient():
    """f(E) = sum of c * lookup(E): linear in E, so (f(E + h e) - f(E)) / h is
    the gradient exactly when all values are whole numbers."""
    rng = np.random.default_rng(6)
    rows, dim, tokens, scale = 11, 24, 60, 2.0
    e = torch.from_numpy(rng.integers(-4, 5, (rows, dim))).float()
    c = torch.from_numpy(rng.integers(-4, 5, (tokens, dim))).float()
    ids = grad_ids(rows, tokens, "any", 7)
    grad = dfw.embed_grad(ids.cuda(), c.cuda(), rows, scale=scale).cpu()

    def f(t):
        return float((dfw.embed_rows(t.to(torch.bfloat16).cuda(), ids.cuda(), scale=scale).cpu().double() * c.double()).sum())

    f0 = f(e)
    for r, d in ((0, 0), (3, 5), (10, 23), (6, 11)):
        t = e.clone()
        t[r, d] += 1.0
        assert f(t) - f0 == float(grad[r, d])


def test_gradient_strides_and_neighbours():
    ids = grad_ids(30, 400, "any")
    wide = torch.randn(400, 90, device="cuda")
    for off in (0, 1, 4, 8):
        for dtype in (torch.float32, torch.bfloat16):
            dy = wide.to(dtype)[:, off: off + 64]
            buf = torch.full((32, 64), 7.0, device="cuda")
            dfw.embed_grad(ids.cuda(), dy, 30, out=buf[1:31])
            assert torch.equal(buf[1:31], dfw.embed_grad(ids.cuda(), dy.contiguous(), 30))
            assert (buf[0] == 7).all() and (buf[31] == 7).all()
    flat = torch.full((30 * 64 + 2,), 7.0, device="cuda", dtype=torch.bfloat16)  # a result that is only 2-byte aligned
    dfw.embed_grad(ids.cuda(), wide[:, :64], 30, out=flat[1:-1].view(30, 64))
    assert torch.equal(flat[1:-1].view(30, 64), dfw.embed_grad(ids.cuda(), wide[:, :64], 30, out_dtype=torch.bfloat16))
    assert flat[0] == 7 and flat[-1] == 7
    with pytest.raises(ValueError):
        dfw.embed_grad(ids.cuda(), torch.ones(1, device="cuda").expand(400, 64), 30)
    with pytest.raises(dfw.DfwError):
        dfw.embed_grad(ids.cuda(), torch.ones(1, 64, device="cuda").expand(400, 64), 30)
    with pytest.raises(dfw.DfwError):
        dfw.embed_grad(ids.cuda(), wide, 30, scratch=torch.empty(0, dtype=torch.uint8, device="cuda"))


def test_two_streams_and_a_graph():
    u = table(500 * 2048)
    dl = coded(u)
    ids = [ids_for(500, t, t).cuda() for t in (3, 900, 4000)]
    dy = [torch.randn(i.numel(), 96, device="cuda") for i in ids]
    run = lambda st=None: [(dfw.embed_lanes(dl, i, 2048, scale=2.0, stream=st), dfw.embed_grad(i, d, 500, stream=st))  # noqa: E731
                           for i, d in zip(ids, dy)]
    want = run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [run(st) for _ in range(4) for st in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for p, q in zip(g, want) for a, b in zip(p, q))
    i, d = ids[1].clone(), dy[1].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a, b = dfw.embed_lanes(dl, i, 2048, scale=2.0), dfw.embed_grad(i, d, 500)
    i.copy_(ids[1].flip(0))
    d.copy_(dy[1].flip(0) * 2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, want[1][0].flip(0))
    check_grad(b, i.cpu(), d, 500, 1.0)


def test_lookup_products_and_a_training_step_together():
    """As a serving loop uses them: token -> coded embedding row -> a 4-bit
    projection and a coded one -> 4-bit logits; then a step on the table: its
    gradient, an update in bf16, coded again, and the new rows read back."""
    rows, dim, wide = 700, 512, 1024
    gen = torch.Generator("cuda").manual_seed(3)
    emb = (torch.randn(rows, dim, generator=gen, device="cuda") * 0.02).to(torch.bfloat16)
    up = (torch.randn(wide, dim, generator=gen, device="cuda") * 0.05).to(torch.bfloat16)
    head = (torch.randn(rows, wide, generator=gen, device="cuda") * 0.05).to(torch.bfloat16)
    scope, up_scope = dfw.encode_device(emb), dfw.encode_device(up)
    q_up, q_head = dfw.q4_quantise(up, group=64, zeros=True), dfw.q4_quantise(head, group=128)
    ids = torch.tensor([5, 699, 5, 0], device="cuda")
    x = dfw.embed_lanes(scope, ids, dim, scale=16.0)
    assert torch.equal(x, (emb[ids].float() * 16).to(torch.bfloat16))
    h = dfw.q4_gemv(q_up, x, out_dtype=torch.bfloat16)
    logits = dfw.q4_gemv(q_head, h)
    wu, wh = dfw.q4_dequantise(q_up).double(), dfw.q4_dequantise(q_head).double()  # each weight off by at most 2^-8 of itself
    xh = x.double()
    hb = xh.abs() @ wu.abs().t()
    assert ((h.double() - xh @ wu.t()).abs() <= 2.0 ** -7 * (hb + h.double().abs())).all()
    hd = h.double()
    assert ((logits.double() - hd @ wh.t()).abs() <= 2.0 ** -7 * (hd.abs() @ wh.abs().t())).all()
    ref = dfw.decode_gemv_lanes(up_scope, [x[1]], [dim])[0]  # the lossless neighbour: within the 4-bit step of each weight
    step = (up.float().view(wide, -1, 64).amax(-1) - up.float().view(wide, -1, 64).amin(-1)) / 15
    slack = (xh[1].abs().view(-1, 64).sum(-1) * step.double()).sum(-1)
    assert ((ref.double() - (xh[1] @ wu.t())).abs() <= slack * 1.05 + 1e-6).all()
    # a step on the table
    dy = torch.randn(4, dim, generator=gen, device="cuda").to(torch.bfloat16)
    grad = dfw.embed_grad(ids, dy, rows, scale=16.0)
    new = (emb.float() - 0.001 * grad).to(torch.bfloat16)
    again = dfw.encode_device(new)
    every = torch.arange(rows, device="cuda", dtype=torch.int32)
    assert torch.equal(dfw.embed_lanes(again, every, dim), new)
    assert torch.equal(new[[1, 2, 3]], emb[[1, 2, 3]]) and not torch.equal(new[5], emb[5])


def test_offsets_past_32_bits():
    """Rows and gradient rows past element 2^32: 2^20 tokens of 4104."""
    rows, dim, tokens = 100, 4104, 1 << 20
    u = table(rows * dim, seed=9)
    ids = torch.randint(0, rows, (tokens,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    w = torch.from_numpy(u.view(np.int16)).view(torch.bfloat16).view(rows, dim).cuda()
    out = torch.empty(tokens, dim, dtype=torch.bfloat16, device="cuda")
    for look in (lambda: dfw.embed_rows(w, ids, out=out), lambda: dfw.embed_lanes(coded(u), ids, dim, out=out)):
        out.fill_(7.0)
        look()
        for at in (slice(0, 1000), slice(tokens // 2 - 500, tokens // 2 + 500), slice(tokens - 1000, tokens)):
            assert torch.equal(out[at], w[ids[at]])
    out[:, 1:-1] = 0.0  # whole numbers in the first and the last column
    out[:, 0] = (torch.arange(tokens, device="cuda") % 5).to(torch.bfloat16)
    out[:, -1] = (torch.arange(tokens, device="cuda") % 3).to(torch.bfloat16)
    grad = dfw.embed_grad(ids, out, rows)
    for col in (0, dim - 1):
        want = torch.zeros(rows, dtype=torch.float64, device="cuda").index_add_(0, ids, out[:, col].double())
        assert torch.equal(grad[:, col].double(), want)
    assert not grad[:, 1:-1].any()


@pytest.mark.parametrize("rows,dim,tokens", [(7, 96, 40), (50, 96, 400000), (11, 5365, 9000), (4, 20000, 700), (30, 2048, 200000)])
@pytest.mark.parametrize("every", [0, 1, 3, 4097])
def test_padding_and_batches_of_many_units(rows, dim, tokens, every):
    """Only every n-th token (or none) has a row; warps take many more units than they look at once."""
    u = table(rows * dim, seed=dim)
    w = torch.from_numpy(u.view(np.int16)).view(torch.bfloat16).view(rows, dim).cuda()
    ids = torch.full((tokens,), -5, dtype=torch.int32, device="cuda")
    if every:
        ids[::every] = (torch.arange(tokens, device="cuda", dtype=torch.int32) * 7 % rows)[::every]
    want = torch.where((ids >= 0)[:, None], w[ids.clamp(min=0).long()], torch.zeros((), dtype=torch.bfloat16, device="cuda"))
    for look in (lambda out: dfw.embed_lanes(coded(u), ids, dim, out=out), lambda out: dfw.embed_rows(w, ids, out=out)):
        assert torch.equal(look(torch.full((tokens, dim), 3.0, dtype=torch.bfloat16, device="cuda")), want)


def once(exact):
    """64-bit values that are exact, rounded to bf16 in one step, ties to even."""
    exact = np.asarray(exact, dtype=np.float64)
    step = np.exp2(np.maximum(np.frexp(exact)[1] - 8, -133).astype(np.float64))  # of a bf16 of this size
    near = np.where(np.isfinite(exact), np.rint(exact / step) * step, exact)
    return torch.from_numpy(np.where(np.abs(near) >= 2.0 ** 128, np.copysign(np.inf, near), near)).float().to(torch.bfloat16)


def scales_that_tie():
    """fp32 scales of which some bf16 weight makes a product that fp32 rounds
    to the middle of two bf16, from where the next rounding goes the wrong way."""
    rng = np.random.default_rng(12)
    m = rng.integers(1 << 23, 1 << 24, 60000)
    low = m[:, None] * np.arange(128, 256)  # 32 bits: of those, fp32 keeps 24 and bf16 8
    drop = np.where(low >> 31, 8, 7)
    up = (low + (1 << (drop - 1)) - 1 + (low >> drop & 1)) >> drop  # rounded to 24 bits, ties to even
    wrong = np.where(up >> 16 & 1, (up << drop) > low, (up << drop) < low)
    hits = m[(((up & 0xFFFF) == 0x8000) & wrong).any(1)]
    assert len(hits) > 40
    return [float(np.float32(v * 2.0 ** -e)) for v, e in zip(hits[:40], [23, 20, 24, 30, 17] * 8)]


def test_a_scaled_row_is_rounded_once():
    """Every bf16 pattern times scales of 24 bits, among them products that
    land next to a tie, below the normal range and past the largest bf16."""
    u = (np.arange(65536, dtype=np.int64) * 40503 % 65536).astype(np.uint16)
    one = table(64 * 1024, "single")
    ids, few = torch.arange(64, device="cuda"), torch.arange(63, -1, -2, device="cuda")
    cases = [(u, dim, coded(u)) for dim in (1024, 1000)] + [(one, dim, coded(one)) for dim in (1024, 999)]
    w = torch.from_numpy(u.view(np.int16)).view(torch.bfloat16)
    assert len(set(w.view(torch.int16).tolist())) == 65536
    for scale in scales_that_tie() + [0.1, -1 / 3, float(np.float32(1e-38) * 3), float(np.float32(2.0 ** 127 * 1.2345678)), 1e-45]:
        for v, dim, dl in cases:
            rows = v.size // dim
            t = torch.from_numpy(v.view(np.int16)).view(torch.bfloat16)[: rows * dim].view(rows, dim)
            want = once(t.double().numpy() * np.float64(np.float32(scale)))
            at = ids[:rows]
            for got, sel in ((dfw.embed_rows(t.cuda(), at, scale=scale), at), (dfw.embed_lanes(dl, at, dim, scale=scale), at),
                             (dfw.embed_lanes(dl, few, dim, scale=scale), few)):
                assert same(got, want[sel.cpu()]), (scale, dim)


def values_that_tie(scale, base):
    """fp32 values v (and bf16 numbers o to add to them, 0 without base) whose
    scale v + o, exact in 64 bits, misses its nearest bf16 by way of fp32."""
    rng = np.random.default_rng(21)
    v = rng.integers(-(1 << 24), 1 << 24, 12_000_000).astype(np.float64)  # scale v: 48 bits
    o = torch.from_numpy(rng.integers(-(1 << 47), 1 << 47, v.size)).double().float().to(torch.bfloat16).double().numpy() if base else 0 * v
    exact = scale * v + o
    hit = once(exact).view(torch.int16) != torch.from_numpy(exact.astype(np.float32)).to(torch.bfloat16).view(torch.int16)
    hit = hit.numpy()
    assert hit.sum() > 40
    return v[hit], o[hit]


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("rows,dim,each", [(60, 40, 1), (2, 33, 40), (2000, 24, 1), (900, 17, 7), (40, 64, 60), (3, 31, 900), (2, 72, 700)])
def test_a_bf16_gradient_is_rounded_once(rows, dim, each, accumulate):
    """Rows of one token that counts, the others' gradients being zero: the
    sum is exact, and scale x sum (+ the old value) is rounded once.  Few
    tokens, rows inside a window, over a few windows and over many."""
    scale = float((1 << 23) + 5_000_001)
    v, o = values_that_tie(scale, accumulate)
    at = np.arange(rows * dim) % v.size
    rng = np.random.default_rng(each)
    ids = rng.permutation(np.repeat(np.arange(rows), each))
    dy = np.zeros((ids.size, dim), dtype=np.float32)
    counts = np.array([rng.choice(np.nonzero(ids == r)[0]) for r in range(rows)])
    dy[counts] = v[at].reshape(rows, dim)
    old = torch.from_numpy(o[at].reshape(rows, dim)).float().to(torch.bfloat16).cuda()
    want = once(scale * v[at] + o[at]).view(rows, dim)
    got = dfw.embed_grad(torch.from_numpy(ids).cuda(), torch.from_numpy(dy).cuda(), rows, scale=scale, out=old, accumulate=accumulate)
    assert torch.equal(got.cpu(), want)


def test_a_bf16_gradient_at_the_ends_of_the_range():
    """Zeros, infinities, NaN, results past the largest bf16 and below the normal range."""
    ids = torch.arange(12, device="cuda", dtype=torch.int32)
    big, tiny = 3.3e38, 2.0 ** -120
    dy = torch.tensor([0.0, 2.0, float("inf"), -float("inf"), float("nan"), big, -big, tiny, -tiny, 1e-45, 1.0, -1.0], device="cuda")
    dy = dy[:, None].expand(12, 8).contiguous()
    for scale in (1.0, 1.1, -3.7, 1e-12, 1e30):
        s = np.float64(np.float32(scale))
        exact = dy.double().cpu().numpy() * s
        assert same(dfw.embed_grad(ids, dy, 12, scale=scale, out_dtype=torch.bfloat16), once(exact))
        for old in (0.0, -2.0 ** -133, 2.0 ** 127, -float("inf")):
            out = torch.full((12, 8), old, dtype=torch.bfloat16, device="cuda")
            with np.errstate(invalid="ignore"):  # infinities of both signs
                want = once(exact + float(out[0, 0]))
            dfw.embed_grad(ids, dy, 12, scale=scale, out=out, accumulate=True)
            assert same(out, want), (scale, old)


@pytest.fixture(scope="module")
def long_groups():
    """A scope of 2.15e6 weights whose rare exponents lie together: two groups
    of codewords of 17 bits among groups of 2, (patterns, first of the rare
    weights, scope)."""
    rng = np.random.default_rng(17)
    rare = rng.permutation(np.repeat(np.arange(200), 21))
    chain = rng.permutation(np.repeat(200 + np.arange(9), 4200 << np.arange(9)))
    at = 1_000_003
    e = np.concatenate([chain[:at], rare, chain[at:]]) + 20
    u = ((rng.integers(0, 2, e.size) << 15) | (e << 7) | rng.integers(0, 128, e.size)).astype(np.uint16)
    return u, at, coded(u)


@pytest.mark.parametrize("dim,first", [(1024, 0), (2048, 2048), (4096, 16), (1000, 8), (6000, 0), (777, 5), (3001, 0)])
@pytest.mark.parametrize("tokens", [1, 9, 2000])
def test_coded_rows_of_long_codewords(long_groups, dim, first, tokens):
    """Slots so long that not even 16 warps of them fit an SM with the table:
    the smallest CTAs, of one warp, looking up the long groups and others."""
    u, at, dl = long_groups
    slot = int(dl.info.max_group_bytes)
    warp = 32 + 2 * (64 + slot) + 2048 + 17 * 136 + 8  # barriers, two slots, raw bytes, exponents (a multiple of 16)
    assert (8 << int(dl.info.fast_bits)) + 16 * warp > 227 * 1024
    rows = (u.size - first) // dim
    mid = (at - first) // dim
    rng = np.random.default_rng(dim)
    ids = np.where(rng.random(tokens) < 0.5, mid + rng.integers(0, 4200 // dim + 2, tokens), rng.integers(0, rows, tokens))
    ids[:4] = (mid, rows - 1, -1, 0)[:tokens]
    ids = torch.from_numpy(ids)
    want = rows_of(u, first, rows, dim, ids, 1.0)
    assert torch.equal(dfw.embed_lanes(dl, ids.cuda(), dim, first=first).cpu().view(torch.int16), want.view(torch.int16))
    for scale in (-45.25, 0.1):
        exact = torch.from_numpy(u.view(np.int16)).view(torch.bfloat16)[first: first + rows * dim].view(rows, dim)[ids.clamp(min=0)].double().numpy()
        exact[(ids < 0).numpy()] = 0.0
        got = dfw.embed_lanes(dl, ids.cuda(), dim, scale=scale, first=first)
        assert torch.equal(got.cpu(), once(exact * np.float64(np.float32(scale))))


def test_rows_of_one_exponent_between_other_calls():
    """Lookups in a scope of one exponent that follow each other and other
    calls without a gap: each reads ids, or writes rows, that the calls around
    it write or read."""
    rows, dim, tokens = 4000, 1024, 6000
    one, u = table(rows * dim, "single", 3), table(rows * dim, seed=4)
    a, b = coded(one), coded(u)
    assert int(a.table.total_bits) == 0
    lists = [ids_for(rows, tokens, 10 + i).cuda() for i in range(3)]
    want = [[rows_of(v, 0, rows, dim, i.cpu(), 2.0).cuda() for i in lists] for v in (one, u)]
    ids, x = torch.empty_like(lists[0]), torch.empty(tokens, dim, dtype=torch.bfloat16, device="cuda")
    for step in range(12):
        kept = []
        for i in lists:
            ids.copy_(i)
            for dl in (a, a, b, a):
                dfw.embed_lanes(dl, ids, dim, scale=2.0, out=x)
                kept.append(dfw.embed_rows(x, torch.arange(0, tokens, 50, device="cuda")))
        for n, got in enumerate(kept):
            assert torch.equal(got, want[1 if n % 4 == 2 else 0][n // 4][::50]), (step, n)


def test_ids_and_tables_that_the_call_before_writes():
    """Each call's ids, and some calls' table and gradient rows, come from the
    launch right before it, which writes over what earlier calls read there."""
    gen = torch.Generator("cuda").manual_seed(12)
    rows, dim = 3000, 96
    u = table(rows * dim, seed=8)
    coded_table, one = coded(u), coded(table(rows * dim, "single", 9))
    w = torch.from_numpy(u.view(np.int16)).view(torch.bfloat16).view(rows, dim).cuda()
    for tokens in (100, 6000):
        # ids as the bits of bf16 rows: a lookup writes them
        pools = torch.randint(0, rows, (8 * tokens,), generator=gen, device="cuda").view(torch.bfloat16).view(-1, 4)
        picks = [torch.randperm(8 * tokens, generator=gen, device="cuda")[:tokens] for _ in range(6)]
        bits = torch.empty(tokens, 4, dtype=torch.bfloat16, device="cuda")
        ids = bits.view(torch.int64).view(-1)

        def chain(wait):
            pause = torch.cuda.synchronize if wait else lambda: None
            kept = []

            def pick(i):
                pause()
                dfw.embed_rows(pools, picks[i], out=bits)
                pause()

            tab, kept = w.clone(), []
            for i in range(6):
                pick(i)
                kept.append(dfw.embed_lanes(coded_table, ids, dim, scale=2.0))
                pick((i + 1) % 6)
                kept.append(dfw.embed_lanes(one, ids, dim))
                pick((i + 2) % 6)
                x = dfw.embed_rows(tab, ids, scale=0.5)
                pause()
                kept.append(dfw.embed_rows(x, ids.clamp(max=tokens - 1)))
                pick((i + 3) % 6)
                kept.append(dfw.embed_grad(ids, x, rows))
                pick((i + 4) % 6)
                dfw.embed_grad(ids, x, rows, out=tab, accumulate=True)
                pause()
                kept.append(dfw.embed_rows(tab, picks[0][:200].clamp(max=rows - 1)))
            torch.cuda.synchronize()
            return kept

        want = chain(True)
        for _ in range(4):
            assert all(torch.equal(a, b) for a, b in zip(chain(False), want))

"""Numerics of the training-step operators (libtide_step.so) on the GPU, against their definitions in
64 bits on the same inputs.

Tolerances are error bounds of the formulas, not measured: `u` is the unit roundoff of fp32 (2^-24),
`uo(dtype)` that of the output's type, and a sum of n terms in any order is off by at most
(n - 1) u times the sum of their magnitudes.  Where sums are of whole numbers they are exact in fp32
and results have to be equal.
"""
import math

import pytest
import torch

from all_gather_placement_amd import (clip_grad_norm, embedding, embedding_bwd, grad_clip, grad_norm, layer_norm,
                                      layer_norm_bwd)

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, FP32 = torch.bfloat16, torch.float32
DTYPES = [BF16, FP32]


def uo(dtype):
    return torch.finfo(dtype).eps / 2


def say(*a):
    print(*a, flush=True)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(shape, dtype, seed, scale=1.0, shift=0.0):
    x = torch.empty(shape, device="cuda", dtype=FP32).normal_(shift, scale, generator=gen(seed))
    return x.to(dtype)


def whole(shape, dtype, seed, lo=-4, hi=5):
    return torch.randint(lo, hi, shape, device="cuda", generator=gen(seed)).to(dtype)


def off_by_one(t):
    """The same values, starting one element past an allocation's start."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    v = buf[1:].view(t.shape)
    v.copy_(t)
    return v


def within(got, want, tol, what):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), float((err - tol)[bad].max()))


# ------------------------------------------------------------------------------------------------
# Gradient norm and clipping
# ------------------------------------------------------------------------------------------------

def exact_sumsq(grads):
    return math.fsum(float(g.double().square().sum()) for g in grads)


# tensors of one chunk of 16 KiB, of several, of none; more tensors than one launch names (250, 160)
SIZES = [
    [1], [7, 0, 5], [31] * 4, [4095, 4096, 4097, 8191, 8192, 8193], [0], [0, 0],
    [3 * 8192 + 5, 2, 70001], [64 + 3 * i for i in range(520)], [9000] * 251, [1 << 22, 12345],
]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
def test_norm_and_clip(gpu_available, sizes, dtype):
    say("norm and clip", len(sizes), max(sizes), dtype)
    grads = [normal((n,), dtype, 10 + i, 1e-3 * (1 + i % 5)) for i, n in enumerate(sizes)]
    grads = [off_by_one(g) if i % 3 == 1 else g for i, g in enumerate(grads)]
    total = exact_sumsq(grads)
    want = math.sqrt(total)
    sumsq = torch.full((), float("nan"), dtype=torch.float64, device="cuda")
    norm = grad_norm(grads, sumsq=sumsq)
    # eight squares and their sum in fp32: 8 u on the sum of squares, half of it on the norm, and its rounding
    assert abs(float(sumsq) - total) <= 8 * U * total
    assert abs(float(norm) - want) <= 5 * U * want
    for max_norm in (want / 3, want * 2 + 1):
        coef = min(1.0, max_norm / (want + 1e-6))
        outs = [torch.full_like(g, float("nan")) for g in grads]
        got = clip_grad_norm(grads, max_norm, outs=outs)
        given = [torch.full_like(g, float("nan")) for g in grads]
        again = grad_clip(grads, sumsq, max_norm, outs=given)
        assert torch.equal(got, norm) and torch.equal(again, norm)
        for g, o, p in zip(grads, outs, given):
            # the norm's error and three roundings of fp32, then the output's
            within(o, g.double() * coef, (uo(dtype) + 8 * U) * (g.double() * coef).abs() + 1e-40, max_norm)
            assert torch.equal(o, p)
            if coef == 1.0:
                assert torch.equal(o, g)
    inplace = [g.clone() for g in grads]
    clip_grad_norm(inplace, want / 3)
    outs = [torch.empty_like(g) for g in grads]
    clip_grad_norm(grads, want / 3, outs=outs)
    assert all(torch.equal(a, b) for a, b in zip(inplace, outs))


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_norm_over_the_whole_range(gpu_available, dtype):
    """Squares that leave the range of fp32 at either end still count."""
    for scale in (1e30, 1e-30, 1e-38):
        g = whole((5000,), FP32, 3).mul_(scale).to(dtype)
        want = math.sqrt(exact_sumsq([g]))
        assert abs(float(grad_norm([g])) - want) <= 5 * U * want + 1e-45, scale
    # one large value among tiny ones, and denormal values
    g = torch.full((20000,), 1e-25, dtype=dtype, device="cuda")
    g[777] = 2.0 ** 90
    assert float(grad_norm([g])) == 2.0 ** 90
    tiny = torch.full((4096,), 2.0 ** -130, dtype=dtype, device="cuda")
    assert float(grad_norm([tiny])) == 2.0 ** -124


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("n", [5, 9000, 300001])
def test_norm_of_nan_and_infinity(gpu_available, n, dtype):
    for bad, at in ((float("nan"), n - 1), (float("inf"), 0), (float("-inf"), n // 2)):
        g = normal((n,), dtype, 4)
        g[at] = bad
        norm = float(grad_norm([g, normal((17,), dtype, 5)]))
        assert math.isnan(norm) if math.isnan(bad) else norm == math.inf
        out = torch.zeros_like(g)
        clip_grad_norm([g], 1.0, outs=[out])
        if math.isnan(bad):
            assert bool(out.isnan().all())
        else:  # finite values times 0; infinity times 0 is NaN
            assert bool(out[at].isnan()) and int(out.isnan().sum()) == 1 and float(out.nan_to_num().abs().max()) == 0
    g = normal((n,), dtype, 6)
    out = torch.empty_like(g)
    clip_grad_norm([g], math.inf, outs=[out])
    assert torch.equal(out, g)
    clip_grad_norm([g], 0.0, outs=[out])
    assert float(out.abs().max()) == 0.0


def test_norm_of_nothing(gpu_available):
    sumsq = torch.full((), float("nan"), dtype=torch.float64, device="cuda")
    assert float(grad_norm([], sumsq=sumsq)) == 0.0 and float(sumsq) == 0.0
    assert float(clip_grad_norm([], 1.0)) == 0.0
    sumsq.fill_(9.0)
    assert float(grad_clip([], sumsq, 1.0)) == 3.0


def test_norm_does_not_depend_on_the_run(gpu_available):
    grads = [normal((100_003 + 7 * i,), FP32, i) for i in range(20)]
    first = grad_norm(grads)
    assert all(torch.equal(grad_norm(grads), first) for _ in range(5))


# ------------------------------------------------------------------------------------------------
# Layer norm
# ------------------------------------------------------------------------------------------------

def adds(cols):
    """Additions that a term of a row's sum goes through, at most: a lane's elements (eight for each of
    up to four vectors, more only where a row is streamed), six within the wave, one for each wave."""
    return cols / 1024 + 64


def ln_reference(x, w, b, eps):
    x = x.double()
    mean = x.mean(-1, keepdim=True)
    d = x - mean
    var = d.square().mean(-1, keepdim=True)
    rstd = (var + eps).rsqrt()
    w = torch.ones(x.shape[-1], device=x.device, dtype=torch.float64) if w is None else w.double()
    b = torch.zeros(x.shape[-1], device=x.device, dtype=torch.float64) if b is None else b.double()
    xhat = d * rstd
    y = xhat * w + b
    # the mean is off by adds * u of the row's magnitude, each difference by that and its rounding
    dd = (adds(x.shape[-1]) + 2) * U * x.abs().amax(-1, keepdim=True)
    # relative error of rstd: half of the variance's, from the differences and from their sum
    dr = dd * var.sqrt() / (var + eps) + dd.square() / (var + eps) + (adds(x.shape[-1]) + 6) * U
    tol = w.abs() * (rstd * dd * (1 + dr) + xhat.abs() * (dr + 4 * U)) + 2 * U * (y.abs() + b.abs())
    return y, mean[..., 0], rstd[..., 0], tol, dd[..., 0], dr[..., 0] * rstd[..., 0]


def check_ln(x, w, b, eps=1e-5, **kw):
    y, mean, rstd = layer_norm(x, w, b, eps, **kw)
    assert y.dtype == x.dtype and y.shape == x.shape and mean.dtype == rstd.dtype == FP32
    ry, rmean, rrstd, tol, tmean, trstd = ln_reference(x, w, b, eps)
    within(mean, rmean, tmean + U * rmean.abs(), "mean")
    within(rstd, rrstd, trstd + 2 * U * rrstd, "rstd")
    within(y, ry, tol + uo(x.dtype) * (ry.abs() + tol), "y")
    return y, mean, rstd


# every row shape of the kernels: within a wave (up to 1024), a workgroup, streamed beyond 32768
COLS = [1, 2, 7, 8, 63, 64, 65, 255, 257, 512, 513, 1000, 1024, 1025, 2049, 4096, 5120, 6145, 8192, 8193, 16384, 16389,
        32768, 40001]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("cols", COLS)
def test_layer_norm(gpu_available, cols, dtype):
    say("layer norm", cols, dtype)
    for rows, pdtype in ((1, dtype), (3, FP32), (67, BF16)):
        x = normal((rows, cols), dtype, cols + rows) * 2 + normal((rows, 1), dtype, 5)
        w, b = normal((cols,), pdtype, 1, 0.2, 1.0), normal((cols,), pdtype, 2)
        check_ln(x, w, b)
    x = normal((5, cols), dtype, cols)
    check_ln(x, None, None)
    check_ln(x, w, None)
    check_ln(x, None, b)
    check_ln(off_by_one(x), off_by_one(w), off_by_one(b), out=off_by_one(torch.zeros_like(x)))


def test_layer_norm_many_rows(gpu_available):
    for rows, cols in ((70001, 8), (3001, 64), (5000, 256), (2500, 1024), (1500, 2048)):
        say("layer norm rows", rows, cols)
        check_ln(normal((rows, cols), BF16, rows, 3.0, 1.0), normal((cols,), BF16, 1), normal((cols,), BF16, 2))


def test_layer_norm_shapes_and_strides(gpu_available):
    x = normal((2, 3, 5, 40), FP32, 1)
    y, mean, _ = check_ln(x, normal((40,), FP32, 2), None)
    assert mean.shape == (2, 3, 5)
    check_ln(normal((33,), BF16, 3), None, None)
    wide = normal((50, 301), BF16, 4)
    out = torch.full((50, 333), float("nan"), dtype=BF16, device="cuda")
    check_ln(wide[:, 5:282], None, None, out=out[:, 11:288])
    assert bool(out[:, :11].isnan().all()) and bool(out[:, 288:].isnan().all())
    y, mean, rstd = layer_norm(torch.empty((0, 16), device="cuda"))
    assert y.shape == (0, 16) and mean.shape == (0,)


def test_layer_norm_hard_values(gpu_available):
    # a mean a thousand times the deviation: the centred squares keep it exact
    check_ln(normal((9, 4096), FP32, 1, 1.0, 1000.0), None, None)
    # rows of one value have no deviation: y is the bias, up to the mean's own error
    x = torch.full((4, 1000), 3.0, device="cuda")
    y, mean, rstd = check_ln(x, normal((1000,), FP32, 2), normal((1000,), FP32, 3))
    # a row with a NaN or an infinity is NaN, its neighbours are not touched
    x = normal((6, 777), BF16, 4)
    x[1, 776], x[4, 0] = float("nan"), float("inf")
    y, mean, rstd = layer_norm(x)
    assert bool(y[[1, 4]].isnan().all()) and not bool(y[[0, 2, 3, 5]].isnan().any())


def ln_bwd_reference(dy, x, w, mean, rstd):
    x, dy = x.double(), dy.double()
    cols = x.shape[-1]
    wd = torch.ones(cols, device=x.device, dtype=torch.float64) if w is None else w.double()
    r = rstd.double()[:, None]
    xhat = (x - mean.double()[:, None]) * r
    g = dy * wd
    m1, m2 = g.mean(1, keepdim=True), (g * xhat).mean(1, keepdim=True)
    dx = r * (g - m1 - xhat * m2)
    a1, a2, n = g.abs().mean(1, keepdim=True), (g * xhat).abs().mean(1, keepdim=True), adds(cols)
    # xhat carries 2 u, g 1 u, the means their sums', and three operations follow
    tol = r * (5 * U * (g.abs() + m1.abs() + (xhat * m2).abs()) + (n + 2) * U * a1 + xhat.abs() * (n + 6) * U * a2)
    rows = x.shape[0]
    dw, db = (dy * xhat).sum(0), dy.sum(0)
    tw, tb = (rows + 3) * U * (dy * xhat).abs().sum(0), rows * U * dy.abs().sum(0)
    return dx, dw, db, tol, tw, tb


def check_ln_bwd(dy, x, w, **kw):
    _, mean, rstd = layer_norm(x.contiguous(), w)
    want_dtype = x.dtype if w is None else w.dtype
    rdx, rdw, rdb, tol, tw, tb = ln_bwd_reference(dy, x, w, mean, rstd)
    dx, dw, db = layer_norm_bwd(dy, x, w, mean, rstd, **kw)
    assert dx.dtype == x.dtype and dw.dtype == db.dtype == want_dtype
    within(dx, rdx, tol + uo(x.dtype) * (rdx.abs() + tol), "dx")
    within(dw, rdw, tw + uo(want_dtype) * (rdw.abs() + tw), "dweight")
    within(db, rdb, tb + uo(want_dtype) * (rdb.abs() + tb), "dbias")
    return dx, dw, db


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("cols", COLS)
def test_layer_norm_bwd(gpu_available, cols, dtype):
    say("layer norm gradient", cols, dtype)
    for rows, pdtype in ((1, dtype), (5, FP32), (131, BF16)):
        x = normal((rows, cols), dtype, cols + rows) * 2 + normal((rows, 1), dtype, 5)
        check_ln_bwd(normal((rows, cols), dtype, 7), x, normal((cols,), pdtype, 1, 0.2, 1.0))
    x, dy = normal((6, cols), dtype, cols), normal((6, cols), dtype, 8)
    dx, dw, db = check_ln_bwd(dy, x, None)
    w = normal((cols,), FP32, 3)
    _, mean, rstd = layer_norm(x, w)
    want = layer_norm_bwd(dy, x, w, mean, rstd)
    inplace = off_by_one(dy)
    got = layer_norm_bwd(inplace, off_by_one(x), off_by_one(w), mean, rstd, dx=inplace)
    assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("rows,cols", [(70001, 8), (9001, 50), (5003, 256), (3001, 513), (4100, 1000), (2049, 2048),
                                       (1300, 8192), (600, 9000), (300, 33000)])
def test_layer_norm_bwd_sums_are_of_every_row(gpu_available, rows, cols):
    """Whole numbers: the bias's gradient is exact, so no row is missed or counted twice."""
    say("layer norm gradient sums", rows, cols)
    x, dy = normal((rows, cols), BF16, 1), whole((rows, cols), BF16, 2)
    _, mean, rstd = layer_norm(x)
    dx, dw, db = layer_norm_bwd(dy, x, None, mean, rstd, dweight=torch.empty(cols, device="cuda"),
                                dbias=torch.empty(cols, device="cuda"))
    assert torch.equal(db, dy.float().sum(0))
    # xhat of whole numbers: mean 0 and rstd 1 given
    xw = whole((rows, cols), BF16, 3)
    _, dw, db = layer_norm_bwd(dy, xw, None, torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda"),
                               dweight=dw, dbias=db)
    assert torch.equal(dw, (dy.double() * xw.double()).sum(0).float())


def test_layer_norm_bwd_shapes(gpu_available):
    x, dy = normal((50, 301), FP32, 1), normal((50, 310), FP32, 2)
    out = torch.full((50, 333), float("nan"), device="cuda")
    check_ln_bwd(dy[:, 3:280], x[:, 5:282], normal((277,), BF16, 3), dx=out[:, 9:286])
    assert bool(out[:, :9].isnan().all()) and bool(out[:, 286:].isnan().all())
    none = torch.empty((0, 24), device="cuda")
    stats = torch.empty((0,), device="cuda")
    dx, dw, db = layer_norm_bwd(none, none, torch.ones(24, device="cuda"), stats, stats)
    assert dx.shape == (0, 24) and not bool(dw.any()) and not bool(db.any())


@pytest.mark.parametrize("cols", [3, 40, 700, 2100])
def test_layer_norm_bwd_against_differences(gpu_available, cols):
    """Central differences, in 64 bits, of the forward definition."""
    rows, eps, h = 4, 1e-3, 1e-5
    x, dy, w = normal((rows, cols), FP32, 1), normal((rows, cols), FP32, 2), normal((cols,), FP32, 3, 0.3, 1.0)
    _, mean, rstd = layer_norm(x, w, eps=eps)
    dx, dw, db = layer_norm_bwd(dy, x, w, mean, rstd)

    def loss(xx, ww, bb):
        xx = xx.double()
        d = xx - xx.mean(1, keepdim=True)
        y = d * (d.square().mean(1, keepdim=True) + eps).rsqrt() * ww + bb
        return float((y * dy.double()).sum())

    b = torch.zeros(cols, dtype=torch.float64, device="cuda")
    for k in {0, 1, cols // 2, cols - 1}:
        for r in range(rows):
            e = torch.zeros((rows, cols), dtype=torch.float64, device="cuda")
            e[r, k] = h
            diff = (loss(x.double() + e, w.double(), b) - loss(x.double() - e, w.double(), b)) / (2 * h)
            # the difference's own error: h^2 of the third derivative, 2^-53 of the loss over h
            assert abs(float(dx[r, k]) - diff) <= 1e-4 * (1 + abs(diff)) * float(rstd[r]) ** 1
        e = torch.zeros(cols, dtype=torch.float64, device="cuda")
        e[k] = h
        diff = (loss(x, w.double() + e, b) - loss(x, w.double() - e, b)) / (2 * h)
        assert abs(float(dw[k]) - diff) <= 1e-4 * (1 + abs(diff))
        diff = (loss(x, w.double(), b + e) - loss(x, w.double(), b - e)) / (2 * h)
        assert abs(float(db[k]) - diff) <= 1e-4 * (1 + abs(diff))


# ------------------------------------------------------------------------------------------------
# Embedding
# ------------------------------------------------------------------------------------------------

def emb_reference(ids, table, scale):
    ids = ids.long().reshape(-1)
    inside = (ids >= 0) & (ids < table.shape[0])
    out = torch.zeros((ids.numel(), table.shape[1]), dtype=torch.float64, device="cuda")
    out[inside] = table[ids[inside]].double() * scale
    return out


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("dim", [1, 5, 8, 9, 64, 100, 512, 513, 1000, 4096, 5125])
def test_embedding(gpu_available, dim, dtype):
    say("embedding", dim, dtype)
    for tokens, vocab, idt in ((1, 1, torch.int64), (17, 300, torch.int32), (1025, 77, torch.int64)):
        table = normal((vocab, dim), dtype, dim)
        ids = torch.randint(-2, vocab + 2, (tokens,), device="cuda", generator=gen(tokens)).to(idt)
        for scale in (1.0, math.sqrt(dim)):
            want = emb_reference(ids, table, torch.tensor(scale, dtype=FP32).double().item())
            got = embedding(ids, table, scale)
            # one product in fp32, one rounding
            within(got, want, (U + uo(dtype)) * (1 + U) * want.abs(), (tokens, vocab, scale))
            assert torch.equal(embedding(off_by_one(ids), off_by_one(table), scale,
                                         out=off_by_one(torch.zeros_like(got))), got)
        if tokens > 1:
            assert torch.equal(embedding(ids, table), emb_reference(ids, table, 1.0).to(dtype))


def test_embedding_outside_ids_and_shapes(gpu_available):
    table = normal((10, 24), BF16, 1)
    ids = torch.tensor([[-1, 10, 9], [2 ** 62, -2 ** 62, 0]], device="cuda")
    out = embedding(ids, table, 2.0)
    assert out.shape == (2, 3, 24)
    assert torch.equal(out[0, 2], table[9] * 2) and torch.equal(out[1, 2], table[0] * 2)
    assert not bool(out[0, :2].any()) and not bool(out[1, :2].any())
    assert not bool(torch.signbit(out[0, :2]).any())
    assert embedding(torch.empty((0, 4), dtype=torch.int32, device="cuda"), table).shape == (0, 4, 24)
    none = torch.empty((0, 24), dtype=BF16, device="cuda")
    assert not bool(embedding(ids, none).any())
    # values outside the table's rows in use do not leak through a zero scale or a padded id
    table[3] = float("nan")
    assert not bool(embedding(ids, table).isnan().any())


def emb_bwd_reference(ids, dy, vocab, scale, old=None):
    ids = ids.long().reshape(-1)
    dy = dy.reshape(ids.numel(), -1).double()
    inside = (ids >= 0) & (ids < vocab)
    s = torch.zeros((vocab, dy.shape[1]), dtype=torch.float64, device="cuda").index_add_(0, ids[inside], dy[inside])
    m = torch.zeros_like(s).index_add_(0, ids[inside], dy[inside].abs())
    count = torch.bincount(ids[inside], minlength=vocab)[:, None].double()
    want = s * scale
    tol = (count + 1) * U * abs(scale) * m
    if old is not None:
        want = want + old.double()
        tol = tol + U * (want.abs() + tol)
    return want, tol


EMB_BWD = [  # tokens, vocab, dim
    (1, 1, 1), (1, 5, 9), (31, 7, 8), (32, 3, 40), (33, 2, 17), (64, 1, 100), (65, 1, 513), (1000, 1, 64),
    (1000, 255, 257), (1025, 256, 1000), (4096, 257, 64), (3000, 4000, 1001), (2049, 70000, 24), (777, 140001, 40),
    (5000, 300000, 8), (20000, 600, 2056), (100, 50, 5125), (65536, 33, 16),
]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("tokens,vocab,dim", EMB_BWD)
def test_embedding_bwd(gpu_available, tokens, vocab, dim, dtype):
    say("embedding gradient", tokens, vocab, dim, dtype)
    ids = torch.randint(-1, vocab + 1, (tokens,), device="cuda", generator=gen(tokens + vocab))
    ids = torch.where(torch.rand(tokens, device="cuda", generator=gen(1)) < 0.3, vocab // 2, ids)  # a frequent one
    dy = normal((tokens, dim), dtype, 2)
    scale = 1.5
    want, tol = emb_bwd_reference(ids, dy, vocab, scale)
    out = torch.full((vocab, dim), float("nan"), dtype=dtype, device="cuda")
    got = embedding_bwd(ids, dy, vocab, scale, out=out)
    within(got, want, tol + uo(dtype) * (want.abs() + tol), "gradient")
    assert torch.equal(embedding_bwd(ids.to(torch.int32), off_by_one(dy), vocab, scale), got)
    old = normal((vocab, dim), dtype, 3)
    want, tol = emb_bwd_reference(ids, dy, vocab, scale, old)
    got = embedding_bwd(ids, dy, vocab, scale, out=old.clone(), accumulate=True)
    within(got, want, tol + uo(dtype) * (want.abs() + tol), "accumulated")
    absent = torch.ones(vocab, dtype=torch.bool, device="cuda")
    absent[ids[(ids >= 0) & (ids < vocab)]] = False
    assert torch.equal(got[absent], old[absent])


@pytest.mark.parametrize("tokens,vocab,dim", [(50021, 1, 24), (50021, 513, 40), (12345, 100003, 8), (70000, 3, 9)])
def test_embedding_bwd_sums_are_of_every_token(gpu_available, tokens, vocab, dim):
    """Whole numbers: fp32 sums are exact, whatever their order."""
    say("embedding gradient sums", tokens, vocab, dim)
    ids = (torch.rand(tokens, device="cuda", generator=gen(1)).square() * vocab).long().clamp_(max=vocab - 1)
    dy = whole((tokens, dim), FP32, 2)
    want = torch.zeros((vocab, dim), dtype=torch.float64, device="cuda").index_add_(0, ids, dy.double())
    assert torch.equal(embedding_bwd(ids, dy, vocab).double(), want)


def test_embedding_bwd_order(gpu_available):
    """The sum of a row goes by ascending token within a piece: the same bits for any run, and for tokens
    of other rows in between."""
    dy = normal((40, 16), FP32, 1)
    ids = torch.zeros(40, dtype=torch.int64, device="cuda")
    first = embedding_bwd(ids, dy, 3)
    assert all(torch.equal(embedding_bwd(ids, dy, 3), first) for _ in range(4))
    mixed = torch.full((80,), 2, dtype=torch.int64, device="cuda")
    mixed[::2] = 0
    both = torch.zeros((80, 16), device="cuda")
    both[::2] = dy
    assert torch.equal(embedding_bwd(mixed, both, 3)[0], first[0])


def test_embedding_bwd_edges(gpu_available):
    none = torch.empty((0,), dtype=torch.int64, device="cuda")
    out = torch.full((5, 3), float("nan"), device="cuda")
    assert not bool(embedding_bwd(none, torch.empty((0, 3), device="cuda"), 5, out=out).any())
    kept = torch.ones((5, 3), device="cuda")
    embedding_bwd(none, torch.empty((0, 3), device="cuda"), 5, out=kept, accumulate=True)
    assert bool((kept == 1).all())
    ids = torch.tensor([-1, 5, -2 ** 40, 2 ** 40], device="cuda")
    bad = torch.full((4, 3), float("nan"), device="cuda")
    assert not bool(embedding_bwd(ids, bad, 5).any())  # nothing inside the table: NaN gradients do not reach it
    assert embedding_bwd(ids, bad, 0).shape == (0, 3)
    grad = embedding_bwd(torch.tensor([[0, 1], [1, 1]], device="cuda"), torch.ones((2, 2, 4), device="cuda"), 3)
    assert grad[:, 0].tolist() == [1, 3, 0]


# ------------------------------------------------------------------------------------------------
# Far offsets, streams, graphs
# ------------------------------------------------------------------------------------------------

def test_offsets_beyond_32_bits(gpu_available):
    """Tables and matrices of more than 2^31 elements (and 2^32 bytes)."""
    dim, vocab = 8192, 270_000  # 2.2e9 elements
    table = torch.empty((vocab, dim), dtype=BF16, device="cuda")
    ids = torch.tensor([0, vocab - 1, 262_200, 5], device="cuda")
    table[ids] = normal((4, dim), BF16, 1)
    assert torch.equal(embedding(ids, table), table[ids])
    dy = normal((4, dim), BF16, 2)
    table.fill_(1.0)
    grad = embedding_bwd(ids, dy, vocab, out=table)
    assert torch.equal(grad[ids], dy)
    assert int(torch.count_nonzero(grad[262_300:262_400])) == 0 and int(torch.count_nonzero(grad[-100:-1])) == 0
    # rows further than 2^31 elements apart, in the same memory
    stride = (1 << 30) + 8
    x = table.view(-1).as_strided((3, 1000), (stride, 1))
    values = normal((3, 1000), BF16, 3)
    x.copy_(values)
    y, mean, rstd = layer_norm(x)
    assert torch.equal(y, layer_norm(values)[0])
    dx, _, _ = layer_norm_bwd(values, x, None, mean, rstd, dx=x.new_empty((3, 1000)))
    assert torch.equal(dx, layer_norm_bwd(values, values, None, mean, rstd)[0])
    table.zero_()
    table[-1, -1] = 3.0
    table[0, 0] = 4.0
    assert float(grad_norm([table.view(-1)])) == 5.0


def _step(t):
    """Every operator once, on buffers of `t`."""
    embedding(t["ids"], t["table"], 2.0, out=t["h"], stream=t["stream"])
    layer_norm(t["h"], t["w"], t["b"], out=t["y"], mean=t["mean"], rstd=t["rstd"], stream=t["stream"])
    layer_norm_bwd(t["y"], t["h"], t["w"], t["mean"], t["rstd"], dx=t["dx"], dweight=t["dw"], dbias=t["db"],
                   workspace=t["ws"], stream=t["stream"])
    embedding_bwd(t["ids"], t["dx"], t["table"].shape[0], 2.0, out=t["dtable"], workspace=t["ws"], stream=t["stream"])
    clip_grad_norm([t["dtable"], t["dw"], t["db"]], 0.5, norm=t["norm"], workspace=t["ws"], stream=t["stream"])
    return [t[k].clone() for k in ("y", "dtable", "dw", "db", "norm")]


def _buffers(stream=None):
    tokens, vocab, dim = 300, 500, 264
    t = dict(ids=torch.randint(0, vocab, (tokens,), device="cuda", generator=gen(1)), table=normal((vocab, dim), BF16, 2),
             w=normal((dim,), BF16, 3, 0.2, 1.0), b=normal((dim,), BF16, 4), stream=stream)
    for k in ("h", "y", "dx"):
        t[k] = torch.empty((tokens, dim), dtype=BF16, device="cuda")
    t.update(mean=torch.empty(tokens, device="cuda"), rstd=torch.empty(tokens, device="cuda"),
             dtable=torch.empty((vocab, dim), dtype=BF16, device="cuda"), dw=torch.empty_like(t["w"]),
             db=torch.empty_like(t["b"]), norm=torch.empty((), device="cuda"),
             ws=torch.empty(8 << 20, dtype=torch.uint8, device="cuda"))
    return t


def test_on_another_stream(gpu_available):
    t = _buffers()
    want = _step(t)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        u = _buffers(stream)
        for k in ("y", "dtable", "dw", "db", "norm"):
            u[k].zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            got = _step(u)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # outputs and workspaces that the binding allocates, on a stream that is not the current one
    y, mean, rstd = layer_norm(t["h"], t["w"], t["b"], stream=side)
    dx, dw, db = layer_norm_bwd(y, t["h"], t["w"], mean, rstd, stream=side)
    grad = embedding_bwd(t["ids"], dx, t["table"].shape[0], 2.0, stream=side)
    norm = grad_norm([grad, dw, db], stream=side)
    side.synchronize()
    assert torch.equal(y, want[0])
    assert abs(float(norm) - float(want[4])) <= 4 * U * float(want[4])


def test_in_a_graph(gpu_available):
    """Captured once, replayed on new contents, with eager work of the same kind between replays."""
    t = _buffers()
    _step(t)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _step(t)
    eager = _buffers()
    for k in range(4):
        t["table"].copy_(normal(tuple(t["table"].shape), BF16, 20 + k))
        t["ids"].copy_(torch.randint(-1, 501, (300,), device="cuda", generator=gen(30 + k)))
        eager["table"].copy_(t["table"])
        eager["ids"].copy_(t["ids"])
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        want = _step(eager)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), k

"""The training-step operators where their kernels change form: many rows, tensors beyond the last-level
cache, rows that end inside a vector, lists around one workgroup, runs of equal ids around a wave's and
a workgroup's task; the binding's refusals; and the example that runs them with the collectives.

Tolerances are error bounds of the formulas (see test_gpu_step.py, whose references are used here)."""
import importlib.util
import math
import os

import pytest
import torch

import all_gather_placement_amd as tide
from all_gather_placement_amd import (TideError, clip_grad_norm, embedding, embedding_bwd, grad_clip, grad_norm,
                                      layer_norm, layer_norm_bwd)
from test_gpu_step import (BF16, FP32, U, check_ln, check_ln_bwd, emb_bwd_reference, gen, ln_bwd_reference,
                           ln_reference, normal, say, uo, whole, within)

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# ------------------------------------------------------------------------------------------------
# Layer norm
# ------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, FP32], ids=str)
@pytest.mark.parametrize("rows,cols", [(2048, 1026), (2049, 2050), (2500, 1400), (2047, 3000), (2300, 5120),
                                       (2111, 8200), (2050, 12289), (2049, 25000)])
def test_layer_norm_of_many_rows(gpu_available, rows, cols, dtype):
    say("layer norm of many rows", rows, cols, dtype)
    x = normal((rows, cols), dtype, cols, 2.0) + normal((rows, 1), dtype, 5)
    w, b = normal((cols,), BF16, 1, 0.2, 1.0), normal((cols,), BF16, 2)
    check_ln(x, w, b)
    check_ln_bwd(normal((rows, cols), dtype, 7), x, w.to(dtype))


@pytest.mark.parametrize("rows,cols,dtype", [(30001, 5119, BF16), (30000, 5120, BF16), (1_200_003, 63, FP32),
                                             (90_007, 1024, BF16), (15_000, 8192, BF16), (9_001, 8193, FP32)])
def test_layer_norm_beyond_the_cache(gpu_available, rows, cols, dtype):
    """More bytes than the last-level cache holds; references in parts, for their size."""
    say("layer norm beyond the cache", rows, cols, dtype)
    x = normal((rows, cols), dtype, 1, 2.0, 0.5)
    w, b = normal((cols,), dtype, 2, 0.2, 1.0), normal((cols,), dtype, 3)
    dy = normal((rows, cols), dtype, 4)
    y, mean, rstd = layer_norm(x, w, b)
    dx, dw, db = layer_norm_bwd(dy, x, w, mean, rstd)
    sums = [torch.zeros(cols, dtype=torch.float64, device="cuda") for _ in range(4)]
    part = max(1, 20_000_000 // cols)
    for r in range(0, rows, part):
        s = slice(r, min(r + part, rows))
        ry, rmean, rrstd, tol, tmean, trstd = ln_reference(x[s], w, b, 1e-5)
        within(mean[s], rmean, tmean + U * rmean.abs(), "mean")
        within(rstd[s], rrstd, trstd + 2 * U * rrstd, "rstd")
        within(y[s], ry, tol + uo(dtype) * (ry.abs() + tol), "y")
        rdx, rdw, rdb, tol, _, _ = ln_bwd_reference(dy[s], x[s], w, mean[s], rstd[s])
        within(dx[s], rdx, tol + uo(dtype) * (rdx.abs() + tol), "dx")
        xhat = (x[s].double() - mean[s].double()[:, None]) * rstd[s].double()[:, None]
        for t, v in zip(sums, (rdw, rdb, (dy[s].double() * xhat).abs().sum(0), dy[s].double().abs().sum(0))):
            t += v
    for got, want, mag in ((dw, sums[0], sums[2]), (db, sums[1], sums[3])):
        tol = (rows + 3) * U * mag
        within(got, want, tol + uo(dtype) * (want.abs() + tol), "parameter gradient")


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=str)
@pytest.mark.parametrize("cols", [1, 3, 4, 5, 7, 8, 9, 15, 17, 61, 66, 259, 515, 1001, 2051, 4099, 8195, 16389, 33001])
def test_rows_end_where_they_end(gpu_available, cols, dtype):
    """NaN all round the rows: nothing beyond a row's end or before its start enters a result, and nothing
    beyond is written."""
    say("rows among NaN", cols, dtype)
    rows = 5

    def among_nan(values, lead):
        buf = torch.full((rows, cols + 2 * lead), float("nan"), dtype=values.dtype, device="cuda")
        v = buf[:, lead:lead + cols]
        v.copy_(values)
        return buf, v

    x0, dy0 = normal((rows, cols), dtype, cols), normal((rows, cols), dtype, cols + 1)
    w, b = normal((cols,), BF16, 1, 0.2, 1.0), normal((cols,), BF16, 2)
    want = layer_norm(x0, w, b)
    wantb = layer_norm_bwd(dy0, x0, w, want[1], want[2])
    for lead in (1, 3):
        _, x = among_nan(x0, lead)
        _, dy = among_nan(dy0, lead)
        obuf, out = among_nan(torch.zeros_like(x0), lead)
        gbuf, dx = among_nan(torch.zeros_like(x0), lead)
        wb = torch.full((cols + 2,), float("nan"), dtype=BF16, device="cuda")
        wb[1:-1] = w
        bb = torch.full((cols + 2,), float("nan"), dtype=BF16, device="cuda")
        bb[1:-1] = b
        got = layer_norm(x, wb[1:-1], bb[1:-1], out=out)
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        got = layer_norm_bwd(dy, x, wb[1:-1], want[1], want[2], dx=dx)
        assert all(torch.equal(p, q) for p, q in zip(got, wantb))
        for buf in (obuf, gbuf):
            assert bool(buf[:, :lead].isnan().all()) and bool(buf[:, lead + cols:].isnan().all())
    # a table whose other rows are NaN, and gradients of tokens outside it
    table = torch.full((7, cols), float("nan"), dtype=dtype, device="cuda")
    table[3] = x0[0]
    assert torch.equal(embedding(torch.tensor([3, -1, 3], device="cuda"), table), torch.stack([x0[0], 0 * x0[0], x0[0]]))
    bad = torch.full((3, cols), float("nan"), dtype=dtype, device="cuda")
    bad[1] = dy0[0]
    grad = embedding_bwd(torch.tensor([-1, 2, 9], device="cuda"), bad, 4)
    assert torch.equal(grad[2], dy0[0]) and int(torch.count_nonzero(grad[[0, 1, 3]])) == 0
    many = torch.full((400,), -1, device="cuda")
    many[123] = 2
    bad = torch.full((400, cols), float("nan"), dtype=dtype, device="cuda")
    bad[123] = dy0[0]
    grad = embedding_bwd(many, bad, 4)
    assert torch.equal(grad[2], dy0[0]) and int(torch.count_nonzero(grad[[0, 1, 3]])) == 0


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=str)
@pytest.mark.parametrize("cols", [2, 40, 63, 130, 300, 1001, 4096, 8192, 8203, 16384])
@pytest.mark.parametrize("rows", [15, 16, 17, 33])
def test_layer_norm_bwd_around_few_rows(gpu_available, rows, cols, dtype):
    say("layer norm gradient of few rows", rows, cols, dtype)

    def among_nan(values):
        buf = torch.full((rows, cols + 2), float("nan"), dtype=values.dtype, device="cuda")
        buf[:, 1:-1] = values
        return buf[:, 1:-1]

    x, dy = normal((rows, cols), dtype, cols, 2.0), normal((rows, cols), dtype, 7)
    w = normal((cols,), FP32, 1, 0.2, 1.0)
    want = check_ln_bwd(among_nan(dy), among_nan(x), w)
    _, mean, rstd = layer_norm(x, w)
    inplace = dy.clone()
    got = layer_norm_bwd(inplace, x, w, mean, rstd, dx=inplace)
    assert got[0] is inplace and all(torch.equal(p, q) for p, q in zip(got, want))


# ------------------------------------------------------------------------------------------------
# Gradient norm and clipping
# ------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, FP32], ids=str)
@pytest.mark.parametrize("sizes", [[1] * 8, [1] * 9, [0, 3, 0, 5, 0], [8 * 4096], [8 * 4096 + 1], [8 * 8192], [8 * 8192 + 1],
                                   [4096, 4097, 8191, 8193, 1], [10] * 300, [100_000] * 170], ids=lambda s: f"{len(s)}x{max(s)}")
def test_lists_around_one_workgroup(gpu_available, sizes, dtype):
    say("lists around one workgroup", len(sizes), max(sizes), dtype)
    grads = [whole((n,), dtype, 10 + i) for i, n in enumerate(sizes)]
    total = sum(int(g.double().square().sum()) for g in grads)  # sums of whole numbers: exact in 64 bits
    sumsq = torch.full((), float("nan"), dtype=torch.float64, device="cuda")
    norm = grad_norm(grads, sumsq=sumsq)
    assert float(sumsq) == total and float(norm) == float(torch.tensor(math.sqrt(total), dtype=torch.float64).float())
    max_norm = math.sqrt(total) / 2 + 0.25
    coef = min(1.0, max_norm / (math.sqrt(total) + 1e-6))
    outs = [torch.full_like(g, float("nan")) for g in grads]
    sumsq.fill_(float("nan"))
    assert torch.equal(clip_grad_norm(grads, max_norm, outs=outs, sumsq=sumsq), norm) and float(sumsq) == total
    given = [torch.full_like(g, float("nan")) for g in grads]
    assert torch.equal(grad_clip(grads, sumsq, max_norm, outs=given), norm)
    inplace = [g.clone() for g in grads]
    clip_grad_norm(inplace, max_norm)
    for g, o, p, q in zip(grads, outs, given, inplace):
        # the coefficient's rounding, the product's and the output's
        within(o, g.double() * coef, (uo(dtype) + 2 * U) * (1 + U) * (g.double() * coef).abs(), "clipped")
        assert torch.equal(o, p) and torch.equal(o, q)


# ------------------------------------------------------------------------------------------------
# Embedding
# ------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("tokens", [255, 256, 257, 31 * 32 + 1, 511, 512, 513, 544, 545, 5000, 20000])
def test_runs_of_every_length(gpu_available, tokens):
    """One run of all tokens, and runs that begin and end around borders of pieces."""
    say("runs", tokens)
    for dim, dtype in ((24, FP32), (260, BF16), (1001, FP32)):
        dy = whole((tokens, dim), dtype, tokens)
        for ids in (torch.zeros(tokens, dtype=torch.int64, device="cuda"),
                    torch.arange(tokens, device="cuda") // 31, torch.arange(tokens, device="cuda") // 33,
                    (torch.arange(tokens, device="cuda") * 7) % 5, torch.arange(tokens, device="cuda") // 520):
            vocab = int(ids.max()) + 2
            want = torch.zeros((vocab, dim), dtype=torch.float64, device="cuda").index_add_(0, ids, dy.double())
            got = embedding_bwd(ids, dy, vocab)
            # sums of whole numbers below 2^24: exact in fp32, rounded once
            assert torch.equal(got, want.float().to(dtype))


@pytest.mark.parametrize("vocab", [256, 257, 131072, 131073, 400_000])
def test_many_rows_of_one_workgroup(gpu_available, vocab):
    """Ids that one sorting workgroup owns: more than its lists hold, of hundreds of rows."""
    say("rows of one workgroup", vocab)
    tokens, dim = 30_000, 9
    step = 256 if vocab <= 131072 else 512 if vocab <= 262144 else 1024
    ids = 5 + step * torch.randint(0, max(1, (vocab - 5 + step - 1) // step), (tokens,), device="cuda", generator=gen(1))
    dy = whole((tokens, dim), FP32, 2)
    want = torch.zeros((vocab, dim), dtype=torch.float64, device="cuda").index_add_(0, ids, dy.double())
    assert torch.equal(embedding_bwd(ids, dy, vocab).double(), want)
    assert torch.equal(embedding_bwd(ids.int(), dy, vocab).double(), want)


@pytest.mark.parametrize("vocab,dim,dtype", [(70_001, 1001, FP32), (70_000, 2048, BF16)])
def test_embedding_bwd_of_a_large_table(gpu_available, vocab, dim, dtype):
    """Zeros in a launch of their own, before the sort."""
    say("large table", vocab, dim, dtype)
    tokens = 3000
    ids = torch.randint(-1, vocab + 1, (tokens,), device="cuda", generator=gen(3))
    ids[::3] = 17
    dy = normal((tokens, dim), dtype, 4)
    out = torch.full((vocab, dim), float("nan"), dtype=dtype, device="cuda")
    want, tol = emb_bwd_reference(ids, dy, vocab, 0.5)
    within(embedding_bwd(ids, dy, vocab, 0.5, out=out), want, tol + uo(dtype) * (want.abs() + tol), "gradient")


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=str)
@pytest.mark.parametrize("tokens", [511, 512, 513, 1023, 1024, 1025])
@pytest.mark.parametrize("vocab,dim", [(3, 40), (5, 700), (90, 1001), (4000, 2100), (9000, 12)])
def test_embedding_bwd_around_few_tokens(gpu_available, vocab, dim, tokens, dtype):
    """With and without a sort: every token once, rows of none zero, in place and added."""
    say("few tokens", tokens, vocab, dim, dtype)
    ids = torch.randint(-1, vocab + 1, (tokens,), device="cuda", generator=gen(tokens))
    ids[::4] = vocab // 2
    dy = whole((tokens, dim), dtype, 3)
    inside = (ids >= 0) & (ids < vocab)
    want = torch.zeros((vocab, dim), dtype=torch.float64, device="cuda").index_add_(0, ids[inside], dy[inside].double())
    out = torch.full((vocab, dim), float("nan"), dtype=dtype, device="cuda")
    assert torch.equal(embedding_bwd(ids, dy, vocab, out=out), want.float().to(dtype))
    old = whole((vocab, dim), dtype, 4)
    got = embedding_bwd(ids.int(), dy, vocab, out=old.clone(), accumulate=True)
    assert torch.equal(got, (want + old.double()).float().to(dtype))


def test_embedding_bwd_does_not_depend_on_the_run(gpu_available):
    """The list of runs is made in any order; the sums are not."""
    ids = (torch.rand(40_000, device="cuda", generator=gen(1)).square().square() * 900).long()
    dy = normal((40_000, 130), FP32, 2)
    first = embedding_bwd(ids, dy, 900)
    assert all(torch.equal(embedding_bwd(ids, dy, 900), first) for _ in range(6))


@pytest.mark.parametrize("dim", [1, 9, 300, 1001])
@pytest.mark.parametrize("tokens", [200, 700])
def test_embedding_bwd_against_differences(gpu_available, dim, tokens):
    """The lookup is linear in the table: the loss's difference along one entry is its gradient."""
    vocab, scale = 37, 1.25
    ids = torch.randint(-1, vocab + 1, (tokens,), device="cuda", generator=gen(5))
    dy = normal((tokens, dim), FP32, 6)
    grad = embedding_bwd(ids, dy, vocab, scale)
    table = normal((vocab, dim), FP32, 7)
    base = embedding(ids, table, scale).double()
    for row, col in ((0, 0), (int(ids.max().clamp(max=vocab - 1)), dim - 1), (vocab // 2, dim // 2)):
        moved = table.clone()
        moved[row, col] += 1.0
        diff = (embedding(ids, moved, scale).double() - base) * dy.double()
        # each lookup off by one rounding of an entry below 8 times the scale; the gradient by its sum's
        tol = 2 * U * 8 * scale * float(dy.double()[:, col].abs().sum()) * 2
        assert abs(float(diff.sum()) - float(grad[row, col])) <= tol


# ------------------------------------------------------------------------------------------------
# Refusals
# ------------------------------------------------------------------------------------------------

def test_refusals(gpu_available):
    x, w = normal((6, 40), FP32, 1), normal((40,), FP32, 2)
    y, mean, rstd = layer_norm(x, w)
    ids = torch.tensor([1, 2, 3], device="cuda")
    table = normal((9, 16), BF16, 3)
    dy = normal((3, 16), BF16, 4)
    half = torch.zeros(6, 40, device="cuda", dtype=torch.float16)
    small = torch.empty(8, dtype=torch.uint8, device="cuda")
    none = torch.zeros((), device="cuda")
    for call in (
        lambda: layer_norm(half), lambda: layer_norm(x.cpu()), lambda: layer_norm(x, w.cpu()), lambda: layer_norm(x, w[:-1]),
        lambda: layer_norm(x, w, w.bfloat16()), lambda: layer_norm(x.t()), lambda: layer_norm(x, out=x[:3]),
        lambda: layer_norm(x, out=y.bfloat16()), lambda: layer_norm(x, mean=mean[:2]), lambda: layer_norm(x, rstd=rstd.double()),
        lambda: layer_norm(none), lambda: layer_norm(torch.empty(3, 0, device="cuda")), lambda: layer_norm(x[:, ::2]),
        lambda: layer_norm_bwd(y[:3], x, w, mean, rstd), lambda: layer_norm_bwd(y, x, w, mean[:3], rstd),
        lambda: layer_norm_bwd(y, x, w, mean, rstd, dweight=w.bfloat16()), lambda: layer_norm_bwd(y, x, w, mean, rstd, workspace=small),
        lambda: layer_norm_bwd(y.bfloat16(), x, w, mean, rstd), lambda: layer_norm_bwd(y, x, w, mean, rstd, dbias=w[::2]),
        lambda: embedding(ids.float(), table), lambda: embedding(ids, table.t()), lambda: embedding(ids, table[0]),
        lambda: embedding(ids.cpu(), table), lambda: embedding(ids, table.half()), lambda: embedding(ids, table, out=dy[:2]),
        lambda: embedding(torch.stack([ids, ids])[:, ::2], table), lambda: embedding(ids, table, out=dy.float()),
        lambda: embedding_bwd(ids, dy[:2], 9), lambda: embedding_bwd(ids, dy, -1), lambda: embedding_bwd(ids, dy, 9, accumulate=True),
        lambda: embedding_bwd(ids, dy, 9, out=table[:8]), lambda: embedding_bwd(ids, dy, 9, workspace=small),
        lambda: embedding_bwd(ids, dy, 9, out=table.float()), lambda: embedding_bwd(ids, none, 9),
        lambda: grad_norm([x, x.bfloat16()]), lambda: grad_norm([half]), lambda: grad_norm([x.t()]), lambda: grad_norm([x.cpu()]),
        lambda: grad_norm([x, x.cpu()]), lambda: grad_norm([x], norm=mean), lambda: grad_norm([x], sumsq=none),
        lambda: grad_norm([x], workspace=small), lambda: clip_grad_norm([x], 1.0, outs=[y, y]), lambda: clip_grad_norm([x], 1.0, outs=[w]),
        lambda: clip_grad_norm([x], 1.0, outs=[y.bfloat16()]), lambda: grad_clip([x], none, 1.0),
    ):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: layer_norm(3), lambda: embedding(None, table), lambda: grad_norm(5), lambda: grad_norm([x, 1]),
                 lambda: embedding(ids, table, "a"), lambda: embedding_bwd(ids, dy, 1.5), lambda: layer_norm(x, 1.0)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: layer_norm(x, w, out=x), lambda: layer_norm(x, eps=-1.0), lambda: layer_norm_bwd(y, x, w, mean, rstd, dx=x),
                 lambda: clip_grad_norm([x], -1.0), lambda: clip_grad_norm([x], math.nan), lambda: clip_grad_norm([x, x], 1.0),
                 lambda: embedding_bwd(ids, table[:3], 9, out=table)):
        with pytest.raises(TideError):
            call()
    # what was refused has left no trace
    assert torch.equal(layer_norm(x, w)[0], y)


def test_results_belong_to_the_caller(gpu_available):
    """Outputs passed in are returned as they are; those made have no gradient history."""
    x = normal((4, 24), FP32, 1).requires_grad_()
    out = torch.empty(4, 24, device="cuda")
    y, mean, rstd = layer_norm(x, out=out)
    assert y is out and not mean.requires_grad and mean.shape == (4,)
    norm = torch.empty((), device="cuda")
    assert grad_norm([out], norm=norm) is norm
    assert not layer_norm(x)[0].requires_grad


# ------------------------------------------------------------------------------------------------
# Together
# ------------------------------------------------------------------------------------------------

def test_training_step_example(gpu_available):
    spec = importlib.util.spec_from_file_location("training_step", os.path.join(ROOT, "examples", "training_step.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    say("training step example")
    losses, norms = example.train(steps=30, report=lambda *_: None)
    assert all(map(math.isfinite, losses + norms)) and min(norms) > 0
    assert losses[-1] < 0.9 * losses[0]
    again, _ = example.train(steps=3, report=lambda *_: None)
    assert again == losses[:3]

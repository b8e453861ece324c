"""Calls of the training-step operators as a program makes them: lists that live only as long as the call,
sizes beyond one launch, outputs that autograd has saved, blocks of one buffer."""
import weakref

import pytest
import torch

from all_gather_placement_amd import TideError, clip_grad_norm, embedding, embedding_bwd, grad_clip, grad_norm, layer_norm, layer_norm_bwd, load_step_binding
from test_gpu_step import BF16, FP32, gen, normal, say, uo, whole, within

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------------
# Sequences of tensors
# ------------------------------------------------------------------------------------------------

class Sequence:
    """A sequence that makes its tensors when it is asked for them."""

    def __init__(self, make, n):
        self.make, self.n = make, n

    def __len__(self):
        return self.n

    def __getitem__(self, i):
        if i >= self.n:
            raise IndexError(i)
        return self.make(i)


@pytest.mark.parametrize("kind", ["generator", "sequence", "map"])
@pytest.mark.parametrize("call", ["grad_norm", "clip_grad_norm", "grad_clip"])
def test_made_tensors_live_until_the_call_is_enqueued(gpu_available, call, kind):
    """The stream is asked for last, when everything has been allocated and before a kernel is launched.
    It is refused here, so the call ends without one."""
    say("made tensors", call, kind)
    made = []

    def make(i):
        t = torch.zeros(5000, device="cuda")
        made.append(weakref.ref(t))
        return t

    def tensors():
        return {"generator": lambda: (make(i) for i in range(3)), "sequence": lambda: Sequence(make, 3),
                "map": lambda: map(make, range(3))}[kind]()

    alive = []

    def stream_of(device):
        alive.append([r() is not None for r in made[-n:]])
        raise KeyError("no stream")

    sumsq = torch.ones((), dtype=torch.float64, device="cuda")
    kept = [torch.zeros(5000, device="cuda") for _ in range(3)]
    binding = load_step_binding()
    binding.configure(TideError, stream_of)
    try:
        for args, n in ((dict(grads=tensors), 3), (dict(grads=lambda: kept, outs=tensors), 3),
                        (dict(grads=tensors, outs=tensors), 6)):
            if call == "grad_norm" and "outs" in args:
                continue
            args = {k: f() for k, f in args.items()}
            with pytest.raises(KeyError):
                if call == "grad_norm":
                    grad_norm(args["grads"])
                elif call == "clip_grad_norm":
                    clip_grad_norm(args["grads"], 1.0, outs=args.get("outs"))
                else:
                    grad_clip(args["grads"], sumsq, 1.0, outs=args.get("outs"))
            assert alive.pop() == [True] * n
    finally:
        binding.configure(TideError, torch._C._cuda_getCurrentRawStream)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=str)
def test_generators_give_what_lists_give(gpu_available, dtype):
    say("generators", dtype)
    grads = [normal((20_000 + 4097 * i,), dtype, i) for i in range(40)]
    want = grad_norm([g * 0.5 for g in grads])
    outs = [torch.empty_like(g) for g in grads]
    clip_grad_norm([g * 0.5 for g in grads], 1.0, outs=outs)
    for _ in range(3):
        assert torch.equal(grad_norm(g * 0.5 for g in grads), want)
        got = [torch.empty_like(g) for g in grads]
        assert torch.equal(clip_grad_norm((g * 0.5 for g in grads), 1.0, outs=(o for o in got)), want)
        assert all(map(torch.equal, got, outs))
    assert torch.equal(grad_norm(tuple(g * 0.5 for g in grads)), want)


def test_a_matrix_is_a_list_of_its_rows(gpu_available):
    m = normal((7, 501), FP32, 1)
    want = grad_norm(list(m))
    assert torch.equal(grad_norm(m), want)
    got = m.clone()
    assert torch.equal(clip_grad_norm(got, 1.0), want)
    rows = [r.clone() for r in m]
    clip_grad_norm(rows, 1.0)
    assert torch.equal(got, torch.stack(rows))
    assert float(grad_norm(m[:0])) == 0.0 and float(grad_norm(iter(()))) == 0.0


# ------------------------------------------------------------------------------------------------
# Sizes beyond one launch
# ------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("vocab", [(1 << 30) - 1, (1 << 30) + 3, (1 << 31) - 1])
def test_table_gradient_of_more_rows_than_one_launch_sorts(gpu_available, vocab):
    say("table of many rows", vocab)
    tokens = 1100  # above what is summed without a sort
    ids = torch.randint(0, vocab, (tokens,), device="cuda", generator=gen(1))
    ids[:6] = torch.tensor([0, vocab - 1, vocab // 2, vocab - 2, 1 << 29, (1 << 22) - 1], device="cuda")
    ids[100:200] = vocab - 1
    ids[200:300] = 7
    ids[300] = vocab
    dy = whole((tokens, 1), BF16, 2, 1, 5)
    rows, places = ids.unique(return_inverse=True)
    want = torch.zeros((rows.numel(), 1), dtype=torch.float64, device="cuda").index_add_(0, places, dy.double())
    keep = rows < vocab
    rows, want = rows[keep], want[keep]
    grad = embedding_bwd(ids, dy, vocab)
    # sums of whole numbers: exact in fp32, rounded once
    assert torch.equal(grad[rows], want.float().bfloat16())
    assert int(torch.count_nonzero(grad)) == rows.numel()
    embedding_bwd(ids, dy, vocab, out=grad, accumulate=True)
    assert torch.equal(grad[rows], (want + want.float().bfloat16().double()).float().bfloat16())
    assert int(torch.count_nonzero(grad)) == rows.numel()


@pytest.mark.parametrize("cols", [(1 << 29) + 5, (1 << 29) + 4096])
def test_parameter_gradients_of_more_columns_than_one_launch_joins(gpu_available, cols):
    say("row of many columns", cols)
    x, dy = whole((1, cols), BF16, 1, -2, 3), whole((1, cols), BF16, 2, -2, 3)
    stat = torch.zeros(1, device="cuda")
    dw, db = torch.full((2, cols), float("nan"), dtype=BF16, device="cuda")
    dx, _, _ = layer_norm_bwd(dy, x, None, stat, stat + 1, dweight=dw, dbias=db)
    # one row of whole numbers, mean 0 and rstd 1: products of fp32 are exact, and fit bf16
    assert torch.equal(dw, (x * dy)[0]) and torch.equal(db, dy[0])
    # a thread's sums stay below 2^24; ten additions of sums of at most 4 a column follow, and three operations
    m1 = float(dy.sum(dtype=torch.float64)) / cols
    m2 = float((x * dy).sum(dtype=torch.float64)) / cols
    for part in (slice(0, 1 << 20), slice(cols - (1 << 20), cols)):
        want = dy[0, part].double() - m1 - x[0, part].double() * m2
        tol = 16 * 2.0 ** -24 * 24
        within(dx[0, part], want, tol + uo(BF16) * (want.abs() + tol), "dx")


# ------------------------------------------------------------------------------------------------
# Outputs and autograd
# ------------------------------------------------------------------------------------------------

def _calls():
    """Every call with all of its outputs passed in: (call, inputs, outputs)."""
    x, w = normal((6, 40), FP32, 1), normal((40,), FP32, 2)
    y, mean, rstd = layer_norm(x, w)
    ids, table = torch.tensor([1, 2, 1], device="cuda"), normal((9, 40), FP32, 3)
    dy, dx, h = x.clone(), x.clone(), x[:3].clone()
    dw, db, dtable = w.clone(), w.clone(), table.clone()
    norm, total = torch.zeros(1, device="cuda"), torch.zeros(1, dtype=torch.float64, device="cuda")
    grads, outs = [x.clone(), w.clone(), w[:0]], [x.clone(), w.clone(), w[:0].clone()]
    given = torch.ones(1, dtype=torch.float64, device="cuda")
    return [
        (lambda: layer_norm(x, w, out=y, mean=mean, rstd=rstd), [x, w], [y, mean, rstd]),
        (lambda: layer_norm_bwd(dy, x, w, mean, rstd, dx=dx, dweight=dw, dbias=db), [dy, x, w, mean, rstd], [dx, dw, db]),
        (lambda: layer_norm_bwd(dy, x, w, mean, rstd, dx=dy), [x, w, mean, rstd], [dy]),
        (lambda: embedding(ids, table, out=h), [ids, table], [h]),
        (lambda: embedding_bwd(ids, h, 9, out=dtable), [ids, h], [dtable]),
        (lambda: embedding_bwd(ids, h, 9, out=dtable, accumulate=True), [ids, h], [dtable]),
        (lambda: grad_norm(grads, norm=norm, sumsq=total), grads, [norm, total]),
        (lambda: grad_clip(grads, given, 1.0, outs=outs, norm=norm), [*grads, given], [*outs, norm]),
        (lambda: grad_clip(grads, given, 1.0), [given], grads),
        (lambda: clip_grad_norm(grads, 1.0, outs=outs, norm=norm, sumsq=total), grads, [*outs, norm, total]),
        (lambda: clip_grad_norm((g for g in grads), 1.0), [], grads),
    ]


def test_outputs_passed_in_count_as_written(gpu_available):
    for i, (call, ins, outs) in enumerate(_calls()):
        before = [t._version for t in (*ins, *outs)]
        call()
        after = [t._version for t in (*ins, *outs)]
        assert after[:len(ins)] == before[:len(ins)], i
        assert all(a > b for a, b in zip(after[len(ins):], before[len(ins):])), i
    # refused calls write nothing
    x = normal((4, 8), FP32, 1)
    before = x._version
    with pytest.raises(TideError):
        layer_norm(x, out=x)
    assert x._version == before


def test_backward_refuses_what_was_written_over(gpu_available):
    x = normal((4, 8), FP32, 1).requires_grad_()
    saved = x.exp()
    layer_norm(x, out=saved.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        saved.sum().backward()
    saved = x.exp()
    clip_grad_norm([saved.detach()], 1e-3)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        saved.sum().backward()


def test_outputs_of_inference_mode(gpu_available):
    with torch.inference_mode():
        for call, _, _ in _calls():
            call()
        kept = _calls()
    for call, _, _ in kept:  # used outside it
        call()


def test_negated_views_are_refused(gpu_available):
    """The imaginary part of a conjugate is a view whose memory holds the values of the other sign."""
    z = torch.complex(normal((5, 1), FP32, 1), normal((5, 1), FP32, 2))
    x = z.conj().imag
    assert x.is_neg()
    dense = x.resolve_neg()
    ids = torch.tensor([0, 4], device="cuda")
    for call in (lambda x: layer_norm(x), lambda x: grad_norm([x[0]]), lambda x: clip_grad_norm([x[0]], 1.0),
                 lambda x: embedding(ids[:1], x[:1]), lambda x: embedding_bwd(ids[:1], x[:1], 3)):
        with pytest.raises(ValueError, match="negated view"):
            call(x)
        call(dense)


# ------------------------------------------------------------------------------------------------
# Blocks of columns of one buffer
# ------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, FP32], ids=str)
@pytest.mark.parametrize("rows,cols", [(2, 1), (3, 5), (70, 64), (40, 333), (3000, 1024), (9, 5001), (20, 40001)])
def test_blocks_of_one_buffer(gpu_available, rows, cols, dtype):
    """Inputs and outputs side by side in one buffer: the same bits as apart, and nothing beside them."""
    say("blocks", rows, cols, dtype)
    x, dy = normal((rows, cols), dtype, 1), normal((rows, cols), dtype, 2)
    w = normal((cols,), dtype, 3)
    y, mean, rstd = layer_norm(x, w)
    want = layer_norm_bwd(dy, x, w, mean, rstd)
    buf = torch.full((rows, 4 * cols + 3), float("nan"), dtype=dtype, device="cuda")
    xb, yb, db, gb = (buf[:, i * cols + max(0, i - 1):][:, :cols] for i in range(4))
    xb.copy_(x)
    db.copy_(dy)
    assert torch.equal(layer_norm(xb, w, out=yb)[0], y)
    got = layer_norm_bwd(db, xb, w, mean, rstd, dx=gb)
    assert all(map(torch.equal, got, want))
    for block, value in ((xb, x), (yb, y), (db, dy), (gb, want[0])):
        assert torch.equal(block, value)
    assert bool(buf[:, [2 * cols, 3 * cols + 1, 4 * cols + 2]].isnan().all())
    assert layer_norm_bwd(db, xb, w, mean, rstd, dx=db)[0] is db and torch.equal(db, want[0])
    if cols > 1:
        with pytest.raises(TideError):
            layer_norm(xb, w, out=buf[:, cols - 1:2 * cols - 1])

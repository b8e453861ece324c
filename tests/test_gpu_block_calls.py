"""Calls of the block operators as a program makes them: arguments that do not fit, streams, captured and
replayed calls, outputs that autograd has saved, and all of them together in a block's forward and backward
pass."""
import math

import pytest
import torch

import block_oracle as oracle
from all_gather_placement_amd import (ExpertSort, TideError, dropout, dropout_bwd, expert_combine, expert_combine_bwd,
                                      expert_dispatch, expert_dispatch_bwd, expert_sort, layer_norm, layer_norm_bwd,
                                      load_step_library, rotary, rotary_bwd, rotary_freqs)
from test_gpu_step import BF16, FP32, gen, normal, say, whole, within

pytestmark = pytest.mark.gpu


def ids_of(tokens, choices, experts, seed=1):
    ids = torch.randint(0, experts, (tokens, choices), device="cuda", generator=gen(seed))
    return ids.masked_fill(torch.rand(ids.shape, device="cuda", generator=gen(seed + 1)) < 0.1, -1)


# ------------------------------------------------------------------------------------------------
# Refusals
# ------------------------------------------------------------------------------------------------

def refused(call, *errors):
    with pytest.raises(errors or (ValueError, TypeError, TideError)):
        call()


def test_expert_refusals(gpu_available):
    ids = ids_of(6, 2, 4)
    sort = expert_sort(ids, 4, align=2)
    assert isinstance(sort, ExpertSort) and isinstance(sort, tuple)
    rows = sort.source.numel()
    x, big = normal((6, 16), FP32, 1), normal((rows, 16), FP32, 2)
    w = normal((6, 2), FP32, 3)
    for bad in (ids.float(), ids.short(), ids.T, ids[:, :0], torch.zeros((), dtype=torch.int64, device="cuda"),
                torch.zeros(3, 65, dtype=torch.int64, device="cuda"), ids.cpu(), None, [[1, 2]]):
        refused(lambda: expert_sort(bad, 4))
    for args in (dict(num_experts=0), dict(num_experts=2049), dict(num_experts=-1), dict(num_experts=1 << 40),
                 dict(num_experts=4, align=0), dict(num_experts=4, align=1 << 31), dict(num_experts=4, align=(1 << 31) - 1),
                 dict(num_experts=4, align=2, place=sort.place.long()), dict(num_experts=4, align=2, place=sort.place[:5]),
                 dict(num_experts=4, align=2, source=sort.source[:rows - 1]), dict(num_experts=4, offsets=sort.offsets[:4]),
                 dict(num_experts=4, align=2, source=sort.source.repeat(2)[::2]),
                 dict(num_experts=4, offsets=sort.offsets.float()), dict(num_experts=2.5), dict(num_experts=None)):
        refused(lambda: expert_sort(ids, **args))
    many = ids_of(3000, 2, 4)
    refused(lambda: expert_sort(many, 4, workspace=torch.empty(8, dtype=torch.uint8, device="cuda")))
    for bad in ((sort.place, sort.source), [*sort], None, (sort.place.long(), sort.source, sort.offsets),
                (sort.place[:5], sort.source, sort.offsets), (sort.place, sort.source[:, None], sort.offsets),
                (sort.place.cpu(), sort.source, sort.offsets), (None, None, None), (sort.place.T, sort.source, sort.offsets)):
        refused(lambda: expert_dispatch(x, bad))
        refused(lambda: expert_combine(big, w, bad))
        refused(lambda: expert_combine_bwd(x, big, w, bad))
    for bad in (x.double(), x.half(), x[:5], x[:, :0], x.T, x.cpu(), x[0]):
        refused(lambda: expert_dispatch(bad, sort))
    refused(lambda: expert_dispatch(x, sort, out=big.bfloat16()))
    refused(lambda: expert_dispatch(x, sort, out=big[:-1]))
    refused(lambda: expert_dispatch(x, sort, out=big[:, :15]))
    for bad in (big[:-1], big.double(), big[:, :0], big.cpu()):
        refused(lambda: expert_combine(bad, w, sort))
        refused(lambda: expert_combine_bwd(x, bad, w, sort))
    for bad in (w[:5], w[:, :1], w.double(), w.T, w.cpu(), w.view(-1)):
        refused(lambda: expert_combine(big, bad, sort))
        refused(lambda: expert_combine_bwd(x, big, bad, sort))
    refused(lambda: expert_combine_bwd(x, big, None, sort))
    refused(lambda: expert_combine_bwd(x.bfloat16(), big, w, sort))
    refused(lambda: expert_combine_bwd(x, big, w, sort, dweights=w.bfloat16()))
    refused(lambda: expert_combine_bwd(x, big, w, sort, dweights=w), TideError)  # over the weights
    buf = torch.zeros((rows + 6, 16), device="cuda")
    refused(lambda: expert_combine(buf[:rows], w, sort, out=buf[rows - 1:rows + 5]), TideError)
    refused(lambda: expert_dispatch(buf[:6], sort, out=buf[5:5 + rows]), TideError)
    refused(lambda: expert_combine_bwd(x, buf[:rows], w, sort, drows=buf[1:rows + 1]), TideError)


def test_sort_refuses_outputs_over_each_other(gpu_available):
    ids = ids_of(6, 2, 4).int()
    refused(lambda: expert_sort(ids, 4, place=ids), TideError)
    buf = torch.empty(12, dtype=torch.int32, device="cuda")
    refused(lambda: expert_sort(ids, 4, place=buf.view(6, 2), source=buf), TideError)
    refused(lambda: expert_sort(ids, 4, source=buf, offsets=buf[7:]), TideError)


def test_rotary_refusals(gpu_available):
    x, positions, freqs = normal((6, 2, 8), FP32, 1), torch.zeros((2, 6), device="cuda"), rotary_freqs((1, 3))
    ok = dict(x=x, positions=positions, freqs=freqs, sections=(1, 3))
    rotary(**ok)
    for bad in (dict(x=x.double()), dict(x=x[0, 0]), dict(x=x.transpose(1, 2)), dict(x=x.cpu()), dict(x=x[..., :7]),
                dict(x=x.view(2, 3, 2, 8).transpose(0, 1)), dict(x=torch.zeros(6, 1, 1026, device="cuda")),
                dict(positions=positions.double()), dict(positions=positions[:1]), dict(positions=positions[:, :5]),
                dict(positions=positions.T.contiguous().T), dict(positions=positions[0]), dict(positions=positions.cpu()),
                dict(freqs=freqs.float()), dict(freqs=freqs[:3]), dict(freqs=freqs.repeat(2)[::2]), dict(freqs=freqs.cpu()),
                dict(sections=()), dict(sections=(1, 0)), dict(sections=(1, -1)), dict(sections=(1, 4)), dict(sections=(4,)),
                dict(sections=(1,) * 9), dict(sections=(1, 1 << 40)), dict(sections=4), dict(sections=(1, 3.0)),
                dict(sections=None), dict(pairing="pairs"), dict(pairing=0), dict(pairing=None), dict(out=x.bfloat16()),
                dict(out=x[:5]), dict(out=x.transpose(0, 1)), dict(out=x[:, :1].expand(6, 2, 8))):
        refused(lambda: rotary(**{**ok, **bad}))
        if "x" not in bad:
            refused(lambda: rotary_bwd(**{**{("dy" if k == "x" else k): v for k, v in ok.items()}, **bad}))
    buf = torch.zeros((7, 2, 8), device="cuda")
    refused(lambda: rotary(buf[:6], positions, freqs, (1, 3), out=buf[1:]), TideError)
    refused(lambda: rotary(x, positions, freqs, (1, 3), out=x.view(2, 6, 8).transpose(0, 1)), TideError)


def test_dropout_refusals(gpu_available):
    x = normal((6, 8), FP32, 1)
    seed = torch.zeros(1, dtype=torch.int64, device="cuda")
    ok = dict(x=x, p=0.5, seed=1)
    dropout(**ok)
    for bad in (dict(x=x.double()), dict(x=x.T), dict(x=x.cpu()), dict(x=x[:, :0]), dict(x=x[0, 0]), dict(p=-0.1), dict(p=1.1),
                dict(p=math.nan), dict(p="x"), dict(p=None), dict(seed=1 << 64), dict(seed=-(1 << 63) - 1), dict(seed=1.5),
                dict(seed=None), dict(seed=seed.int()), dict(seed=seed.repeat(2)), dict(seed=seed.cpu()), dict(offset=-1),
                dict(offset=1 << 62), dict(offset=1 << 63), dict(offset=0.5), dict(residual=x.bfloat16()),
                dict(residual=x[:5]), dict(residual=1.0), dict(out=x.bfloat16()), dict(out=x[:5])):
        refused(lambda: dropout(**{**ok, **bad}), ValueError, TypeError, TideError, OverflowError)
    buf = torch.zeros((7, 8), device="cuda")
    refused(lambda: dropout(buf[:6], 0.5, 1, out=buf[1:]), TideError)
    refused(lambda: dropout(x, 0.5, 1, residual=buf[:6], out=buf[1:]), TideError)


def test_negated_views_are_refused(gpu_available):
    z = torch.complex(normal((5, 1, 2), FP32, 1), normal((5, 1, 2), FP32, 2))
    x = z.conj().imag
    assert x.is_neg()
    sort = expert_sort(torch.zeros((5, 1), dtype=torch.int64, device="cuda"), 1)
    positions, freqs = torch.zeros((1, 5), device="cuda"), rotary_freqs((1,))
    flat = x[:, 0, :1]
    for call in (lambda: expert_dispatch(flat, sort), lambda: expert_combine(flat, None, sort), lambda: dropout(flat, 0.5, 1),
                 lambda: dropout(flat.resolve_neg(), 0.5, 1, residual=flat), lambda: rotary(x, positions, freqs, (1,))):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------------------------------------------
# Outputs and autograd
# ------------------------------------------------------------------------------------------------

def test_outputs_passed_in_count_as_written(gpu_available):
    ids = ids_of(6, 2, 4)
    sort = expert_sort(ids, 4)
    x, rows, w = normal((6, 16), FP32, 1), normal((12, 16), FP32, 2), normal((6, 2), FP32, 3)
    y, out, dw = x.clone(), rows.clone(), w.clone()
    h, positions, freqs = x.view(6, 2, 8).clone(), torch.ones((1, 6), device="cuda"), rotary_freqs((4,))
    t = h.clone()
    calls = [
        (lambda: expert_sort(ids, 4, place=sort.place, source=sort.source, offsets=sort.offsets), [ids], [*sort]),
        (lambda: expert_dispatch(x, sort, out=out), [x, *sort], [out]),
        (lambda: expert_dispatch_bwd(rows, sort, out=y), [rows, *sort], [y]),
        (lambda: expert_combine(rows, w, sort, out=y), [rows, w, *sort], [y]),
        (lambda: expert_combine_bwd(x, rows, w, sort, drows=out, dweights=dw), [x, rows, w], [out, dw]),
        (lambda: expert_combine_bwd(x, rows, w, sort, drows=rows), [x, w], [rows]),
        (lambda: rotary(h, positions, freqs, (4,), out=t), [h, positions, freqs], [t]),
        (lambda: rotary_bwd(h, positions, freqs, (4,), out=h), [positions, freqs], [h]),
        (lambda: dropout(x, 0.5, 1, residual=w.new_ones(6, 16), out=y), [x], [y]),
        (lambda: dropout_bwd(x, 0.5, 1, out=x), [], [x]),
    ]
    for i, (call, ins, outs) in enumerate(calls):
        before = [v._version for v in (*ins, *outs)]
        call()
        after = [v._version for v in (*ins, *outs)]
        assert after[:len(ins)] == before[:len(ins)], i
        assert all(a > b for a, b in zip(after[len(ins):], before[len(ins):])), i
    saved = x.clone().requires_grad_().exp()
    dropout(x, 0.5, 1, out=saved.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        saved.sum().backward()
    with torch.inference_mode():
        a = normal((6, 16), FP32, 1)
        dropout(a, 0.5, 1, out=a)
        expert_sort(ids, 4)


# ------------------------------------------------------------------------------------------------
# Streams, workspaces and graphs
# ------------------------------------------------------------------------------------------------

class Step:
    """The operators in a row, on buffers of its own: forward and backward."""

    def __init__(self, tokens=700, heads=4, dim=32, choices=3, experts=12, seed=1):
        self.experts = experts
        self.x, self.dy = normal((tokens, heads, dim), BF16, seed), normal((tokens, heads * dim), BF16, seed + 1)
        self.positions = torch.arange(2 * tokens, device="cuda").view(2, tokens) + seed
        self.freqs = rotary_freqs((6, 10))
        self.ids, self.w = ids_of(tokens, choices, experts, seed + 2), normal((tokens, choices), FP32, seed + 4)
        self.seed = torch.tensor([seed], device="cuda")

    def run(self, stream=None):
        on = dict(stream=stream)
        flat = (len(self.x), -1)
        q = rotary(self.x, self.positions, self.freqs, (6, 10), "neighbours", **on)
        h = dropout(q.view(flat), 0.2, self.seed, offset=5, residual=self.x.view(flat), **on)
        sort = expert_sort(self.ids, self.experts, align=8, **on)
        rows = expert_dispatch(h, sort, **on)
        y = expert_combine(rows, self.w, sort, **on)
        drows, dw = expert_combine_bwd(self.dy, rows, self.w, sort, **on)
        dh = expert_dispatch_bwd(drows, sort, **on)
        dq = dropout_bwd(dh, 0.2, self.seed, offset=5, **on)
        dx = rotary_bwd(dq.view(self.x.shape), self.positions, self.freqs, (6, 10), "neighbours", **on)
        return [q, h, *sort, rows, y, drows, dw, dh, dq, dx]

    def change(self, seed):
        other = Step(*self.sizes(), seed=seed)
        for name in ("x", "dy", "positions", "ids", "w", "seed"):
            getattr(self, name).copy_(getattr(other, name))

    def sizes(self):
        return (*self.x.shape, self.ids.shape[1], self.experts)


def test_two_streams(gpu_available):
    """Calls on two streams at once, tensors of the current one: what one call after another gives.  The tensors
    live until both streams are done."""
    a, b = Step(seed=1), Step(tokens=4001, seed=40)
    want = [a.run(), b.run()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for given in (True, False):
        kept = []
        for _ in range(5):
            for s, stream in ((a, streams[0]), (b, streams[1])):
                if given:
                    kept.append(s.run(stream.cuda_stream if s is a else stream))
                else:
                    with torch.cuda.stream(stream):
                        kept.append(s.run())
        torch.cuda.synchronize()
        for i, got in enumerate(kept):
            assert all(map(torch.equal, got, want[i % 2])), i


def test_captured_and_replayed(gpu_available):
    """A graph of all operators reads the tensors and the seed of the moment; eager work goes on between."""
    for tokens in (700, 6000):  # a sort in one launch and in two
        step = Step(tokens=tokens)
        step.run()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step.run()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step.run()
        seen = []
        for seed in (3, 4, 5, 3):
            step.change(seed)
            for g in got:
                g.zero_()
            graph.replay()
            torch.cuda.synchronize()
            want = step.run()
            other = Step(tokens=300, seed=seed).run()
            assert all(map(torch.equal, got, want)), (tokens, seed)
            seen.append(got[1].clone())
            del want, other
        assert torch.equal(seen[0], seen[3]) and not torch.equal(seen[0], seen[1])


def test_workspaces_and_results_of_every_run_are_the_same(gpu_available):
    step = Step(tokens=9000, choices=7)
    want = step.run()
    size = load_step_library().tide_expert_sort_workspace(9000, 7, 12)
    assert size > 0
    ws = torch.full((size + 64,), 255, dtype=torch.uint8, device="cuda")
    sort = expert_sort(step.ids, 12, align=8, workspace=ws[:size])
    assert all(map(torch.equal, sort, want[2:5])) and bool((ws[size:] == 255).all())
    for _ in range(3):
        assert all(map(torch.equal, step.run(), want))


# ------------------------------------------------------------------------------------------------
# Together
# ------------------------------------------------------------------------------------------------

def test_a_block_forward_and_backward(gpu_available):
    """Rotary positions, dropout and a residual, experts and their weights, dropout again: forward and every
    gradient against autograd of the definitions in 64 bits.  Quarter turns, p = 1/2 and whole numbers keep each
    result a whole number below 2^24 and a rest: of 8 quarters, off by 2^-51 of 4 pi, a sine or cosine that should
    be 0 is below 2^-46.  With |x| <= 2 that is 2^-45 beside a whole number; what follows multiplies it by less
    than 2 (dropout), 48 (a matrix of at most 1), 6 (three weights of at most 2) and 2 again, 2^11 in all, and fp32
    keeps no rest beside a number other than 0.  The products that the weights' and matrices' gradients add up are
    of at most 2^13 such numbers, of which the other factor is below 2^10: less than 2^-45 + 11 + 23 in all."""
    say("a block")
    tokens, heads, dim, choices, experts, width = 90, 3, 16, 3, 5, 48
    x = whole((tokens, heads, dim), FP32, 1, -2, 3)
    ids, w = ids_of(tokens, choices, experts), whole((tokens, choices), FP32, 2, -2, 3)
    mats = [whole((width, width), FP32, 10 + e, -1, 2) for e in range(experts)]
    positions = torch.randint(0, 9, (3, tokens), device="cuda", generator=gen(3))
    freqs = torch.full((8,), math.pi / 2, dtype=torch.float64, device="cuda")
    dy = whole((tokens, width), FP32, 4, -1, 2)
    sections, seeds = (3, 3, 2), (5, -9)

    q = rotary(x, positions, freqs, sections).view(tokens, width)
    h = dropout(q, 0.5, seeds[0], residual=x.view(tokens, width))
    sort = expert_sort(ids, experts, align=4)
    rows = expert_dispatch(h, sort)
    at = sort.offsets.tolist()
    mid = torch.zeros_like(rows)
    for e in range(experts):
        mid[at[e]:at[e + 1]] = rows[at[e]:at[e + 1]] @ mats[e]
    y = dropout(expert_combine(mid, w, sort), 0.5, seeds[1], offset=1000, residual=h)

    dc = dropout_bwd(dy, 0.5, seeds[1], offset=1000)
    dmid, dw = expert_combine_bwd(dc, mid, w, sort)
    drows, dmats = torch.zeros_like(rows), []
    for e in range(experts):
        part = slice(at[e], at[e + 1])
        drows[part] = dmid[part] @ mats[e].T
        dmats.append(rows[part].T @ dmid[part])
    dh = expert_dispatch_bwd(drows, sort) + dy
    dq = dropout_bwd(dh, 0.5, seeds[0])
    dx = rotary_bwd(dq.view(x.shape), positions, freqs, sections) + dh.view(x.shape)

    X, W = x.cpu().double().requires_grad_(), w.cpu().double().requires_grad_()
    M = [m.cpu().double().requires_grad_() for m in mats]
    keep = [oracle.keep(tokens * width, 0.5, s, o).view(tokens, width).double() * 2 for s, o in zip(seeds, (0, 1000))]
    axis = torch.repeat_interleave(torch.arange(3), torch.tensor(sections))
    turns = positions.cpu()[axis].T[:, None] % 4
    c, s = torch.tensor([1.0, 0, -1, 0]).double()[turns], torch.tensor([0.0, 1, 0, -1]).double()[turns]
    u, v = X[..., :8], X[..., 8:]
    Q = torch.cat([u * c - v * s, v * c + u * s], -1).reshape(tokens, width)
    H = Q * keep[0] + X.reshape(tokens, width)
    C = torch.zeros(tokens, width, dtype=torch.float64)
    for j in range(choices):
        of = ids.cpu()[:, j]
        C = C + sum(torch.where((of == e)[:, None], H @ M[e], 0.0) for e in range(experts)) * W[:, j, None]
    Y = C * keep[1] + H
    Y.backward(dy.cpu().double())
    assert float(Y.detach().abs().max()) < 2 ** 23 and float(X.grad.abs().max()) < 2 ** 23
    for name, got, want in (("y", y, Y), ("dx", dx, X.grad), ("dw", dw, W.grad)):
        within(got.cpu(), want.detach(), 2.0 ** -11, name)
    for got, want in zip(dmats, M):
        within(got.cpu(), want.grad, 2.0 ** -11, "matrix")
    assert float(Y.detach().abs().max()) > 0 and float(W.grad.abs().max()) > 0


def test_beside_layer_norm(gpu_available):
    """Layer norm's results go through the experts and back, each stage against its definition on its inputs."""
    x, weight = normal((300, 200), FP32, 1), normal((200,), FP32, 2)
    y, mean, rstd = layer_norm(x, weight)
    sort = expert_sort(ids_of(300, 2, 6), 6, align=16)
    rows = expert_dispatch(y, sort)
    back = expert_dispatch_bwd(rows, sort)
    times = (sort.place >= 0).sum(1, keepdim=True)
    assert torch.equal(back, y * times)  # one or two times the same number: exact
    dx, _, _ = layer_norm_bwd(back, x, weight, mean, rstd)
    again, _, _ = layer_norm_bwd(y * times, x, weight, mean, rstd)
    assert torch.equal(dx, again)

"""The operators around the routed experts together, as a block runs them: norm ->
expert selection -> sort -> 8-bit products -> back with weights -> norm and residual,
in serving (eager, captured, on streams of their own) and in training."""
import numpy as np
import pytest
import torch

import dequant_iqk_moe_amd as q
from oracle import block

pytestmark = pytest.mark.gpu

HIDDEN, INNER, E, K = 256, 192, 12, 3


class Block:
    def __init__(self, seed=0, dtype=torch.bfloat16):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)
        weights = lambda out, n: q.Int8Weights((r(E, out, n) * 40).round().clamp(-127, 127).to(torch.int8).cuda(),
                                               (torch.rand(E, out, generator=g) + 0.5).cuda() / (40 * n ** 0.5))
        self.dtype = dtype
        self.router = (r(E, HIDDEN) / HIDDEN ** 0.5).cuda()
        self.first, self.post, self.next = ((1 + 0.1 * r(HIDDEN)).to(dtype).cuda() for _ in range(3))
        self.gate = torch.sigmoid(r(HIDDEN)).to(dtype).cuda()
        self.up, self.down = weights(2 * INNER, HIDDEN), weights(HIDDEN, INNER)

    def __call__(self, x, stream=None):
        s = dict(stream=stream)
        _, h = q.block_norm(x, next_weight=self.first, **s)
        ids, w = q.router_topk(h.float() @ self.router.t(), K, **s)
        xs, offsets, place = q.moe_sort(h, ids, E, **s)
        act = q.swiglu(q.int8_grouped(self.up, xs, offsets, **s), **s)
        ys = q.int8_grouped(self.down, act, offsets, out_dtype=self.dtype, **s)
        y = q.moe_unsort(ys, place, w, out_dtype=self.dtype, **s)
        return q.block_norm(x, y, self.post, self.gate, self.next, beta=0.5, **s)


def _x(T, seed=1, dtype=torch.bfloat16):
    return torch.randn(T, HIDDEN, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def _oracle(b, x, routed):
    """The block in float64, from the library's choice of experts; int8 codes by the oracle."""
    d = lambda t: t.double().cpu().numpy()
    ids, w = (t.cpu().numpy() for t in routed)
    h = block.block_norm(d(x), nxt=d(b.first))[1]
    xs, offsets, place = block.sort(h, ids, E)
    codes = lambda m: (m.codes.cpu().numpy(), m.scales.cpu().numpy())
    gu = block.int8_grouped(*codes(b.up), *block.quantize(xs), offsets).astype(np.float64)
    act = gu[:, :INNER] / (1 + np.exp(-gu[:, :INNER])) * gu[:, INNER:]
    ys = block.int8_grouped(*codes(b.down), *block.quantize(act), offsets)
    y, _ = block.unsort(ys, place, w)
    return block.block_norm(d(x), y, d(b.post), d(b.gate), d(b.next), beta=0.5)


@pytest.mark.parametrize("T", [1, 5, 130, 1000])
def test_block_against_the_oracle(T):
    """A bfloat16 value is off by 2^-9 of itself in the mean of squares / sqrt(3) (h, act, ys, y) and a code by 1 / (2 sqrt 3)
    of a step of 2 / 127 of the rms and more: 1.5 % of a row's norm for a largest value of three to four times the rms,
    twice; the residual, twice the routed part's norm and more, carries none of it.  Bar: 3 % in norm."""
    b, x = Block(), _x(T)
    r, h = b(x)
    routed = q.router_topk(q.block_norm(x, next_weight=b.first)[1].float() @ b.router.t(), K)
    for got, want in zip((r, h), _oracle(b, x, routed)):
        off = np.linalg.norm(got.double().cpu().numpy() - want) / np.linalg.norm(want)
        assert off <= 0.03, off


@pytest.mark.parametrize("T", [1, 70, 3100])
def test_captured_and_replayed(T):
    b = Block()
    static, inputs = _x(T), [_x(T, s) for s in (2, 3, 4)]
    eager = [[t.clone() for t in b(x)] for x in inputs]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b(static)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = b(static)
    for _ in range(2):
        for x, want in zip(inputs, eager):
            static.copy_(x)
            g.replay()
            assert torch.equal(b(inputs[0])[0], eager[0][0])  # the program's own work between the replays
            torch.cuda.synchronize()
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_two_graphs_do_not_share_memory():
    b = Block()
    xs = [_x(3100, 2), _x(2900, 3)]
    want = [[t.clone() for t in b(x)] for x in xs]
    graphs, outs = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(b(x))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for out, w in zip(outs, want):
            assert torch.equal(out[0], w[0]) and torch.equal(out[1], w[1])


def test_calls_on_other_streams():
    b, x = Block(), _x(900)
    want = b(x)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(b(x))
    torch.cuda.synchronize()
    for out in got:
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    # the stream as an argument, as an object and as a handle: results belong to it
    s = streams[0]
    for given in (s, s.cuda_stream):
        s.wait_stream(torch.cuda.current_stream())
        r, h = q.block_norm(x, x, b.post, b.gate, b.next, stream=given)
        xs, offsets, place = q.moe_sort(x, torch.zeros(900, 2, dtype=torch.int32, device="cuda"), E, stream=given)
        y = q.moe_unsort(xs, place, stream=given)
        z = q.int8_grouped(b.up, xs, offsets, stream=given)
        torch.cuda.synchronize()
        r2, h2 = q.block_norm(x, x, b.post, b.gate, b.next)
        assert torch.equal(r, r2) and torch.equal(h, h2) and torch.equal(y, 2 * x.float())
        assert torch.equal(z, q.int8_grouped(b.up, xs, offsets))


def _train(b, x, w_first, w_post, w_gate, w_next, router, experts):
    """Norms, router and float experts, all trained: through the library's calls."""
    _, h = q.block_norm(x, next_weight=w_first)
    ids, w = q.router_topk(h @ router.t(), K, scoring="sigmoid")
    xs, offsets, place = q.moe_sort(h, ids, E)
    parts = offsets.tolist()
    ys = torch.cat([xs[parts[e]:parts[e + 1]] @ experts[e] for e in range(E)])
    y = q.moe_unsort(ys, place, w)
    return (*q.block_norm(x, y, w_post, w_gate, w_next, beta=0.5), ids)


def _train_plain(x, w_first, w_post, w_gate, w_next, router, experts, ids):
    rms = lambda v: v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6)
    h = rms(x) * w_first
    s = torch.sigmoid(h @ router.t()).gather(1, ids.long())
    w = s / s.sum(-1, keepdim=True)
    y = (w[..., None] * torch.einsum("tn,tknm->tkm", h, experts[ids.long()])).sum(1)
    r = x + 0.5 * (w_gate * (rms(y) * w_post))
    return r, rms(r) * w_next


def test_training_step_against_autograd_in_float64():
    """Gradients of every leaf.  Sums of up to 256 float32 products, thrice in a row and back, of rounding 2^-24 each that
    grows like its root: 1e-6 of a gradient's norm; bar 2e-5."""
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g)
    T = 50
    leaves = [r(T, HIDDEN), 1 + 0.1 * r(HIDDEN), 1 + 0.1 * r(HIDDEN), r(HIDDEN), 1 + 0.1 * r(HIDDEN), r(E, HIDDEN) / 16,
              r(E, HIDDEN, HIDDEN) / 16]
    dr, dh = r(T, HIDDEN), r(T, HIDDEN)
    mine = [t.cuda().requires_grad_() for t in leaves]
    out_r, out_h, ids = _train(None, *mine)
    torch.autograd.backward([out_r, out_h], [dr.cuda(), dh.cuda()])
    theirs = [t.double().requires_grad_() for t in leaves]
    want_r, want_h = _train_plain(*theirs, ids.cpu())
    torch.autograd.backward([want_r, want_h], [dr.double(), dh.double()])
    rel = lambda a, b: float((a.detach().cpu().double() - b).norm() / b.norm())
    assert rel(out_r, want_r.detach()) < 2e-5 and rel(out_h, want_h.detach()) < 2e-5
    for a, b in zip(mine, theirs):
        assert rel(a.grad, b.grad) < 2e-5


def test_captured_training_calls():
    """Forward and gradient calls in one graph, replayed with other inputs, every replay against eager ones."""
    T, n = 700, 264
    g = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g).cuda()
    w = [1 + 0.1 * r(n), r(n), 1 + 0.1 * r(n)]
    route = r(T, 15)
    ids = torch.randint(-1, E, (T, 15), generator=g, dtype=torch.int32).cuda()

    def step(x, ids, route, dr):
        xs, offsets, place = q.moe_sort(x, ids, E)  # 10500 pairs: with a workspace
        y = q.moe_unsort(xs, place, route)
        r, h = q.block_norm(x, y, w[0], w[1], w[2])
        grads = q.block_norm_grad(x, y, dr, dr, post_weight=w[0], gate=w[1], next_weight=w[2])
        d_xs, d_route = q.moe_unsort_grad(grads[1], xs, place, route)
        return (r, h, *grads, d_route, q.moe_unsort(d_xs, place), offsets, place)

    static = [r(T, n), ids.clone(), route.clone(), r(T, n)]
    inputs = [[r(T, n), torch.randint(-1, E, (T, 15), generator=g, dtype=torch.int32).cuda(), r(T, 15), r(T, n)] for _ in range(3)]
    want = [[t.clone() for t in step(*v)] for v in inputs]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(*static)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*static)
    for _ in range(2):
        for v, ref in zip(inputs, want):
            for a, b in zip(static, v):
                a.copy_(b)
            graph.replay()
            assert torch.equal(step(*inputs[0])[0], want[0][0])
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, ref))


def test_autograd_on_another_stream():
    """The stream argument with gradients: the forward call and its gradient both run there."""
    x = _x(300, dtype=torch.float32).requires_grad_()
    w = torch.ones(HIDDEN, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    _, h = q.block_norm(x, next_weight=w, stream=s)
    dh = _x(300, 9, torch.float32)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        loss = (h * dh).sum()  # h's gradient is dh, unrounded
    s.synchronize()
    loss.backward()
    torch.cuda.synchronize()
    assert torch.equal(x.grad, q.block_norm_grad(x.detach(), None, None, dh, next_weight=w)[0])

"""The example of a prompt with branches: the recurrence, normed and turned heads into the cache, a window with first tokens
kept, and attention behind a shared prefix, together against a dense fp32 computation.

Bounds.  Every bf16 rounding is off by at most 2^-8 of its value, about 2^-9.5 of it in the mean square.  The served path
rounds some eight times per layer and a few times more at the ends, 30 in all; independent roundings of that size add up to
sqrt(30) 2^-9.5 < 0.008 of a signal, and the layers pass an error on with a gain of about one each: 0.03.  A gradient passes
as many roundings again on its way back, sqrt(60) 2^-9.5 < 0.011; behind a softmax it is a difference from a mean, which
loses a few times that: 0.06."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def branches():
    import __graft_entry__
    __graft_entry__.build()
    from examples import branches
    return branches


def test_branches_of_a_prompt(branches):
    assert branches.serve(quiet=True) < 0.03


def test_gradients_of_a_training_step(branches):
    errs = branches.gradients(quiet=True)
    assert all(e < 0.06 for e in errs.values()), errs


def test_decoding_from_a_graph(branches):
    """A captured step of all branches, replayed over new tokens and lengths, gives the bits of the same calls made one by one."""
    w, gen = branches.weights("cuda"), torch.Generator().manual_seed(3)
    prompt = torch.randint(0, branches.VOCAB, (1, 75), generator=gen).tolist()
    more = torch.randint(0, branches.VOCAB, (4, branches.BRANCHES, 1), generator=gen).cuda()
    slots = list(range(1, 1 + branches.BRANCHES))
    rows, prefix = torch.tensor(slots, device="cuda"), torch.tensor([64], dtype=torch.int32, device="cuda")

    def server():
        s = branches.Server(w)
        s.step([0], prompt)
        s.fork(0, slots)
        return s

    eager, want = server(), []
    for ids in more:
        eager.grow(slots, 1)
        want.append(eager.forward(rows, ids, prefix))
    s, ids = server(), more[0].clone()
    s.grow(slots, 1)
    assert torch.equal(s.forward(rows, ids, prefix), want[0])  # also loads what a capture must not
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        logits = s.forward(rows, ids, prefix)
    for i in range(1, len(more)):
        ids.copy_(more[i])
        s.grow(slots, 1)
        graph.replay()
        assert torch.equal(logits, want[i]), i
    assert torch.equal(s.state, eager.state)


def test_captured_training_pass(branches):
    """Forward and backward() of both operators with gradients, captured and replayed over new inputs: the bits of eager
    calls.  The eager graphs are gone by then, and the leaves of the captured one are its own."""
    import gated_deltanet_linear_15_gb300 as g
    t, width = 130, branches.WIDTH
    gen = torch.Generator().manual_seed(4)
    angles = g.rotary_table(t, branches.D)
    positions = torch.arange(t, dtype=torch.int32, device="cuda")
    draws = [[torch.randn(1, t, width, generator=gen).cuda() for _ in range(3)] for _ in range(2)]

    def run(u, a, dy, weight):
        y, last = g.gated_linear_recurrence(u, branches.log_gate(a))
        q, _ = g.norm_rotary_embedding(y.view(t, branches.H, branches.D), None, weight, None, angles, positions)
        (q * dy.view_as(q)).sum().add(last.sum()).backward()
        return q

    def leaves(u, a, dy):
        weight = torch.linspace(0.5, 1.5, branches.D, device="cuda")
        return [x.clone().requires_grad_() for x in (u, a)] + [dy.clone(), weight.requires_grad_()]

    def eager(draw):
        args = leaves(*draw)
        q = run(*args).detach()
        return [q] + [args[i].grad for i in (0, 1, 3)]

    want = [eager(d) for d in draws]
    args = leaves(*draws[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(*args)
    torch.cuda.current_stream().wait_stream(side)
    for i in (0, 1, 3):
        args[i].grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = run(*args).detach()
    for d, wanted in zip(draws, want):
        with torch.no_grad():
            for i in range(3):
                args[i].copy_(d[i])
        for i in (0, 1, 3):
            args[i].grad.zero_()
        graph.replay()
        for got, exact in zip([q] + [args[i].grad for i in (0, 1, 3)], wanted):
            assert torch.equal(got, exact)

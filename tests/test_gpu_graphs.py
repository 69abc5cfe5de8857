"""What a stream capture records of a plan, on the GPU: a scan or an assign that is only recorded
does not count for eager calls, and a graph replayed after another route of its plan computes with
that route."""

import numpy as np
import pytest
import torch

import combine_shuffling_amd as cs

from gpu_util import say

pytestmark = pytest.mark.gpu

PLANS = [
    ("fused scan", 600, dict(num_ranks=4)),
    ("dedup", 600, dict(num_ranks=4, ranks_per_node=2, node_dedup=True)),
    ("banded", 600, dict(num_ranks=4, band_tokens=256)),
    ("many tiles", 16300, dict(num_ranks=4)),      # the route scans by itself
]
E, K, H, N = 66, 3, 72, 40


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


class Calls:
    """The calls that read a plan's slots or offsets, on inputs that stay the same."""

    def __init__(self, T, kw, dev):
        g = torch.Generator(device=dev)
        g.manual_seed(T)
        rand = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
        self.T, self.kw, self.dev = T, kw, dev
        self.x, self.grad_out = rand(T, H).bfloat16(), rand(T, H).bfloat16()
        self.rows, self.w = rand(T * K, H).bfloat16(), rand(T, K)
        self.weights = rand(E, N, H).bfloat16()
        self.codes = torch.randint(0, 0x78, (T * K, H), generator=g, dtype=torch.uint8, device=dev)
        self.scales = torch.ones(T * K, (H + 127) // 128, device=dev)
        skew = torch.arange(E, device=dev) / 16
        self.routes = [torch.topk(rand(T, E) + s, K, dim=1).indices.int().contiguous()
                       for s in (0 * skew, skew)]
        self.want = [self.all(self.plan().route(r)) for r in self.routes]
        torch.cuda.synchronize()
        for n in self.want[0]:
            assert not torch.equal(self.want[0][n], self.want[1][n]), n

    def plan(self):
        return cs.Plan(self.T, H, E, K, **self.kw)

    def routed(self, route):
        # a workspace whose slots are out of range until something writes them
        p = self.plan()
        ws = torch.full((p.workspace_bytes,), 255, dtype=torch.uint8, device=self.dev)
        return p.route(route, ws)

    def all(self, p, which=("grad_x", "grad_y", "out", "y", "fp8", "hier")):
        r = {}
        if "grad_x" in which:
            r["grad_x"] = p.dispatch_backward(self.rows)
        if "grad_y" in which:
            r["grad_y"], r["grad_w"] = p.combine_backward(self.grad_out, self.rows, self.w)
        if "out" in which:
            r["out"] = p.combine(self.rows, self.w)
        if "y" in which:
            r["y"] = p.expert_linear(self.rows, self.weights)[0]
        if "fp8" in which:
            r["fp8"] = p.combine_fp8(self.codes, self.scales, self.w)
        if "hier" in which and p.node_dedup:
            r["hier"] = p.combine_hier(self.rows, self.w)
        return r

    def check(self, got, i, what):
        bad = [n for n in got if not torch.equal(got[n], self.want[i][n])]
        assert bad == [], (what, i, bad)


def captured(call):
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    return graph, out


ALONE = [(w, *p) for w in ("grad_x", "grad_y", "out", "y", "fp8", "hier") for p in PLANS
         if w != "hier" or "node_dedup" in p[2]]


@pytest.mark.parametrize("which,name,T,kw", ALONE, ids=[f"{a[0]}-{a[1]}" for a in ALONE])
@pytest.mark.parametrize("dispatched", [False, True], ids=["routed", "dispatched"])
def test_call_captured_on_its_own(which, name, T, kw, dispatched, dev):
    say(f"[graphs] {which} captured alone, {name}, dispatched before: {dispatched}")
    c = Calls(T, kw, dev)
    p = c.routed(c.routes[0])
    if dispatched:
        p.dispatch(c.x)
    graph, outs = captured(lambda: [c.all(p, (which,)) for _ in range(2)])
    c.check(c.all(p), 0, "eager, before the first replay")
    for n, i in enumerate((0, 1, 0, 1)):
        p.route(c.routes[i])
        if n % 2:
            c.check(c.all(p), i, "eager, before the replay")
        for o in outs:
            for t in o.values():
                t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for o in outs:
            c.check(o, i, "replayed")
        c.check(c.all(p), i, "eager, after the replay")


@pytest.mark.parametrize("name,T,kw", PLANS, ids=[p[0] for p in PLANS])
def test_captured_dispatch_does_not_count_for_eager_calls(name, T, kw, dev):
    say(f"[graphs] dispatch captured alone, {name}")
    c = Calls(T, kw, dev)
    p = c.routed(c.routes[0])
    graph, (recv, _) = captured(lambda: p.dispatch(c.x))
    c.check(c.all(p), 0, "eager, before the first replay")
    want = recv.clone().zero_()
    p.dispatch(c.x, want)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(recv, want)


@pytest.mark.parametrize("name,T,kw", PLANS, ids=[p[0] for p in PLANS])
@pytest.mark.parametrize("inside", ["route", "route and dispatch", "everything"])
def test_captured_route(name, T, kw, inside, dev):
    # The route itself is recorded and replayed on other routings: eager calls between the replays
    # take the routing of the last one.
    say(f"[graphs] {inside} captured, {name}")
    c = Calls(T, kw, dev)
    ids = c.routes[0].clone()
    p = c.routed(ids)

    def call():
        p.route(ids)
        if inside != "route":
            p.dispatch(c.x)
        return c.all(p) if inside == "everything" else {}

    graph, outs = captured(call)
    for n, i in enumerate((0, 1, 0, 1, 1, 0)):
        ids.copy_(c.routes[i])
        for t in outs.values():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        c.check(outs, i, "replayed")
        for _ in range(1 + n % 2):
            c.check(c.all(p), i, "eager, after the replay")
    # and an eager route of the plan ends that
    p.route(c.routes[1])
    for _ in range(2):
        c.check(c.all(p), 1, "eager, after a route")


@pytest.mark.parametrize("name,T,kw", PLANS, ids=[p[0] for p in PLANS])
def test_graphs_that_share_a_plan(name, T, kw, dev):
    # Two graphs that route one plan on ids of their own, and one with the calls alone, recorded
    # after them.
    say(f"[graphs] three graphs of one plan, {name}")
    c = Calls(T, kw, dev)
    p = c.routed(c.routes[0])
    routes = [captured(lambda r=r: p.route(r))[0] for r in c.routes]
    alone, outs = captured(lambda: c.all(p))
    for n, i in enumerate((1, 0, 0, 1, 0, 1, 0)):
        if n < 5:
            routes[i].replay()
        else:
            p.route(c.routes[i])      # eager ones
        for t in outs.values():
            t.zero_()
        if n % 2:
            c.check(c.all(p), i, "eager")
        alone.replay()
        torch.cuda.synchronize()
        c.check(outs, i, "replayed")
        c.check(c.all(p), i, "eager")


@pytest.mark.parametrize("name,T,kw", PLANS, ids=[p[0] for p in PLANS])
def test_what_a_graph_did_is_not_done_again(name, T, kw, dev):
    c = Calls(T, kw, dev)
    p = c.routed(c.routes[0])

    def launched(call):
        p.timing(16)
        call()
        names = [n for n, _, _ in p.timing_read()]
        p.timing(0)
        return names

    combine = lambda: p.combine(c.rows, c.w)  # noqa: E731
    graph, _ = captured(lambda: p.route(c.routes[0]).dispatch(c.x))
    graph.replay()
    for _ in range(2):       # the graph holds the route and the dispatch, which assigns
        assert launched(combine) == ["combine_kernel"]
    c.check(c.all(p, ("out",)), 0, "after the replay")
    p.route(c.routes[1])
    p.dispatch(c.x)
    for _ in range(2):
        assert launched(combine) == ["combine_kernel"]
    c.check(c.all(p, ("out",)), 1, "eager")


@pytest.mark.parametrize("band", [0, 256])
def test_captured_pipeline(band, dev):
    # A pipeline routes and finishes its plan in its own launch, recorded or not.
    T, H2 = 600, 64
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    x = torch.randn(T, H2, generator=g, device=dev).bfloat16()
    w = torch.randn(T, K, generator=g, device=dev)
    rows = torch.randn(T * K, H2, generator=g, device=dev).bfloat16()
    routes = [torch.topk(torch.randn(T, E, generator=g, device=dev), K, dim=1).indices.int().contiguous()
              for _ in range(2)]
    plan = lambda: cs.Plan(T, H2, E, K, 4, band_tokens=band)  # noqa: E731
    want = [plan().route(r).dispatch_backward(rows) for r in routes]
    ids = routes[0].clone()
    p = plan().route(ids)
    graph, (recv, out) = captured(lambda: p.pipeline(ids, x, w))
    for i in (0, 1, 0, 1):
        ids.copy_(routes[i])
        graph.replay()
        torch.cuda.synchronize()
        for _ in range(2):
            assert torch.equal(p.dispatch_backward(rows), want[i])
            assert np.array_equal(p.read("slot_of"), plan().route(routes[i]).read("slot_of"))

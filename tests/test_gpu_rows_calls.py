"""The calls of 8-bit rows as a program makes them: captured into graphs, on other streams, two at once, in a chain,
and with a wait that runs out."""
import pytest
import torch

from tests import rows_reference as ref

pytestmark = pytest.mark.gpu
E4 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_45_gb300 as sv

    return sv


def bits(t):
    return t.view(torch.uint8) if t.dtype.itemsize == 1 else t


class Layer:
    """A feed-forward layer between two points of a residual stream, and logits."""

    def __init__(self, sv, width=512, inner=1280, vocab=1003, seed=0):
        g = torch.Generator().manual_seed(seed)

        def weight(outs, ins):
            return sv.weight_quantise((torch.randn(outs, ins, generator=g) / ins ** 0.5).to(torch.bfloat16).cuda())

        self.sv, self.inner = sv, inner
        self.both, self.down, self.head = weight(2 * inner, width), weight(width, inner), weight(vocab, width)
        self.factors = [(1 + 0.1 * torch.randn(width, generator=g)).cuda() for _ in range(2)]

    def __call__(self, delta, stream, seen=None):
        sv, inner = self.sv, self.inner
        rows, stream = sv.rows_norm(delta, self.factors[0], residual=stream)
        both = sv.rows_product(rows, self.both)
        gated = sv.rows_gate(both[..., :inner], both[..., inner:])
        down = sv.rows_product(gated, self.down)
        last, end = sv.rows_norm(down, self.factors[1], residual=stream)
        logits = sv.rows_product(last, self.head, dtype=torch.float32)
        if seen is not None:
            seen.update(rows=rows, stream=stream, both=both, gated=gated, down=down, last=last, end=end)
        return logits


def inputs(batch, n, width=512, seed=1):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(batch, n, width, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]


@pytest.mark.parametrize("batch,n", [(1, 1), (7, 5), (60, 5)])
def test_a_layer(sv, batch, n):
    """Each step against its definition, from what the step before it gave; then the round's verification."""
    layer, seen = Layer(sv), {}
    delta, stream = inputs(batch, n)
    logits = layer(delta, stream, seen)
    flat = lambda t: t.cpu().reshape(-1, t.shape[-1])  # noqa: E731
    two = lambda c: sv.Coded(flat(c.codes), flat(c.scale))  # noqa: E731
    y, _ = ref.norm(flat(delta), flat(stream), layer.factors[0].cpu(), 1e-6)
    ref.check_coded(two(seen["rows"]), y, E4, 2.0 ** -18)
    assert torch.equal(flat(seen["stream"]), (flat(delta).float() + flat(stream).float()).to(torch.bfloat16))
    for rows, weight, got in (("rows", layer.both, seen["both"]), ("gated", layer.down, seen["down"]), ("last", layer.head, logits)):
        want, total = ref.product(two(seen[rows]), sv.Coded(weight.codes.cpu(), weight.scale.cpu()))
        width = weight.codes.shape[1]
        off = (flat(got).double() - want).abs()
        assert (off <= (width / 32 + 32) * 2.0 ** -23 * total + torch.finfo(got.dtype).eps / 2 * want.abs()).all()
    both = flat(seen["both"])
    y, z = ref.gate(both[:, :layer.inner], both[:, layer.inner:], "silu")
    ref.check_coded(two(seen["gated"]), y, E4, 2.0 ** -20 + z.abs() * 2.0 ** -22)
    y, _ = ref.norm(flat(seen["down"]), flat(seen["stream"]), layer.factors[1].cpu(), 1e-6)
    ref.check_coded(two(seen["last"]), y, E4, 2.0 ** -18)
    # greedy verification of the logits: drafts that follow them are accepted, up to the first that does not
    best = logits.argmax(-1).to(torch.int32)
    drafts = best[:, :-1].contiguous()
    if n > 1:
        drafts[:, n // 2] = (drafts[:, n // 2] + 1) % 1003
    zeros = torch.zeros(batch, device="cuda")
    tokens, accepted = sv.verify(logits, None, drafts, torch.full((batch,), n - 1, dtype=torch.int32, device="cuda"),
                                 torch.rand(batch, n, device="cuda"), zeros)
    assert (accepted == n // 2 if n > 1 else accepted == 0).all()
    assert torch.equal(tokens[:, :n // 2 + 1], best[:, :n // 2 + 1])


def test_a_layer_replays_from_graphs(sv):
    """Two captured layers, replayed in turn and on two streams at once, with other inputs: the bits of eager calls."""
    layers = [Layer(sv, seed=s) for s in (0, 1)]
    held, graphs, outs = [inputs(9, 5, seed=s) for s in (2, 3)], [], []
    for layer, x in zip(layers, held):
        layer(*x)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(layer(*x))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for seed in range(4, 10):
        new = [inputs(9, 5, seed=seed * 2 + i) for i in range(2)]
        for x, y in zip(held, new):
            for a, b in zip(x, y):
                a.copy_(b)
        for o in outs:
            o.fill_(-7)
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
                graph.replay()
        torch.cuda.synchronize()
        for layer, x, o in zip(layers, new, outs):
            assert torch.equal(layer(*x), o)


def test_other_streams(sv):
    """Calls given a stream, beside others on the current one; outputs belong to the stream that writes them."""
    layer = Layer(sv)
    a, w = sv.rows_quantise(torch.randn(300, 4096, device="cuda")), sv.weight_quantise(torch.randn(2000, 4096, device="cuda"))
    x, g = torch.randn(300, 4096, device="cuda"), torch.randn(4096, device="cuda")
    want = [sv.rows_product(a, w), *sv.rows_norm(x, g, x)[0], *sv.rows_gate(x, x), *sv.weight_quantise(x)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(30):
        layer(*inputs(20, 5))
        got = [sv.rows_product(a, w, stream=side), *sv.rows_norm(x, g, x, stream=side)[0], *sv.rows_gate(x, x, stream=side),
               *sv.weight_quantise(x, stream=side)]
        with torch.cuda.stream(side):
            same = [torch.equal(bits(p), bits(q)) for p, q in zip(got, want)]
        assert all(same)
    torch.cuda.synchronize()


def test_two_products_at_once(sv):
    """Products of every arrangement side by side on four streams: clusters of different sizes share the SMs."""
    g = torch.Generator().manual_seed(5)
    cases = []
    for rows, outs, dim in ((1, 4096, 4096), (160, 2560, 2560), (600, 20000, 512), (70, 8192, 1024)):
        a, w = ref.random_coded(rows, dim, E4, g, sv), ref.random_coded(outs, dim, E4, g, sv, 128)
        a, w = (sv.Coded(c.codes.cuda(), c.scale.cuda()) for c in (a, w))
        cases.append((a, w, sv.rows_product(a, w), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        got = [[sv.rows_product(a, w, stream=s) for _ in range(5)] for a, w, _, s in cases]
        torch.cuda.synchronize()
        for (_, _, want, _), several in zip(cases, got):
            assert all(torch.equal(x, want) for x in several)


def test_clusters_of_every_size_at_once(sv):
    """Two to sixteen CTAs to a cluster on five streams, behind and beside one another, as captured graphs too."""
    g = torch.Generator().manual_seed(10)
    cases = []
    for rows, outs, dim in ((1, 300, 14336), (33, 1025, 16400), (1, 4096, 4096), (160, 5000, 2048), (240, 1000, 8192)):
        a, w = ref.random_coded(rows, dim, E4, g, sv), ref.random_coded(outs, dim, E4, g, sv, 128)
        a, w = (sv.Coded(c.codes.cuda(), c.scale.cuda()) for c in (a, w))
        cases.append((a, w, sv.rows_product(a, w), torch.cuda.Stream()))
    torch.cuda.synchronize()
    graphs = []
    for a, w, _, s in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            kept = [sv.rows_product(a, w) for _ in range(4)]
        graphs.append((graph, kept))
    for i in range(20):
        got = [[sv.rows_product(a, w, stream=s) for _ in range(3)] for a, w, _, s in cases[i % 2:]]
        for (graph, kept), (_, _, _, s) in zip(graphs, cases):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for (_, _, want, _), several in zip(cases[i % 2:], got):
            assert all(torch.equal(x, want) for x in several)
        for (_, kept), (_, _, want, _) in zip(graphs, cases):
            assert all(torch.equal(x, want) for x in kept)
            for x in kept:
                x.fill_(7)


def test_a_chain_sees_what_the_call_before_it_wrote(sv):
    """Kernels may begin before the one ahead of them has ended: each still reads its results, and writes behind its reads."""
    g = torch.Generator().manual_seed(6)
    w = sv.weight_quantise(torch.randn(512, 512, generator=g).to(torch.bfloat16).cuda() / 512 ** 0.5)
    x0 = torch.randn(64, 512, generator=g).to(torch.bfloat16).cuda()

    def chain(buffers):
        x, coded, out = buffers
        x.copy_(x0)
        for _ in range(40):
            sv.rows_quantise(x, out=coded)
            sv.rows_product(coded, w, out=out)
            sv.rows_norm(out, residual=x, out=coded, out_sum=x)
        return x

    def buffers():
        coded = sv.Coded(torch.empty(64, 512, dtype=E4, device="cuda"), torch.empty(64, 4, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu))
        return torch.empty_like(x0), coded, torch.empty_like(x0)

    slow = x0.clone()
    for _ in range(40):
        coded = sv.rows_quantise(slow)
        torch.cuda.synchronize()
        out = sv.rows_product(coded, w)
        torch.cuda.synchronize()
        slow = sv.rows_norm(out, residual=slow)[1]
        torch.cuda.synchronize()
    assert slow.isfinite().all()
    for _ in range(5):
        assert torch.equal(chain(buffers()), slow)


@pytest.mark.parametrize("rows,outs,dim", [(1, 4096, 4096), (160, 2560, 2560), (5, 32000, 1024)])
def test_a_weight_written_by_the_call_before(sv, rows, outs, dim):
    """A product asks for its weight while the kernel ahead still writes it, and reads what that one wrote."""
    g = torch.Generator().manual_seed(9)
    sources = [torch.randn(outs, dim, generator=g).to(torch.bfloat16).cuda() for _ in range(3)]
    x = torch.randn(rows, dim, generator=g).to(torch.bfloat16).cuda()
    coded = sv.rows_quantise(x)
    want = [sv.rows_product(coded, sv.weight_quantise(s)) for s in sources]
    w = sv.weight_quantise(sources[0])
    torch.cuda.synchronize()
    got = []
    for i in range(30):
        sv.weight_quantise(sources[i % 3], out=w)
        got.append(sv.rows_product(coded, w))
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 3])


@pytest.fixture
def limit(sv):
    from speculative_decoding_verification_45_gb300 import _native

    lib = _native.load()

    def to(clocks):
        assert lib.spec_cache_set_wait_limit(clocks) == 0

    yield to
    to(2 ** 31 - 1)


@pytest.mark.parametrize("rows,outs,dim", [(1, 300, 144), (5, 4096, 4096), (160, 2560, 2560), (700, 5000, 1040), (300, 30000, 512)])
def test_a_wait_that_runs_out_is_reported(sv, limit, rows, outs, dim):
    """The call ends, its status says so, nothing outside of the output is written, and the next call is as ever."""
    g = torch.Generator().manual_seed(7)
    a, w = ref.random_coded(rows, dim, E4, g, sv), ref.random_coded(outs, dim, E4, g, sv, 128)
    a, w = (sv.Coded(c.codes.cuda(), c.scale.cuda()) for c in (a, w))
    want = sv.rows_product(a, w)
    kept = [bits(t).clone() for t in (*a, *w)]
    for clocks in (0, 100, 300, 1000, 3000, 10000, 30000, 2 ** 31 - 1):
        limit(clocks)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        whole = torch.full((rows * outs + 2048,), 7.0, dtype=torch.bfloat16, device="cuda")
        got = sv.rows_product(a, w, out=whole[1024:-1024].view(rows, outs), status=status)
        assert status.item() in (0, sv.STATUS_INTERNAL)
        if status.item() == 0:
            assert torch.equal(got, want)
        assert (whole[:1024] == 7).all() and (whole[-1024:] == 7).all()
        assert all(torch.equal(bits(t), k) for t, k in zip((*a, *w), kept))
        if clocks == 0:
            assert status.item() == sv.STATUS_INTERNAL
        if clocks == 2 ** 31 - 1:
            assert status.item() == 0


@pytest.mark.parametrize("rows,outs,dim", [(1, 300, 14336), (33, 1025, 16400), (200, 250, 12672)])
def test_a_wait_of_many_parts_that_runs_out(sv, limit, rows, outs, dim):
    test_a_wait_that_runs_out_is_reported(sv, limit, rows, outs, dim)


def test_captured_behind_other_work(sv):
    """In a graph, calls behind a memset, a copy, a torch kernel, another stream's work and one another."""
    g = torch.Generator().manual_seed(8)
    w = sv.weight_quantise(torch.randn(640, 512, generator=g).to(torch.bfloat16).cuda())
    src, held, extra = torch.randn(50, 512, generator=g).cuda(), torch.empty(50, 512, device="cuda"), torch.empty(50, 512, device="cuda")
    side = torch.cuda.Stream()

    def work():
        held.zero_()
        zero = sv.rows_quantise(held)
        held.copy_(src)
        first = sv.rows_quantise(held)
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            extra.copy_(src).mul_(2)
            other = sv.rows_product(sv.rows_quantise(extra), w)
        mine = sv.rows_product(first, w)
        main.wait_stream(side)
        joined, total = sv.rows_norm(mine, residual=other)
        held.fill_(3)
        return zero.codes.clone(), mine, other, joined.codes, joined.scale, total, sv.rows_product(sv.rows_quantise(held), w)

    want = work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for t in got:
        bits(t).fill_(7)
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(bits(a), bits(b))

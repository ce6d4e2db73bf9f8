"""The embedding lookup and its gradient by sorted tokens against elementary operations.

The lookup is one product and one rounding: equal bits.  A row's gradient adds runs of up to 16 tokens one after another
and joins the runs in order: at most 16 + count / 16 + 1 roundings of 2^-24 of the absolute sum; one rounding to BF16
(2^-8) or of the scaled sum (2^-23)."""
import pytest
import torch

from linear_recurrence_sequence_gb300 import api

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF = torch.bfloat16


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device=DEV).to(dtype)


def _tokens(gen, T, V, kind):
    if kind == "uniform":
        return torch.randint(0, V, (T,), generator=gen, device=DEV)
    if kind == "frequent":   # the k-th most common has a share of about 1 / k
        u = torch.rand(T, generator=gen, device=DEV, dtype=torch.float64)
        return (torch.exp(u * torch.log(torch.tensor(V + 1.0))).long().clamp(1, V) - 1)
    if kind == "one":
        return torch.full((T,), V - 1, device=DEV)
    if kind == "padding":
        return torch.full((T,), -5, device=DEV)
    t = torch.randint(-2, V, (T,), generator=gen, device=DEV)   # "mixed": a few of many, much padding
    return torch.where(torch.rand(T, generator=gen, device=DEV) < 0.5, t.clamp(max=3), t)


def _check_dw(dw, dy, tokens, V, scale, old=None):
    live = tokens >= 0
    t, d = tokens[live], dy.reshape(-1, dy.shape[-1])[live.view(-1)].double()
    z = torch.zeros(V, dy.shape[-1], dtype=torch.float64, device=DEV)
    want, terms = z.index_add(0, t, d) * scale, z.index_add(0, t, d.abs()) * abs(scale)
    count = torch.zeros(V, device=DEV).index_add(0, t, torch.ones_like(t, dtype=torch.float32)).double()[:, None]
    if old is not None:
        want, terms = want + old.double(), terms + old.double().abs()
    most = 2.0 ** -24 * (18 + count / 16) * terms
    most = most + (2.0 ** -8 if dw.dtype == BF else 2.0 ** -23) * want.abs() + 2.0 ** -134
    if old is None:
        assert float(dw[count[:, 0] == 0].abs().max() if bool((count == 0).any()) else 0) == 0
    else:
        assert torch.equal(dw[count[:, 0] == 0], old[count[:, 0] == 0])
    off = (dw.double() - want).abs() - most
    assert float(off.max()) <= 0, float(off.max())


@pytest.mark.parametrize("T,V,D", [(1, 1, 8), (1, 7, 64), (5, 3, 264), (64, 1000, 1024), (609, 50, 24), (1000, 32768, 136),
                                   (4097, 5003, 2056), (333, 20, 4096)])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("scale", [1.0, -3.7])
def test_lookup(T, V, D, dtype, scale):
    gen = _gen(T + V + D)
    w, tokens = _randn(gen, V, D, dtype=dtype), _tokens(gen, T, V, "mixed")
    y = api.embedding_forward(tokens, w, scale=scale)["y"]
    want = torch.where((tokens >= 0)[:, None], w[tokens.clamp(min=0)].float() * scale, 0.0).to(BF)
    assert torch.equal(y, want)


@pytest.mark.parametrize("T,V,D", [
    (1, 1, 8), (2, 9, 64), (31, 5, 264), (32, 40, 136), (33, 40, 64), (64, 1, 72), (609, 50, 24), (1000, 32768, 136),
    (4097, 5003, 2056), (333, 20, 4096), (9000, 129, 64), (20000, 700000, 8), (3000, 128, 2048)])
@pytest.mark.parametrize("kind", ["uniform", "frequent", "one", "padding", "mixed"])
def test_gradient(T, V, D, kind):
    gen = _gen(T + V + D)
    tokens, dy = _tokens(gen, T, V, kind), _randn(gen, T, D, dtype=BF)
    for fp32 in (False, True):
        g = api.embedding_backward(dy, tokens, V, scale=1.5, grad_fp32=fp32)
        assert g["dw"].dtype == (torch.float32 if fp32 else BF)
        _check_dw(g["dw"], dy, tokens, V, 1.5)
        assert api.device_status(g["scratch"]) == 0
        old = _randn(gen, V, D, dtype=g["dw"].dtype)
        dw = old.clone()
        o = api.embedding_backward(dy, tokens, V, scale=1.5, grad_fp32=fp32, accumulate=True, out={"dw": dw})
        assert o["dw"].data_ptr() == dw.data_ptr()
        _check_dw(dw, dy, tokens, V, 1.5, old)


@pytest.mark.parametrize("T,V", [(1, 3), (2, 3), (63, 40), (9000, 129), (9001, 129), (20001, 5000)])
@pytest.mark.parametrize("kind", ["uniform", "one", "mixed"])
def test_tokens_on_any_word(T, V, kind):
    gen = _gen(T)
    tokens = torch.cat([torch.full((1,), V, device=DEV), _tokens(gen, T, V, kind)])[1:]   # 8 bytes past a boundary of 16
    dy = _randn(gen, T, 72, dtype=BF)
    g = api.embedding_backward(dy, tokens, V, grad_fp32=True)
    _check_dw(g["dw"], dy, tokens, V, 1.0)
    assert api.device_status(g["scratch"]) == 0
    assert torch.equal(g["dw"], api.embedding_backward(dy, tokens.clone(), V, grad_fp32=True)["dw"])


def test_many_occurrences():
    """A token that fills thousands of runs; an owner with more tokens than shared memory holds."""
    gen = _gen(3)
    T, V, D = 100003, 256, 64
    tokens = _tokens(gen, T, V, "frequent")
    tokens[torch.rand(T, generator=gen, device=DEV) < 0.6] = 17
    dy = _randn(gen, T, D, dtype=BF)
    _check_dw(api.embedding_backward(dy, tokens, V, grad_fp32=True)["dw"], dy, tokens, V, 1.0)


@pytest.mark.parametrize("first", [0, 1, 15, 16, 40])
@pytest.mark.parametrize("D", [72, 1032])
def test_rows_of_many_runs(first, D):
    """Rows whose runs of 16 fill groups of 32, less and more than one, side by side in the sorted order."""
    gen = _gen(first)
    # (rows 128 apart lie next to each other)
    counts = [first, 500, 12, 512, 513, 528, 1, 1040, 16, 0, 1600, 511, 17, 16384]
    tokens = torch.cat([torch.full((n,), 128 * k, device=DEV) for k, n in enumerate(counts)])
    tokens = tokens[torch.randperm(tokens.numel(), generator=gen, device=DEV)]
    V, dy = 128 * len(counts), _randn(gen, tokens.numel(), D, dtype=BF)
    dw = api.embedding_backward(dy, tokens, V, grad_fp32=True)["dw"]
    _check_dw(dw, dy, tokens, V, 1.0)
    assert torch.equal(dw, api.embedding_backward(dy, tokens, V, grad_fp32=True)["dw"])


def test_tokens_without_a_row():
    gen = _gen(5)
    w, dy = _randn(gen, 50, 64, dtype=BF), _randn(gen, 40, 64, dtype=BF)
    tokens = _tokens(gen, 40, 50, "uniform")
    tokens[[3, 20]] = torch.tensor([50, 1 << 40], device=DEV)
    y = api.embedding_forward(tokens, w)["y"]
    good = tokens < 50
    assert bool(torch.isnan(y[~good]).all()) and torch.equal(y[good], w[tokens[good]])
    g = api.embedding_backward(dy, tokens, 50, grad_fp32=True)
    _check_dw(g["dw"], dy, torch.where(good, tokens, -1), 50, 1.0)
    assert api.device_status(g["scratch"]) == 1
    g = api.embedding_backward(dy, torch.where(good, tokens, -1), 50, scratch=g["scratch"])
    assert api.device_status(g["scratch"]) == 0


def test_padding_holds_anything():
    gen = _gen(6)
    dy = _randn(gen, 100, 64, dtype=BF)
    tokens = _tokens(gen, 100, 30, "uniform")
    tokens[::3] = -1
    dy[::3] = float("nan")
    g = api.embedding_backward(dy, tokens, 30, grad_fp32=True)["dw"]
    assert bool(torch.isfinite(g).all())
    _check_dw(g, torch.where((tokens >= 0)[:, None], dy, 0), tokens, 30, 1.0)


def test_shapes_streams_bits_and_graphs():
    gen = _gen(9)
    tokens = _tokens(gen, 6 * 500, 3001, "frequent").view(6, 500)
    w, dy = _randn(gen, 3001, 136, dtype=BF), _randn(gen, 6, 500, 136, dtype=BF)
    y, dw = api.embedding_forward(tokens, w)["y"], api.embedding_backward(dy, tokens, 3001)["dw"]
    assert y.shape == (6, 500, 136)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y2, dw2 = api.embedding_forward(tokens, w)["y"], api.embedding_backward(dy, tokens, 3001)["dw"]
    side.synchronize()
    assert torch.equal(y, y2) and torch.equal(dw, dw2)
    scratch = torch.empty(api.embedding_workspace_bytes(3000, 3001, 136), dtype=torch.uint8, device=DEV)
    out = {"y": torch.zeros_like(y), "dw": torch.zeros_like(dw)}

    def step():
        api.embedding_forward(tokens, w, out=out)
        api.embedding_backward(dy, tokens, 3001, out=out, scratch=scratch)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (10, 11):   # the replay takes what the buffers hold by then
        tokens.copy_(_tokens(_gen(seed), 3000, 3001, "mixed").view(6, 500))
        scratch.fill_(0xff)
        graph.replay()
        assert torch.equal(out["y"], api.embedding_forward(tokens, w)["y"])
        assert torch.equal(out["dw"], api.embedding_backward(dy, tokens, 3001)["dw"])


def test_more_than_2_31_values():
    T, V, D = 70000, 66000, 32768
    assert T * D > 1 << 31 and V * D > 1 << 31
    gen = _gen(12)
    w = torch.empty(V, D, dtype=BF, device=DEV).normal_(generator=gen)
    tokens = torch.randint(0, V, (T,), generator=gen, device=DEV)
    tokens[-3:] = torch.tensor([V - 1, 0, V - 1], device=DEV)
    y = api.embedding_forward(tokens, w)["y"]
    for t in (0, T // 2, T - 3, T - 2, T - 1):
        assert torch.equal(y[t], w[tokens[t]])
    dw = api.embedding_backward(y, tokens, V)["dw"]
    for v in (0, V // 2, V - 1):
        rows = torch.nonzero(tokens == v)[:, 0]
        want = y[rows].double().sum(0)
        most = 2.0 ** -8 * want.abs() + 2.0 ** -18 * y[rows].double().abs().sum(0) + 2.0 ** -134
        assert bool(((dw[v].double() - want).abs() <= most).all()), v

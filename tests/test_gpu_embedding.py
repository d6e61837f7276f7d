"""Embedding lookup and its gradient (CUDA, through the C ABI) against the fp64 oracle.

Tolerances.  The lookup is one fp32 product and one rounding to the output's type: compared bit for bit with the same two
roundings in NumPy / torch.  A gradient element is a sum of n fp32 terms, scaled once and added once to the buffer: at most
n + 2 roundings of 2^-24, each relative to no more than the sum of the terms' magnitudes (and the buffer's value)."""
import numpy as np
import pytest
import torch

from oracle import around_layers as A
from hstu_sequential_transducer_b200 import build
from hstu_sequential_transducer_b200 import hstu as H

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    H.lib()


def zipf(rng, T, V, bad=0.05):
    p = np.arange(1, V + 1) ** -1.1
    ids = rng.permutation(V)[rng.choice(V, size=T, p=p / p.sum())]
    out = rng.random(T) < bad
    ids[out] = rng.choice([-1, V, V + 5, -2 ** 31], size=int(out.sum()))
    return ids


def rows_of(rng, T, w, dtype, stride=None):
    """[T][w] on the GPU, rows `stride` elements apart."""
    t = torch.from_numpy(rng.standard_normal((T, stride or w)).astype(np.float32)).to(DEV, dtype)
    return t[:, :w]


def f64(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("table_t,out_t,low", [("f32", "f32", True), ("bf16", "f32", True), ("f32", "f32", False),
                                               ("f32", "bf16", False), ("bf16", "bf16", False)])
@pytest.mark.parametrize("T,dim,width,V,pad", [(1, 64, 64, 1, 0), (7, 50, 64, 3706, 0), (513, 33, 41, 97, 3), (100, 1, 1, 5, 0),
                                               (64, 512, 512, 1000, 8), (1000, 1024, 1024, 300, 0), (3, 2050, 2050, 9, 2), (90, 77, 333, 50, 2)])
def test_lookup(table_t, out_t, low, T, dim, width, V, pad):
    rng = np.random.default_rng(T * 7 + dim)
    ty = {"f32": torch.float32, "bf16": torch.bfloat16}
    table = rows_of(rng, V, dim, ty[table_t], dim + pad)
    ids = zipf(rng, T, V)
    scale = np.float32(np.sqrt(dim))
    for idt in (torch.int64, torch.int32):
        out = torch.full((T, width + pad), 7.0, dtype=ty[out_t], device=DEV)
        lo = torch.full((T, width + pad), 7.0, dtype=torch.bfloat16, device=DEV) if low else None
        H.embedding_fwd(table, torch.from_numpy(ids).to(DEV, idt), float(scale), out=out[:, :width],
                        low=lo[:, :width] if low else None)
        want = np.zeros((T, width), np.float32)
        ok = (ids >= 0) & (ids < V)
        want[ok, :dim] = f64(table).astype(np.float32)[ids[ok]] * scale
        assert np.array_equal(want, A.embedding_fwd(f64(table), ids, scale, width).astype(np.float32))
        want = torch.from_numpy(want)
        assert torch.equal(out[:, :width].cpu(), want.to(ty[out_t]))
        assert bool((out[:, width:] == 7).all())
        if low:
            assert torch.equal(lo[:, :width].cpu(), want.to(torch.bfloat16))
            assert bool((lo[:, width:] == 7).all())


def test_lookup_unaligned_rows():
    """Rows and bases on their element's alignment only."""
    rng = np.random.default_rng(4)
    table = torch.from_numpy(rng.standard_normal(1 + 9 * 17).astype(np.float32)).to(DEV)[1:].view(9, 17)[:, :16]
    ids = torch.tensor([8, 0, 3, 3], device=DEV)
    out = torch.empty(1 + 4 * 16, device=DEV)[1:].view(4, 16)
    H.embedding_fwd(table, ids, out=out)
    assert torch.equal(out, table[ids])


def check_grad(dout, ids, V, dim, scale, prior, got):
    want, mag, n = A.embedding_bwd(f64(dout), ids, V, dim, np.float32(scale))
    tol = (n[:, None] + 2) * U * (mag + np.abs(prior)) + 1e-300
    err = np.abs(got - (want + prior))
    assert np.all(err <= tol), float(np.max(err / tol))
    untouched = n == 0
    np.testing.assert_array_equal(got[untouched], prior[untouched])
    return want, mag, n


CASES = [(1, 64, 1), (31, 50, 10), (32, 8, 2), (33, 1, 1), (64, 128, 1), (1000, 50, 3706), (2049, 96, 300), (5000, 33, 70_000),
         (9000, 256, 17), (4096, 64, 16_777_217), (4097, 48, 513), (8200, 16, 1 << 28), (20_000, 512, 3), (32_768, 8, 4000), (32_769, 8, 4000), (600_001, 3, 777)]


@pytest.mark.parametrize("T,dim,V", [c for c in CASES if c[1] * c[2] <= 1 << 28])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_dense_gradient(T, dim, V, io):
    rng = np.random.default_rng(T + V)
    Vt = min(V, 100_000)             # the oracle's table; ids of a larger catalogue are kept below it
    ids = zipf(rng, T, Vt)
    ids[ids >= Vt] = V + 3           # padding above the catalogue
    dout = rows_of(rng, T, dim, torch.float32 if io == "f32" else torch.bfloat16, dim + (T % 3))
    prior = torch.from_numpy(rng.standard_normal((V, dim)).astype(np.float32)).to(DEV)
    g = prior.clone()
    H.embedding_bwd(dout, torch.from_numpy(ids).to(DEV), g, 1.5)
    p = f64(prior)
    check_grad(dout, np.where(ids > V, -1, ids), V, dim, 1.5, p, f64(g))
    # the same call on the same inputs gives the same bits
    g2 = prior.clone()
    H.embedding_bwd(dout, torch.from_numpy(ids.astype(np.int32)).to(DEV), g2, 1.5)
    assert torch.equal(g, g2)


@pytest.mark.parametrize("T,dim,V", CASES)
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_rows_gradient(T, dim, V, io):
    rng = np.random.default_rng(T + V + 1)
    ids = zipf(rng, T, min(V, 50_000))
    if V > 50_000:
        ok = (ids >= 0) & (ids < 50_000)
        ids[ok] = ids[ok] * (V // 50_000)            # ids over the whole catalogue
        ids[~ok] = -1
    dout = rows_of(rng, T, dim + 2, torch.float32 if io == "f32" else torch.bfloat16)
    cap = min(T, V)
    rows = torch.full((cap, dim + 1), 5.0, device=DEV)[:, :dim]
    row_ids = torch.full((cap,), -7, dtype=torch.int64, device=DEV)
    count = torch.full((1,), -7, dtype=torch.int64, device=DEV)
    H.embedding_bwd_rows(dout, torch.from_numpy(ids).to(DEV), V, row_ids, rows, count, scale=0.5)
    uniq, inv = np.unique(ids[(ids >= 0) & (ids < V)], return_inverse=True)
    n = len(uniq)
    assert int(count.item()) == n
    np.testing.assert_array_equal(row_ids.cpu().numpy()[:n], uniq)
    # entries past the count are as they were
    assert bool((row_ids[n:] == -7).all()) and bool((rows[n:] == 5).all())
    local = np.full(T, -1)
    local[(ids >= 0) & (ids < V)] = inv
    check_grad(dout, local, max(n, 1), dim, 0.5, np.zeros((max(n, 1), dim)), f64(rows)[:max(n, 1)] if n else np.zeros((1, dim)))


@pytest.mark.parametrize("kind", ["all_same", "all_padding", "one_real", "descending", "chunk_borders"])
def test_gradient_of_special_orders(kind):
    rng = np.random.default_rng(9)
    T, V, dim = 3000, 50, 20
    ids = {"all_same": np.full(T, 7), "all_padding": np.full(T, -1), "one_real": np.where(np.arange(T) == 1234, 3, -1),
           "descending": (T - 1 - np.arange(T)) * V // T, "chunk_borders": np.arange(T) // 64 % V}[kind].astype(np.int64)
    dout = rows_of(rng, T, dim, torch.float32)
    g = torch.zeros(V, dim, device=DEV)
    H.embedding_bwd(dout, torch.from_numpy(ids).to(DEV), g)
    check_grad(dout, ids, V, dim, 1.0, np.zeros((V, dim)), f64(g))
    rows, rid, cnt = torch.zeros(V, dim, device=DEV), torch.zeros(V, dtype=torch.int64, device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV)
    H.embedding_bwd_rows(dout, torch.from_numpy(ids).to(DEV), V, rid, rows, cnt)
    n = int(cnt.item())
    np.testing.assert_array_equal(rid.cpu().numpy()[:n], np.unique(ids[ids >= 0]))
    assert torch.equal(rows[:n], g[rid[:n]])


def test_non_finite_rows_stay_with_their_item():
    """A NaN or infinity in one event's row reaches that event's item alone; one in a padding event's row reaches none."""
    ids = torch.tensor([3, 1, -1, 3, 0], device=DEV)
    dout = torch.ones(5, 8, device=DEV)
    dout[0, 2], dout[2, 5], dout[4, 1] = float("nan"), float("nan"), float("inf")
    g = torch.zeros(4, 8, device=DEV)
    H.embedding_bwd(dout, ids, g)
    want = torch.tensor([1.0, 1, 0, 2], device=DEV)[:, None].repeat(1, 8)
    want[3, 2], want[0, 1] = float("nan"), float("inf")
    assert torch.equal(torch.nan_to_num(g, nan=-1.0, posinf=-2.0), torch.nan_to_num(want, nan=-1.0, posinf=-2.0))


def test_empty():
    ids = torch.empty(0, dtype=torch.int64, device=DEV)
    out = H.embedding_fwd(torch.ones(3, 4, device=DEV), ids)
    assert out.shape == (0, 4)
    g = torch.ones(3, 4, device=DEV)
    H.embedding_bwd(torch.empty(0, 4, device=DEV), ids, g)
    assert bool((g == 1).all())
    cnt = torch.full((1,), 9, dtype=torch.int64, device=DEV)
    H.embedding_bwd_rows(torch.empty(0, 4, device=DEV), ids, 3, ids, torch.empty(0, 4, device=DEV), cnt)
    assert int(cnt.item()) == 0


def test_offsets_past_32_bits():
    """A table and a gradient of more than 2^32 elements: the last rows are found."""
    V, dim = (1 << 32) // 1024 + 5, 1024
    table = torch.zeros(V, dim, dtype=torch.bfloat16, device=DEV)
    table[V - 1] = 3.0
    ids = torch.tensor([V - 1, 0, V - 1, V], device=DEV)
    out = H.embedding_fwd(table, ids)
    assert bool((out[[0, 2]] == 3).all()) and bool((out[[1, 3]] == 0).all())
    del table
    g = torch.zeros(V, dim, device=DEV)
    H.embedding_bwd(torch.ones(4, dim, device=DEV), ids, g)
    assert bool((g[V - 1] == 2).all()) and bool((g[0] == 1).all()) and float(g[1:V - 1].abs().max()) == 0


def test_results_made_on_another_stream():
    """A result that the call makes itself comes from the pool of the stream that writes it: memory that work still queued on
    the current stream reads is not handed out for it."""
    side = torch.cuda.Stream()
    table, ids = torch.randn(50, 256, device=DEV), torch.arange(50, device=DEV).repeat(2000)
    want = table[ids]
    torch.cuda.synchronize()
    sums = []
    for _ in range(20):
        old = torch.ones(100_000, 256, device=DEV)
        for _ in range(4):
            old = old * 1.0
        sums.append(old.sum())
        del old
        out = H.embedding_fwd(table, ids, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert all(float(t) == 25_600_000 for t in sums)


@pytest.mark.parametrize("T", [20, 700, 9000, 40_000])
def test_other_stream_and_graph(T):
    """On a side stream, and captured: a replay reads the buffers' new contents; two graphs share no workspace.  One size for
    each form of the sort, and one chunk."""
    rng = np.random.default_rng(2)
    V, dim = 90, 40
    side = torch.cuda.Stream()
    bufs = []
    for seed in (0, 1):
        ids = torch.from_numpy(zipf(rng, T, V)).to(DEV)
        bufs.append((rows_of(rng, T, dim, torch.float32).contiguous(), ids, torch.zeros(V, dim, device=DEV)))
    torch.cuda.synchronize()
    for d, i, g in bufs:
        H.embedding_bwd(d, i, g, stream=side)
    side.synchronize()
    want = [g.clone() for _, _, g in bufs]
    graphs = []
    for d, i, g in bufs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            g.zero_()
            H.embedding_bwd(d, i, g)
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for (d, i, g), w in zip(bufs, want):
        assert torch.equal(g, w)
    bufs[0][0].copy_(bufs[1][0])
    bufs[0][1].copy_(bufs[1][1])
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(bufs[0][2], want[1])


@pytest.mark.parametrize("V", [300, 300_000, 20_000_000, (1 << 28) + 9, (1 << 31) - 1])
@pytest.mark.parametrize("T", [40_001, 400_001])
def test_rows_gradient_of_every_pass_count(T, V):
    """The sort by launches, its tiles' counts added up by each tile or scanned (up to 96 tiles, above): one to four digits, ids over
    the whole catalogue, many of them neighbours of the borders of a digit; the same bits from a second call."""
    rng = np.random.default_rng(V)
    ids = rng.integers(0, V, size=T)
    near = rng.integers(0, 4, size=T) * (V // 4) + rng.integers(-3, 4, size=T)
    some = rng.random(T) < 0.3
    ids[some] = near[some]                                   # popular items, among them -1 .. -3 and V .. V + 2 as padding
    dim = 3
    dout = rows_of(rng, T, dim, torch.float32)
    cap = min(T, V)
    new = lambda: (torch.full((cap,), -7, dtype=torch.int64, device=DEV), torch.full((cap, dim), 5.0, device=DEV),
                   torch.full((1,), -7, dtype=torch.int64, device=DEV))
    dev_ids = torch.from_numpy(ids).to(DEV)
    row_ids, rows, count = H.embedding_bwd_rows(dout, dev_ids, V, *new())
    real = (ids >= 0) & (ids < V)
    uniq, inv = np.unique(ids[real], return_inverse=True)
    n = len(uniq)
    assert int(count.item()) == n
    np.testing.assert_array_equal(row_ids.cpu().numpy()[:n], uniq)
    assert bool((row_ids[n:] == -7).all()) and bool((rows[n:] == 5).all())
    local = np.full(T, -1)
    local[real] = inv
    check_grad(dout, local, n, dim, 1.0, np.zeros((n, dim)), f64(rows)[:n])
    again = H.embedding_bwd_rows(dout, dev_ids, V, *new())
    assert torch.equal(again[0], row_ids) and torch.equal(again[1], rows) and int(again[2]) == n


@pytest.mark.parametrize("T", [40_001, 400_001])
def test_dense_gradient_of_three_digits(T):
    rng = np.random.default_rng(T)
    V, dim = 300_000, 3
    ids = rng.integers(-5, V + 5, size=T)
    dout = rows_of(rng, T, dim, torch.bfloat16)
    prior = torch.from_numpy(rng.standard_normal((V, dim)).astype(np.float32)).to(DEV)
    g = H.embedding_bwd(dout, torch.from_numpy(ids).to(DEV), prior.clone(), 1.5)
    check_grad(dout, ids, V, dim, 1.5, f64(prior), f64(g))
    assert torch.equal(g, H.embedding_bwd(dout, torch.from_numpy(ids).to(DEV), prior.clone(), 1.5))

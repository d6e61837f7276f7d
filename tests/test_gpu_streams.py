"""Training steps on several streams at once, and captured beside eager ones: each call's scratch is its own.

Two runs of a step on the same inputs differ only by the order in which the backward's atomic sums arrive, a few roundings
u of the sums' terms (2^-24 each for fp32 sums, 2^-8 where a bf16 operand in between flips): normwise within 1e-4 (f32) and
1e-2 (bf16) of one another.  Forward outputs are equal bit for bit."""
import pytest
import torch

from hstu_sequential_transducer_b200 import build
from hstu_sequential_transducer_b200 import hstu as H
from hstu_sequential_transducer_b200 import stack as S
from hstu_sequential_transducer_b200 import workloads as W

pytestmark = pytest.mark.gpu
TOL = {"f32": 1e-4, "bf16": 1e-2}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    H.lib()


def batch(dtype, lengths, seed, layers=3):
    return S.DeviceWorkload.from_workload(W.custom(lengths, d=128, H=2, dtype=dtype, N=400.0, with_bias=True, with_affine=True,
                                                   backward=True, layers=layers, mean_gap=900.0, seed=seed))


def make(kind, dw):
    if kind == "train":
        return S.TrainStep(dw)
    return S.NormedTrainStep(dw, [H.BlockNorm() for _ in range(len(dw.layers) + 1)])


def parts(kind, step, dx):
    grads = [t for g in step.grads for t in vars(g).values() if t is not None]
    return [step.y.clone()] + [t.clone() for t in (dx, *grads)]


def same(got, want, dtype):
    assert torch.equal(got[0], want[0])
    for a, b in zip(got[1:], want[1:]):
        a, b = a.double(), b.double()
        assert float((a - b).norm()) <= TOL[dtype] * float(b.norm())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["train", "normed"])
def test_two_streams(kind, dtype):
    dws = [batch(dtype, [300, 17, 0, 250, 399], 1), batch(dtype, [128, 399, 64, 1], 2)]
    steps = [make(kind, dw) for dw in dws]
    want = []
    for s in steps:
        s.zero_grads()
        want.append(parts(kind, s, s.run()))
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(4):
        for s in steps:
            s.zero_grads()
        torch.cuda.synchronize()
        dx = [s.run(stream=st) for s, st in zip(steps, streams)]
        torch.cuda.synchronize()
        for s, d, w in zip(steps, dx, want):
            same(parts(kind, s, d), w, dtype)


@pytest.mark.parametrize("kind", ["train", "normed"])
def test_captured_step_after_a_larger_eager_one(kind):
    """A graph keeps its own scratch: a later eager step that needs more lets none of it go."""
    small, large = make(kind, batch("bf16", [60, 33], 3)), make(kind, batch("bf16", [399] * 12, 4))

    def one(step):
        step.zero_grads()
        return step.run()

    want = parts(kind, small, one(small))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dx = one(small)
    big = parts(kind, large, one(large))
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    fresh = torch.full((64 << 20,), 7.0, device="cuda")              # what the allocator hands out next
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    same(parts(kind, small, dx), want, "bf16")
    assert bool((fresh == 7.0).all())
    same(parts(kind, large, one(large)), big, "bf16")


def test_forward_and_scoring_on_a_side_stream():
    """The whole of a forward stack and of cached scoring runs on the given stream while the current one is busy: rows are
    selected, and buffers in between come and go, on it."""
    w = W.custom([170] * 3, d=128, H=2, dtype="bf16", N=400.0, layers=3, mean_gap=900.0, seed=5, num_targets=[70] * 3)
    dw = S.DeviceWorkload.from_workload(w)
    want = [S.forward_stack(dw), *S.mfalcon_score(dw, 100, 70, 32)]
    side, busy = torch.cuda.Stream(), torch.ones(64 << 20, device="cuda")
    torch.cuda.synchronize()
    for _ in range(3):
        for _ in range(20):
            busy.mul_(1.0)
        got = [S.forward_stack(dw, stream=side), *S.mfalcon_score(dw, 100, 70, 32, stream=side)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert H.validate_inputs(dw.offsets, dw.timestamps, dw.num_targets, 400, stream=side) == 0


def test_gradient_on_a_side_stream_behind_a_busy_current_one():
    """The dense gradient's first use and its clearing, on a side stream while the current one has work queued: no fill comes
    after a gradient.  Sums of one 1.0 for each event are exact."""
    side, busy = torch.cuda.Stream(), torch.ones(64 << 20, device="cuda")
    ids, dx, table = torch.arange(600, device="cuda").repeat(3), torch.ones(1800, 64, device="cuda"), torch.zeros(1000, 64, device="cuda")
    want = torch.zeros(1000, 64, device="cuda")
    want[:600] = 3.0
    torch.cuda.synchronize()
    for _ in range(50):
        busy.mul_(1.0)
    emb = S.ItemEmbedding(table, scale=1.0)
    emb.backward(dx, ids, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(emb.grad, want)
    for _ in range(50):
        busy.mul_(1.0)
    emb.zero_grad(stream=side)
    emb.backward(dx, ids, stream=side)
    side.synchronize()
    assert torch.equal(emb.grad, want)


@pytest.mark.parametrize("kind", ["train", "normed"])
def test_first_run_on_a_side_stream_behind_a_busy_current_one(kind):
    dw = batch("bf16", [60, 33], 3)
    serial = make(kind, dw)
    want = parts(kind, serial, serial.run())
    side, busy = torch.cuda.Stream(), torch.ones(64 << 20, device="cuda")
    torch.cuda.synchronize()
    for again in (False, True):
        for _ in range(50):
            busy.mul_(1.0)
        if again:
            step.zero_grads(stream=side)
        else:
            step = make(kind, dw)
        dx = step.run(stream=side)
        torch.cuda.synchronize()
        same(parts(kind, step, dx), want, "bf16")


def rows_of(emb):
    n = int(emb.count)
    return emb.row_ids[:n].clone(), emb.rows[:n].clone()


def test_rows_gradient_after_a_change_of_stream_and_size():
    """Buffers made on one stream, written on another that is behind, and replaced by larger ones: their memory goes to nobody
    while they are written.  Sums of ones are exact."""
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    busy = torch.ones(64 << 20, device="cuda")
    emb = S.ItemEmbedding(torch.zeros(5000, 64, device="cuda"), scale=1.0, rows=True)
    small, large = torch.arange(2000, device="cuda"), torch.arange(4000, device="cuda").repeat(2)
    one = torch.ones(8000, 64, device="cuda")
    torch.cuda.synchronize()
    emb.backward(one[:2000], small, stream=a)
    a.synchronize()
    with torch.cuda.stream(b):
        for _ in range(50):
            busy.mul_(1.0)
    emb.backward(one[:2000], small, stream=b)
    emb.backward(one, large, stream=b)
    with torch.cuda.stream(a):
        fresh = [torch.full((2000, 64), 7.0, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert all(bool((f == 7.0).all()) for f in fresh)
    ids, rows = rows_of(emb)
    assert torch.equal(ids, torch.arange(4000, device="cuda")) and bool((rows == 2.0).all())


def test_captured_rows_gradient_after_a_larger_batch():
    """A captured gradient's buffers stay when a later batch needs larger ones."""
    emb = S.ItemEmbedding(torch.zeros(5000, 64, device="cuda"), scale=1.0, rows=True)
    small, large = torch.arange(2000, device="cuda"), torch.arange(4000, device="cuda").repeat(2)
    one = torch.ones(8000, 64, device="cuda")
    emb.backward(one[:2000], small)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        emb.backward(one[:2000], small)
    at, where = emb.rows.data_ptr(), emb.rows.shape
    emb.backward(one, large)
    assert emb.rows.data_ptr() != at
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    fresh = [torch.full(where, 7.0, device="cuda") for _ in range(4)]
    graph.replay()
    torch.cuda.synchronize()
    assert all(bool((f == 7.0).all()) and f.data_ptr() != at for f in fresh)
    ids, rows = rows_of(emb)
    assert ids.numel() == 4000 and bool((rows == 2.0).all())


def test_sampled_batch_of_a_run_on_another_stream():
    """batch() right after a run on a stream that is behind: it waits for that run, whatever stream is the current one."""
    w = W.custom([170] * 3, d=128, H=2, dtype="bf16", N=400.0, layers=1, mean_gap=900.0, seed=5)
    dw = S.DeviceWorkload.from_workload(w)
    sl = S.StochasticLength(dw, 1.2)
    assert sl.sub_len < 170
    none, all_ = torch.full((3,), -1, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    keys = torch.arange(dw.T, dtype=torch.int32, device="cuda")
    want = []
    for draw in (none, all_):
        sl.run(draw, keys)
        b = sl.batch()
        want.append((b.T, b.x.clone(), b.timestamps.clone()))
    assert want[0][0] != want[1][0]
    side, busy = torch.cuda.Stream(), torch.ones(64 << 20, device="cuda")
    torch.cuda.synchronize()
    for draw, (t, x, ts) in list(zip((none, all_), want)) * 2:
        with torch.cuda.stream(side):
            for _ in range(50):
                busy.mul_(1.0)
        sl.run(draw, keys, stream=side)
        b = sl.batch()
        assert b.T == t and torch.equal(b.x, x) and torch.equal(b.timestamps, ts)

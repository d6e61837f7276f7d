"""Which buffers the Python calls make, and where (CPU only): the library's launches are replaced by a recorder, its host-side
size queries are its own."""
import ctypes
import types

import pytest
import torch

from hstu_sequential_transducer_b200 import build
from hstu_sequential_transducer_b200 import hstu as H
from hstu_sequential_transducer_b200 import stack as S
from hstu_sequential_transducer_b200 import workloads as W


class Recorder:
    """The library with its launches recorded: (name, arguments) of each."""

    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name.endswith(("_size", "_layout", "_string")):
            return getattr(self.real, name)
        return lambda *args: self.calls.append((name, args)) or 0


@pytest.fixture
def lib(monkeypatch):
    build.build()
    rec = Recorder(H.lib())
    monkeypatch.setattr(H, "lib", lambda: rec)
    monkeypatch.setattr(H, "stream_ptr", lambda s=None: None if s is None else s.cuda_stream)
    return rec


@pytest.fixture
def made(monkeypatch):
    """Every buffer that a call makes: (tensor, stream)."""
    out = []
    real = torch.empty

    def empty(shape, dtype, device, stream):
        out.append((real(shape, dtype=dtype, device=device), stream))
        return out[-1][0]
    monkeypatch.setattr(H, "_empty", empty)
    return out


def layer(T=40, d=64):
    cfg = H.make_config(d, 2, 64.0)
    z = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t)
    low = lambda *s: z(*s, t=torch.bfloat16)
    w = H.LayerWeights(W1=low(d, 4 * d), W2=low(d, d))
    off, ts = torch.tensor([0, T // 2, T]), z(T, t=torch.int64)
    saved = z(H.saved_layout(cfg, T)[-1], t=torch.uint8)
    return {"fwd": lambda s: H.fwd(cfg, w, z(T, d), off, ts, y=z(T, d), stream=s),
            "bwd": lambda s: H.bwd(cfg, w, z(T, d), z(T, d), saved, off, ts, dx=z(T, d), stream=s),
            "fwd_cached": lambda s: H.fwd_cached(cfg, w, z(T, d), off, ts, low(T, 2 * d), off, ts, y=z(T, d), stream=s),
            "attention_fwd": lambda s: H.attention_fwd(cfg, None, None, low(T, 4 * d), off, ts, None, z(T, d), stream=s),
            "softmax_attention_fwd": lambda s: H.softmax_attention_fwd(cfg, None, None, low(T, 4 * d), off, ts, None, z(T, d), stream=s),
            "attention_fwd_cached": lambda s: H.attention_fwd_cached(cfg, None, None, low(T, 4 * d), off, ts, low(T, 2 * d), off, ts,
                                                                     z(T, d), stream=s),
            "attention_bwd": lambda s: H.attention_bwd(cfg, None, None, low(T, 4 * d), low(T, 4 * d), z(T, d), off, ts, None,
                                                       low(T, 4 * d), stream=s)}


@pytest.mark.parametrize("call", sorted(layer()))
def test_scratch_belongs_to_one_call_on_its_stream(lib, made, call):
    """Two calls on two streams run side by side, so each has scratch of its own, from its own stream's pool; nothing that an
    earlier call (or a graph captured from it) uses is kept for a later one or let go by it."""
    a, b = types.SimpleNamespace(cuda_stream=11), types.SimpleNamespace(cuda_stream=22)
    f = layer()[call]
    for stream in (a, b, None):
        f(stream)
    assert [s for _, s in made] == [a, b, None]
    used = [[x for x in args if isinstance(x, int)] for _, args in lib.calls]
    for (t, s), ints in zip(made, used):
        assert t.data_ptr() in ints and t.numel() in ints
        assert s is None or s.cuda_stream in ints
    assert len({t.data_ptr() for t, _ in made}) == 3


def test_results_come_from_the_stream_that_writes_them(lib, made):
    """What a call makes for its caller when given no buffer: on the call's stream, like its scratch."""
    T, d = 40, 64
    cfg = H.make_config(d, 2, 64.0)
    z = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t)
    w = H.LayerWeights(W1=z(d, 4 * d, t=torch.bfloat16), W2=z(d, d, t=torch.bfloat16))
    off, ts = torch.tensor([0, 20, T]), z(T, t=torch.int64)
    side = types.SimpleNamespace(cuda_stream=11)
    saved = z(H.saved_layout(cfg, T)[-1], t=torch.uint8)
    out = [H.fwd(cfg, w, z(T, d), off, ts, stream=side),
           H.fwd_cached(cfg, w, z(T, d), off, ts, z(T, 2 * d, t=torch.bfloat16), off, ts, stream=side),
           H.bwd(cfg, w, z(T, d), z(T, d), saved, off, ts, stream=side),
           *H.stochastic_length(off, None, 5, z(2), z(T), stream=side)]
    assert all(s is side for _, s in made)
    for t in out:
        assert any(t is m for m, _ in made)
    assert [tuple(t.shape) for t in out] == [(T, d)] * 3 + [(3,), (T,)]


def test_gradients_are_cleared_on_the_given_stream(monkeypatch):
    """zero_grad(s) before a run on a side stream: the fill is queued there, in front of the run."""
    build.build()
    w = W.custom([9, 4], d=64, H=2, dtype="bf16", N=16.0, backward=True, layers=2)
    dw = S.DeviceWorkload.from_workload(w, device="cpu")
    emb, train = S.ItemEmbedding(torch.zeros(5, 64)), S.TrainStep(dw)
    normed = S.NormedTrainStep(dw, [H.BlockNorm() for _ in range(3)])
    current, fills = [None], []

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            current.append(self.stream)

        def __exit__(self, *_):
            current.pop()
    monkeypatch.setattr(torch.cuda, "stream", On)
    real = torch.Tensor.zero_
    monkeypatch.setattr(torch.Tensor, "zero_", lambda t: (fills.append(current[-1]), real(t))[1])
    for clear, filled in ((emb.zero_grad, [emb.grad]), (train.zero_grads, [train.flat_grads]),
                          (normed.zero_grads, [t for g in normed.grads for t in vars(g).values() if t is not None])):
        for t in filled:
            t.fill_(3.0)
        fills.clear()
        clear(stream="side")
        assert set(fills) == {"side"} and all(not bool(t.any()) for t in filled)
        clear()


def test_rows_gradient_buffers_grow_and_are_not_cleared(monkeypatch):
    """Batches of changing size share the buffers of the largest so far; what the gradient does not write is not touched."""
    wrote = []

    def rows_gradient(dx, ids, V, row_ids, rows, count, scale, stream=None):
        assert row_ids.shape == (min(ids.shape[0], V),) and rows.shape == (row_ids.shape[0], 8) and rows.is_contiguous()
        wrote.append((row_ids.data_ptr(), rows.data_ptr(), count.data_ptr()))
        count.fill_(1)
        row_ids[:1] = 7
        rows[:1] = 2.0
    monkeypatch.setattr(H, "embedding_bwd_rows", rows_gradient)
    emb = S.ItemEmbedding(torch.zeros(90, 8), rows=True)
    run = lambda T: emb.backward(torch.zeros(T, 8), torch.zeros(T, dtype=torch.int64))
    run(50)
    emb.rows.fill_(9.0)
    emb.row_ids.fill_(3)
    for T in (20, 50, 1, 49):
        run(T)
        assert emb.rows.shape == (T, 8) and bool((emb.rows[1:] == 9).all()) and bool((emb.row_ids[1:] == 3).all())
    assert len(set(wrote)) == 1
    run(70)
    assert emb.rows.shape == (70, 8) and len(set(wrote)) == 2
    run(500)                             # no more rows than items
    assert emb.rows.shape == (90, 8)
    run(0)
    assert emb.rows.shape == (0, 8)


def test_normed_steps_refuse_missing_gates_and_a_missing_gradient(lib):
    """A gate (or None) for each layer, no fewer and no more; a run without an upstream gradient would give zeros for all."""
    w = W.custom([9, 4], d=64, H=2, dtype="bf16", N=16.0, layers=2)
    dw = S.DeviceWorkload.from_workload(w, device="cpu")
    joints, gate = [H.BlockNorm() for _ in range(3)], torch.zeros(dw.T, 64, dtype=torch.bfloat16)
    for gates in ([gate], [gate] * 3, []):
        with pytest.raises(ValueError, match="gate"):
            S.NormedTrainStep(dw, joints, gates)
    step = S.NormedTrainStep(dw, joints, [gate, None])
    assert dw.dy is None
    with pytest.raises(ValueError, match="dy"):
        step.run()
    assert not lib.calls


def test_layer_gradients_are_handed_over_on_the_stream_of_the_run(lib, monkeypatch):
    """on_layer_grads starts collectives, which are ordered after the current stream: that of the run."""
    w = W.custom([9, 4], d=64, H=2, dtype="bf16", N=16.0, backward=True, layers=3)
    step = S.TrainStep(S.DeviceWorkload.from_workload(w, device="cpu"))
    side, current = types.SimpleNamespace(cuda_stream=11), [None]

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            current.append(self.stream)

        def __exit__(self, *_):
            current.pop()
    monkeypatch.setattr(torch.cuda, "stream", On)
    seen = []
    for stream in (side, None):
        step.run(stream=stream, on_layer_grads=lambda i: seen.append((i, current[-1])))
    assert seen == [(i, s) for s in (side, None) for i in (2, 1, 0)]

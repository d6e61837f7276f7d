"""The operators around the layers as a training run uses them: an embedding that feeds a stack and takes its gradient, 8-bit
checkpoints between the forward and the backward, stacks with norms between their blocks; against the fp64 oracles.

Tolerances are those of the layers' parity tests (test_gpu_parity.py): outputs and dX within 1e-4 (fp32) or 2e-2 (bf16) of the
oracle's rms; gradients normwise within half of that (all of it in stacks) and entry-wise within three times rms + |value|.  The
8-bit checkpoints are part of the definition: the oracle's backward starts from the activations as they are restored."""
import numpy as np
import pytest
import torch

from oracle import around_layers as A
from oracle import hstu_ref as R
from hstu_sequential_transducer_b200 import build
from hstu_sequential_transducer_b200 import hstu as H
from hstu_sequential_transducer_b200 import stack as S
from hstu_sequential_transducer_b200 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = {"f32": 1e-4, "bf16": 2e-2}
LAYER_GRADS = ("dW1", "dW2", "db1", "db2", "dgamma", "dbeta", "drab_pos", "drab_time")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    H.lib()


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def lp(p):
    return R.LayerParams(p.W1, p.W2, p.rab_pos, p.rab_time, p.b1, p.b2, p.gamma, p.beta)


def lcfg(w):
    return R.LayerConfig(w.num_heads, w.norm_N, w.num_pos_buckets, w.num_time_buckets, w.ln_eps)


def check(got, ref, tol, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    rms = np.sqrt(np.mean(ref ** 2))
    e = np.max(np.abs(got - ref)) / rms
    assert e <= tol, (what, e)


def check_grad(got, ref, tol, what):
    got = f64(got)
    assert np.linalg.norm(got - ref) <= tol * np.linalg.norm(ref), (what, np.linalg.norm(got - ref) / np.linalg.norm(ref))
    rms = np.sqrt(np.mean(ref ** 2))
    assert np.max(np.abs(got - ref) / (rms + np.abs(ref))) <= 3 * tol, what


def small(dtype, layers=2, lengths=(70, 1, 0, 130, 33), d=128):
    return W.custom(list(lengths), d=d, H=2, dtype=dtype, N=120.0, num_targets=[5, 0, 0, 20, 33][:len(lengths)], with_bias=True,
                    with_affine=True, backward=True, layers=layers, mean_gap=900.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [False, True])
def test_embedding_feeds_a_training_step(dtype, rows):
    w = small(dtype)
    rng = np.random.default_rng(5)
    V, dim = 40, 100                                    # rows of 128 with 28 zero columns
    table = W.round_to_bf16(rng.normal(0, 0.1, (V, dim)).astype(np.float32))
    ids = rng.integers(-1, V, size=w.T).astype(np.int64)
    dw = S.DeviceWorkload.from_workload(w)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    emb = S.ItemEmbedding(torch.from_numpy(table).to(DEV, dt), scale=8.0, rows=rows)
    step = S.TrainStep(dw, embedding=emb, ids=torch.from_numpy(ids).to(DEV))
    step.zero_grads()
    emb.zero_grad()
    dx = step.run()
    x = A.embedding_fwd(table, ids, 8.0, w.d_model)
    y, rdx, rgr = R.stack_forward_backward(x, w.seq_offsets, w.timestamps, w.num_targets, [lp(p) for p in w.params], lcfg(w), w.dy)
    check(step.y, y, TOL[dtype], "Y")
    check(dx, rdx, TOL[dtype], "dX")
    want = A.embedding_bwd(rdx, ids, V, dim, 8.0)[0]
    if rows:
        n = int(emb.count.item())
        got = np.zeros((V, dim))
        got[emb.row_ids.cpu().numpy()[:n]] = f64(emb.rows)[:n]
    else:
        got = f64(emb.grad)
    check_grad(torch.from_numpy(got), want, TOL[dtype], "table")
    for i in range(2):
        for n in LAYER_GRADS:
            check_grad(getattr(step.grads[i], n), getattr(rgr[i], n), TOL[dtype], n)


def backward_of(w, cfg, v, x, params, dy):
    """The layer's backward in fp64 from a saved block's values v and x, with the block's own row statistics."""
    d = w.d_model
    u, pre = v["g"][:, :d], v["pre"]
    gr = {"dW2": v["z"].T @ dy, "db2": dy.sum(0)}
    dz = dy @ params.W2.T
    m, r = v["mean"][:, None], v["rstd"][:, None]
    oh = (v["o"] - m) * r
    gm = params.gamma if params.gamma is not None else np.ones(d)
    dln = dz * u
    gr["dgamma"], gr["dbeta"] = (dln * oh).sum(0), dln.sum(0)
    q = dln * gm
    do = r * (q - q.mean(1, keepdims=True) - oh * (q * oh).mean(1, keepdims=True))
    dg, gr["drab_pos"], gr["drab_time"] = R.attention_backward(v["g"], do, w.seq_offsets, w.timestamps, w.num_targets,
                                                               params.rab_pos, params.rab_time, cfg)
    dg[:, :d] = dz * (oh * gm + (params.beta if params.beta is not None else 0.0))
    dpre = dg * R.silu_grad(pre)
    gr["dW1"], gr["db1"] = x.T @ dpre, dpre.sum(0)
    return dpre @ params.W1.T + dy, gr


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype,io", [("f32", H.HSTU_F32), ("bf16", H.HSTU_F32), ("bf16", H.HSTU_BF16)])
def test_training_step_from_checkpoints(fmt, dtype, io):
    w = small(dtype, layers=3)
    dw = S.DeviceWorkload.from_workload(w, io_dtype=io)
    plain = S.TrainStep(dw)
    plain.zero_grads()
    plain.run()
    step = S.TrainStep(dw, checkpoints=fmt)
    for _ in range(2):                                    # the second run finds the first one's buffers
        step.zero_grads()
        dx = step.run()
    assert torch.equal(step.y, plain.y)
    assert len(set(b.data_ptr() for b in step.saved)) == 2 and len(step.store.ckpt) == 2
    dy = w.dy.astype(np.float64)
    block = torch.empty_like(step.saved[0])
    for i in (2, 1, 0):
        lw = dw.layers[i]
        if i < 2:
            H.checkpoint_restore(dw.cfg, S.CHECKPOINTS[fmt], step.store.ckpt[i], dw.T, lw.ln_gamma, lw.ln_beta, block)
            v = {n: f64(t) for n, t in H.saved_views(dw.cfg, block, dw.T).items()}
        else:
            v = {n: f64(t) for n, t in H.saved_views(dw.cfg, plain.saved[2], dw.T).items()}
        x = v["xlow"] if "xlow" in v else f64(plain.acts[i])
        dy, gr = backward_of(w, lcfg(w), v, x, lp(w.params[i]).as_f64(), dy)
        # a bf16 gradient carries the rounding of every layer above
        for n in LAYER_GRADS:
            check_grad(getattr(step.grads[i], n), gr[n], TOL[dtype], (i, n))
    check_grad(dx, dy, TOL[dtype], "dX")


def normed_oracle(w, joints, gates, dy, kinds):
    """Forward and backward of NormedTrainStep in fp64."""
    cfg, eps, params = lcfg(w), w.ln_eps, [lp(p).as_f64() for p in w.params]
    q = [{n: f64(getattr(j, n)) for n in ("post_gamma", "post_beta", "res_scale", "pre_gamma", "pre_beta")} for j in joints]
    y, keep = w.x.astype(np.float64), []
    h, m2, r2 = A.block_h(kinds, q[0], y, eps)
    one = np.ones((w.T, 1))
    st = np.concatenate([0 * one, one, m2, r2], 1)
    joint = [(y, None, None, st)]
    for i, p in enumerate(params):
        pre = h @ p.W1 + p.b1
        g = R.silu(pre)
        o = R.attention_forward(g, w.seq_offsets, w.timestamps, w.num_targets, p.rab_pos, p.rab_time, cfg)
        z, mean, rstd = R.ln_gate_forward(o, g[:, :w.d_model], p.gamma, p.beta, eps)
        b = z @ p.W2 + p.b2
        keep.append(({"pre": pre, "g": g, "o": o, "z": z, "mean": mean, "rstd": rstd}, h))
        y, m1, r1 = A.block_y(kinds, q[i + 1], y, b, gates[i], eps)
        if i + 1 < len(params):
            h, m2, r2 = A.block_h(kinds, q[i + 1], y, eps)
        joint.append((y, b, gates[i], np.concatenate([m1, r1, m2, r2], 1)))
    out = {"y": y, "layers": [None] * len(params), "joints": [None] * len(joint)}
    dh = None
    for i in range(len(params), 0, -1):
        jg = A.block_bwd(kinds, q[i], *joint[i], dy, dh)
        out["joints"][i] = jg
        v, h = keep[i - 1]
        p = params[i - 1]
        dxh, gr = backward_of(w, cfg, v, h, p, jg["db"])
        out["layers"][i - 1] = gr
        dh, dy = dxh - jg["db"], jg["dx"]               # the block has no residual sum of its own
    out["joints"][0] = A.block_bwd(kinds, q[0], *joint[0], dy, dh)
    out["dx"] = out["joints"][0]["dx"]
    return out


def make_normed(w, dw, kinds, seed=3):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt = H.torch_dtype(dw.cfg.dtype)
    rnd = lambda *s, m=0.0, std=0.3: torch.empty(*s, device=DEV).normal_(m, std, generator=g).to(dt)
    d = w.d_model
    joints = [H.BlockNorm(post=kinds["post"], pre=kinds["pre"], gate_act=kinds["gate"], post_gamma=rnd(d, m=1.0), post_beta=rnd(d),
                          res_scale=rnd(d, m=0.7), pre_gamma=rnd(d, m=1.0), pre_beta=rnd(d)) for _ in range(len(dw.layers) + 1)]
    gates = [rnd(w.T, d, std=1.0) if i != 1 else None for i in range(len(dw.layers))]
    return joints, gates


@pytest.mark.parametrize("dtype,post,pre", [("f32", "layer", "layer"), ("f32", "rms", "rms"), ("bf16", "rms", "layer")])
def test_normed_stack(dtype, post, pre):
    w = small(dtype, layers=3)
    dw = S.DeviceWorkload.from_workload(w)
    kinds = {"post": post, "pre": pre, "gate": "silu"}
    joints, gates = make_normed(w, dw, kinds)
    step = S.NormedTrainStep(dw, joints, gates)
    for _ in range(2):
        step.zero_grads()
        dx = step.run()
    ref = normed_oracle(w, joints, [f64(g) for g in gates], w.dy.astype(np.float64), kinds)
    check(step.y, ref["y"], TOL[dtype], "y")
    check_grad(dx, ref["dx"], TOL[dtype], "dX")
    for i in range(3):
        for n in LAYER_GRADS:
            check_grad(getattr(step.grads[i], n), ref["layers"][i][n], TOL[dtype], (i, n))
        if gates[i] is not None:
            check_grad(step.dgates[i], ref["joints"][i + 1]["dgate"], TOL[dtype], (i, "gate"))
    for i in range(4):
        for n in vars(joints[i]):
            got = getattr(step.joint_grads[i], n, None)
            if got is None:
                continue
            want = ref["joints"][i].get(n)
            if want is None:
                assert not bool(got.any()), (i, n)
            else:
                check_grad(got, want, TOL[dtype], (i, n))


def test_normed_stack_from_checkpoints():
    """int8 checkpoints: the forward is the plain step's bit for bit, and the last layer's gradients (its block is not held) are
    the plain step's; the others start from activations within half a step of theirs, 2^-8 of a group's largest: gradients
    normwise within 2e-2, of which bf16 alone takes a good part."""
    w = small("bf16", layers=3)
    dw = S.DeviceWorkload.from_workload(w)
    joints, gates = make_normed(w, dw, {"post": "layer", "pre": "layer", "gate": "sigmoid"})
    a, b = S.NormedTrainStep(dw, joints, gates), S.NormedTrainStep(dw, joints, gates, checkpoints="int8")
    da, db = a.run().clone(), b.run().clone()
    assert torch.equal(a.y, b.y)
    for n in ("dW1", "dW2"):
        check_grad(getattr(b.grads[2], n), f64(getattr(a.grads[2], n)), 1e-4, n)
        for i in (0, 1):
            x, y = f64(getattr(a.grads[i], n)), f64(getattr(b.grads[i], n))
            assert np.linalg.norm(x - y) <= 2e-2 * np.linalg.norm(x), (i, n)
    assert np.linalg.norm(f64(da - db)) <= 2e-2 * np.linalg.norm(f64(da))


def test_captured_training_step():
    """A step with an embedding and checkpoints captured into a graph, while eager runs of the same buffers go on beside it."""
    w = small("bf16")
    rng = np.random.default_rng(6)
    dw = S.DeviceWorkload.from_workload(w)
    emb = S.ItemEmbedding(torch.from_numpy(rng.normal(0, 0.1, (50, 128)).astype(np.float32)).to(DEV))
    ids = torch.from_numpy(rng.integers(0, 50, size=w.T)).to(DEV)
    step = S.TrainStep(dw, checkpoints="int8", embedding=emb, ids=ids)

    def one():
        step.zero_grads()
        emb.zero_grad()
        return step.run()

    dx = one()
    want = (step.y.clone(), dx.clone(), emb.grad.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dx = one()
    for new in (ids.clone(), ids.flip(0).contiguous()):
        ids.copy_(new)
        graph.replay()
        got = (step.y.clone(), dx.clone(), emb.grad.clone())
        one()
        torch.cuda.synchronize()
        ref = (step.y, step.gbuf[0], emb.grad)
        assert torch.equal(got[0], ref[0])
        for a, b in zip(got[1:], ref[1:]):               # the layers' backward adds in no fixed order
            check_grad(a, f64(b), 1e-2, "replay")
    assert not torch.equal(got[0], want[0])


def test_wrong_stacks_are_refused():
    dw = S.DeviceWorkload.from_workload(small("bf16"))
    with pytest.raises(ValueError):
        S.TrainStep(dw, checkpoints="int4")
    with pytest.raises(ValueError):
        S.TrainStep(dw, ids=torch.zeros(dw.T, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError):
        S.NormedTrainStep(dw, [H.BlockNorm()] * 2)


def test_rows_gradient_on_another_stream():
    """The rows form's first call on a side stream while the current one is busy: the buffers that it makes are cleared on the
    stream that writes them, so no fill comes after the gradient.  Sums of one 1.0 for each event are exact."""
    side = torch.cuda.Stream()
    ids = torch.arange(600, device=DEV).repeat(3)
    dx = torch.ones(1800, 64, device=DEV)
    emb = S.ItemEmbedding(torch.zeros(1000, 64, device=DEV), scale=1.0, rows=True)
    busy = torch.ones(64 << 20, device=DEV)
    torch.cuda.synchronize()
    for _ in range(50):
        busy.mul_(1.0)
    emb.backward(dx, ids, stream=side)
    torch.cuda.synchronize()
    assert int(emb.count) == 600
    assert torch.equal(emb.row_ids[:600], torch.arange(600, device=DEV))
    assert torch.equal(emb.rows[:600], torch.full((600, 64), 3.0, device=DEV))

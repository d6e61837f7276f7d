"""Norms before and after a block with its gate and residual scale (CUDA, through the C ABI) against the fp64 oracle.

Tolerances, with u = 2^-24.  A row's fp32 sums are trees over at most 2048 elements, so a mean or spread is off by no more
than about 16 u relative to the magnitudes it sums; a normalised value takes three more operations, the affine map two, the
gate ten (its exponential's argument, at most 12 in magnitude, is rounded before it is scaled by log2 e: 17 u) and the sum two.
Under K = 64 roundings each relative to the magnitudes that enter (kept below as absolute sums, so cancellation is counted),
then half a step of the type that is written: 2^-8 for bf16, 2^-24 for fp32.  A column sum of T terms adds T + 8 roundings of the
terms' magnitudes.  The backward's reference starts from the statistics and the y that the kernel's forward wrote."""
import numpy as np
import pytest
import torch

from oracle import around_layers as A
from hstu_sequential_transducer_b200 import build
from hstu_sequential_transducer_b200 import hstu as H

pytestmark = pytest.mark.gpu
DEV = "cuda"
U, K = 2.0 ** -24, 64
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
PARAMS = ("post_gamma", "post_beta", "res_scale", "pre_gamma", "pre_beta")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    H.lib()


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def make(T, d, dt, io, post, pre, gate, params, seed=0, gate_cols=1, mean=0.2):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s, m=0.0, std=1.0: torch.empty(*s, device=DEV).normal_(m, std, generator=g)
    heads = d // 32
    cfg = H.make_config(d, heads, 64.0, H.HSTU_F32 if dt == "f32" else H.HSTU_BF16,
                        io_dtype=H.HSTU_F32 if io == "f32" else H.HSTU_BF16)
    p = {n: (rnd(d, m=0.0 if "beta" in n else 1.0, std=0.3).to(DT[dt]) if n in params else None) for n in PARAMS}
    bn = H.BlockNorm(post=post, pre=pre, gate_act=gate, **p)
    x, b = rnd(T, d).to(DT[io]), rnd(T, d, m=mean).to(DT[io])
    wide = rnd(T, d * gate_cols).to(DT[dt]) if gate != "absent" else None
    if gate == "absent":
        bn.gate_act = None
    return cfg, bn, p, x, b, (wide[:, :d] if wide is not None else None), rnd


def close(got, want, err, dtype, what):
    tol = err + HALF[dtype] * (np.abs(want) + err) + 1e-37
    off = np.abs(f64(got) - want) / tol
    assert np.all(off <= 1), (what, float(off.max()))


def magnitudes(kind, a, m, r):
    """Bound of the error of normalised rows, in units of K u."""
    return (np.abs(a) + np.abs(m)) * r


def forward_and_check(cfg, bn, p, x, b, gate, T, d, **kw):
    stats = torch.full((T, 4), np.nan, device=DEV)
    y, h = H.block_norm_fwd(cfg, bn, x, b, gate, stats=stats, **kw)
    c = {"post": bn.post, "pre": bn.pre, "gate": bn.gate_act}
    q = {n: f64(t) for n, t in p.items()}
    eps = float(np.float32(cfg.ln_eps))
    one = lambda n: np.abs(q[n]) if q[n] is not None else 1.0
    zero = lambda n: np.abs(q[n]) if q[n] is not None else 0.0
    if b is not None:
        want, m, r = A.block_y(c, q, f64(x), f64(b), f64(gate), eps)
        amp = magnitudes(bn.post, f64(b), m, r) * (one("post_gamma") if bn.post else 1.0) + (zero("post_beta") if bn.post else 0.0)
        if gate is not None:
            amp = amp * np.maximum(np.abs(A.act(bn.gate_act, f64(gate))[0]), 0)
        close(y, want, K * U * (np.abs(f64(x)) + one("res_scale") * amp), y.dtype, "y")
        st = f64(stats)
        big = np.abs(f64(b)).max(1, keepdims=True)
        assert np.all(np.abs(st[:, :1] - m) <= K * U * big)
        assert np.all(np.abs(st[:, 1:2] - r) <= K * U * r * (1 + big * r))
    want, m, r = A.block_h(c, q, f64(y), eps)
    if h is not None:
        amp = magnitudes(bn.pre, f64(y), m, r) * (one("pre_gamma") if bn.pre else 1.0) + (zero("pre_beta") if bn.pre else 0.0)
        close(h, want, K * U * amp, h.dtype, "h")
    return y, h, stats, c, q


def backward_and_check(cfg, bn, p, y, b, gate, stats, rnd, T, d, c, q, dy=True, dh=True, wide=1):
    io, dt = H.torch_dtype(cfg.io_dtype), H.torch_dtype(cfg.dtype)
    up_y = rnd(T, d).to(io) if dy else None
    up_h = rnd(T, d).to(io) if dh else None
    dx = torch.full((T, d), np.nan, dtype=io, device=DEV)
    db = torch.full((T, d), np.nan, dtype=dt, device=DEV) if b is not None else None
    dg = torch.full((T, d * wide), 3.0, dtype=dt, device=DEV)[:, :d] if gate is not None else None
    grads = H.BlockNormGrads(**{n: (rnd(d) if p[n] is not None else None) for n in PARAMS})
    prior = {n: f64(getattr(grads, n)) for n in PARAMS}
    first = {n: (None if getattr(grads, n) is None else getattr(grads, n).clone()) for n in PARAMS}
    H.block_norm_bwd(cfg, bn, y, b, gate, stats, dy=up_y, dh=up_h, dx=dx, db=db, dgate=dg, grads=grads)
    want = A.block_bwd(c, q, f64(y), f64(b), f64(gate), f64(stats), f64(up_y), f64(up_h))
    st = f64(stats)
    m1, r1, m2, r2 = (st[:, i:i + 1] for i in range(4))
    zero = np.zeros((T, d))
    a = lambda n: np.abs(q[n]) if q[n] is not None else 1.0
    mean = lambda v: v.mean(1, keepdims=True)
    # magnitudes that enter e, dp, ...; n*: bounds of |normalised value| with its own error's reach
    E = zero if up_y is None else np.abs(f64(up_y))
    sums = {}
    if dh:
        g = np.abs(f64(up_h))
        n2 = (np.abs(f64(y)) + np.abs(m2)) * r2
        if bn.pre:
            sums["pre_gamma"], sums["pre_beta"] = g * n2, g
            g = g * a("pre_gamma")
            g = r2 * (g + mean(g) + n2 * mean(g * n2))
        E = E + g
    close(dx, want["dx"], K * U * E, io, "dx")
    if b is not None:
        n1 = (np.abs(f64(b)) + np.abs(m1)) * r1
        v = n1 * a("post_gamma") + (np.abs(q["post_beta"]) if q["post_beta"] is not None else 0.0) if bn.post else np.abs(f64(b))
        act, slope = (np.abs(t) for t in A.act(bn.gate_act, f64(gate))) if gate is not None else (1.0, 0.0)
        sums["res_scale"] = E * v * act
        dv = E * a("res_scale")
        if gate is not None:
            # the slope's own terms: |s| + |u| s (1 - s), bounded by 1 + |u|
            close(dg, want["dgate"], K * U * dv * v * (slope + 1 + np.abs(f64(gate))), dt, "dgate")
            if wide > 1:
                assert bool((dg._base[:, d:] == 3).all())
        dp = dv * act
        if bn.post:
            sums["post_gamma"], sums["post_beta"] = dp * n1, dp
            g = dp * a("post_gamma")
            dp = r1 * (g + mean(g) + n1 * mean(g * n1))
        close(db, want["db"], 2 * K * U * dp, dt, "db")
    for n in PARAMS:
        if prior[n] is None:
            continue
        if n not in want:
            np.testing.assert_array_equal(f64(getattr(grads, n)), prior[n])
            continue
        tol = (2 * K + T + 8) * U * (sums[n].sum(0) + np.abs(prior[n]))
        off = np.abs(f64(getattr(grads, n)) - prior[n] - want[n]) / tol
        assert np.all(off <= 1), (n, float(off.max()))
    # again: the same bits, dx over dy
    again = H.BlockNormGrads(**first)
    dx2 = up_y.clone() if dy else None
    dx2 = H.block_norm_bwd(cfg, bn, y, b, gate, stats, dy=dx2, dh=up_h, dx=dx2, grads=again)
    assert torch.equal(dx2, dx)
    for n in PARAMS:
        if first[n] is not None:
            assert torch.equal(getattr(again, n), getattr(grads, n)), n


ALL = set(PARAMS)


@pytest.mark.parametrize("dt,io", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("T,d", [(1, 32), (5, 64), (333, 96), (1, 256), (37, 288), (70, 512), (9, 544), (1, 1024), (1501, 1024),
                                 (13, 1056), (21, 2048)])
def test_sizes_and_types(dt, io, T, d):
    cfg, bn, p, x, b, gate, rnd = make(T, d, dt, io, "layer", "layer", "silu", ALL, seed=T + d)
    y, h, st, c, q = forward_and_check(cfg, bn, p, x, b, gate, T, d)
    backward_and_check(cfg, bn, p, y, b, gate, st, rnd, T, d, c, q)


@pytest.mark.parametrize("post", ["layer", "rms", None])
@pytest.mark.parametrize("pre", ["layer", "rms", None])
@pytest.mark.parametrize("gate", ["silu", "sigmoid", None, "absent"])
def test_kinds(post, pre, gate):
    T, d = 45, 160
    cfg, bn, p, x, b, u, rnd = make(T, d, "bf16", "f32", post, pre, gate, ALL, gate_cols=3)
    y, h, st, c, q = forward_and_check(cfg, bn, p, x, b, u, T, d)
    backward_and_check(cfg, bn, p, y, b, u, st, rnd, T, d, c, q, wide=2)


@pytest.mark.parametrize("params", [set(), {"post_gamma"}, {"res_scale", "pre_beta"}, {"post_beta", "pre_gamma"}])
def test_absent_parameters(params):
    T, d = 40, 320
    cfg, bn, p, x, b, u, rnd = make(T, d, "bf16", "bf16", "layer", "rms", "sigmoid", params)
    y, h, st, c, q = forward_and_check(cfg, bn, p, x, b, u, T, d)
    backward_and_check(cfg, bn, p, y, b, u, st, rnd, T, d, c, q)


@pytest.mark.parametrize("dy,dh", [(True, False), (False, True), (False, False)])
def test_absent_upstream(dy, dh):
    T, d = 33, 128
    cfg, bn, p, x, b, u, rnd = make(T, d, "bf16", "f32", "rms", "layer", "silu", ALL)
    y, h, st, c, q = forward_and_check(cfg, bn, p, x, b, u, T, d)
    backward_and_check(cfg, bn, p, y, b, u, st, rnd, T, d, c, q, dy=dy, dh=dh)


def test_start_and_end_of_a_stack():
    """Without a block: y is x and only Norm_pre applies.  Without a next block: h is not made."""
    T, d = 50, 192
    cfg, bn, p, x, b, u, rnd = make(T, d, "bf16", "f32", "layer", "layer", "silu", ALL)
    y, h, st, c, q = forward_and_check(cfg, bn, p, x, None, None, T, d)
    assert y is x
    backward_and_check(cfg, bn, p, y, None, None, st, rnd, T, d, c, q)
    y, h = H.block_norm_fwd(cfg, bn, x, b, u, want_h=False)
    assert h is None
    y2 = x.clone()
    H.block_norm_fwd(cfg, bn, y2, b, u, y=y2)          # in place
    assert torch.equal(y2, y)


@pytest.mark.parametrize("dt,io", [("f32", "f32"), ("bf16", "bf16")])
def test_rows_far_from_zero(dt, io):
    """A mean many times the spread costs the statistics nothing but the input's own rounding; constant rows give beta."""
    T, d = 65, 384
    cfg, bn, p, x, b, u, rnd = make(T, d, dt, io, "layer", "layer", "silu", ALL, mean=300.0)
    b[3] = 5.0
    y, h, st, c, q = forward_and_check(cfg, bn, p, x, b, u, T, d)
    backward_and_check(cfg, bn, p, y, b, u, st, rnd, T, d, c, q)


def test_non_finite_rows_stay_alone():
    T, d = 64, 256
    cfg, bn, p, x, b, u, rnd = make(T, d, "bf16", "f32", "layer", "rms", "silu", ALL)
    y0, h0 = H.block_norm_fwd(cfg, bn, x, b, u)
    b[7, 3], x[9, 9], u[11, 200] = float("nan"), float("inf"), float("-inf")
    y, h = H.block_norm_fwd(cfg, bn, x, b, u)
    keep = [t for t in range(T) if t not in (7, 9, 11)]
    assert torch.equal(y[keep], y0[keep]) and torch.equal(h[keep], h0[keep])
    assert bool(torch.isnan(h[7]).all()) and bool(torch.isnan(y[7]).all())


def test_empty():
    cfg, bn, p, x, b, u, rnd = make(0, 64, "bf16", "f32", "layer", "layer", "silu", ALL)
    y, h = H.block_norm_fwd(cfg, bn, x, b, u)
    assert y.shape == (0, 64) and h.shape == (0, 64)
    g = H.BlockNormGrads.zeros_like(bn)
    H.block_norm_bwd(cfg, bn, y, b, u, torch.empty(0, 4, device=DEV), dy=x, dh=x, grads=g)
    assert all(float(getattr(g, n).abs().max()) == 0 for n in PARAMS)


def test_offsets_past_32_bits():
    """[T][d] of more than 2^31 elements: the last rows are computed as they are alone."""
    d = 1024
    T = (1 << 31) // d + 3
    cfg, bn, p, x, b, u, rnd = make(4, d, "bf16", "bf16", "layer", "layer", "silu", ALL)
    big_x = torch.zeros(T, d, dtype=torch.bfloat16, device=DEV)
    big_b, big_u = torch.zeros_like(big_x), torch.zeros_like(big_x)
    for big, t in ((big_x, x), (big_b, b), (big_u, u)):
        big[-4:] = t
    want = H.block_norm_fwd(cfg, bn, x, b, u)
    y, h = H.block_norm_fwd(cfg, bn, big_x, big_b, big_u)
    assert torch.equal(y[-4:], want[0]) and torch.equal(h[-4:], want[1])


def test_other_stream_and_graph():
    T, d = 300, 512
    cfg, bn, p, x, b, u, rnd = make(T, d, "bf16", "f32", "layer", "layer", "silu", ALL)
    stats = torch.empty(T, 4, device=DEV)
    y, h = H.block_norm_fwd(cfg, bn, x, b, u, stats=stats)
    dy, dh = rnd(T, d), rnd(T, d)
    g = H.BlockNormGrads.zeros_like(bn)
    dx = H.block_norm_bwd(cfg, bn, y, b, u, stats, dy=dy, dh=dh, grads=g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    g2, y2, h2, st2, dx2 = H.BlockNormGrads.zeros_like(bn), torch.empty_like(y), torch.empty_like(h), torch.empty_like(stats), torch.empty_like(dx)
    torch.cuda.synchronize()
    H.block_norm_fwd(cfg, bn, x, b, u, y=y2, h=h2, stats=st2, stream=side)
    H.block_norm_bwd(cfg, bn, y2, b, u, st2, dy=dy, dh=dh, dx=dx2, grads=g2, stream=side)
    side.synchronize()
    assert torch.equal(y, y2) and torch.equal(h, h2) and torch.equal(dx, dx2)
    assert all(torch.equal(getattr(g, n), getattr(g2, n)) for n in PARAMS)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        H.block_norm_fwd(cfg, bn, x, b, u, y=y2, h=h2, stats=st2)
        H.block_norm_bwd(cfg, bn, y2, b, u, st2, dy=dy, dh=dh, dx=dx2, grads=g2)
    for n in PARAMS:
        getattr(g2, n).zero_()
    x.mul_(0.5)
    graph.replay()
    g.post_gamma.zero_()
    y, h = H.block_norm_fwd(cfg, bn, x, b, u, stats=stats)
    H.block_norm_bwd(cfg, bn, y, b, u, stats, dy=dy, dh=dh, dx=dx, grads=g)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(h, h2) and torch.equal(dx, dx2) and torch.equal(g.post_gamma, g2.post_gamma)


@pytest.mark.parametrize("T", [1, 2, 300, 20_000])
@pytest.mark.parametrize("shared", [("post_gamma", "pre_gamma"), ("post_beta", "pre_beta", "res_scale"), PARAMS])
def test_parameters_that_share_a_gradient(T, shared):
    """One array for several parameters takes the sum of theirs, added in their order onto what it held: the separate gradients
    give it to within the len(shared) fp32 additions of values no larger than the magnitudes added."""
    d = 224
    cfg, bn, p, x, b, u, rnd = make(T, d, "bf16", "f32", "layer", "layer", "silu", ALL)
    stats = torch.empty(T, 4, device=DEV)
    y, _ = H.block_norm_fwd(cfg, bn, x, b, u, stats=stats)
    dy, dh = rnd(T, d), rnd(T, d)
    apart = H.BlockNormGrads.zeros_like(bn)
    H.block_norm_bwd(cfg, bn, y, b, u, stats, dy=dy, dh=dh, grads=apart)
    prior = rnd(d)
    for _ in range(2):
        one = prior.clone()
        H.block_norm_bwd(cfg, bn, y, b, u, stats, dy=dy, dh=dh, grads=H.BlockNormGrads(**{n: one for n in shared}))
        terms = np.stack([f64(prior)] + [f64(getattr(apart, n)) for n in shared])
        assert np.all(np.abs(f64(one) - terms.sum(0)) <= len(shared) * U * np.abs(terms).sum(0))


# A CTA's loop over its rows: rows are copied ahead into slots that the step before leaves, parameters' sums go on from step to
# step.  A team of threads takes 4 rows at a time forward, 1 or 2 backward.
def team_of(d):
    if d > 256:
        return (d + 255) // 256 * 32
    t = 4
    while 8 * t < d:
        t *= 2
    return t


def rows_a_step(d, backward=False):
    """Rows that the resident CTAs take together in one step."""
    team = team_of(d)
    threads = max(team, 128) if team < 96 else team
    if not backward:
        rows, resident = 4, 2 if threads > 192 else 384 // threads
    else:
        rows = 1 if team == 96 or 128 < team < 256 else 2
        resident = (512 if rows == 1 else 256) // threads
    return threads // team * rows * resident * torch.cuda.get_device_properties(0).multi_processor_count


def three_steps(d):
    """Rows for two steps of every CTA forward, a third of some and a last one in part; more steps backward."""
    assert rows_a_step(d, True) <= rows_a_step(d)
    return 2 * rows_a_step(d) + rows_a_step(d) // 3 + 5


TYPES = [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")]


@pytest.mark.parametrize("d", [32, 224, 512, 768, 1024, 1056, 1536, 1792, 2048])
@pytest.mark.parametrize("kind", range(3))
def test_many_steps(d, kind):
    """Every kind of team (below a warp, whole warps, one or two rows backward), each with three types and kinds of norm and gate."""
    dt, io = TYPES[(kind + d // 32) % 3]
    post, pre, gate = [("layer", "layer", "silu"), (None, "rms", "sigmoid"), ("rms", None, "absent")][kind]
    T = three_steps(d)
    cfg, bn, p, x, b, u, rnd = make(T, d, dt, io, post, pre, gate, ALL, seed=d + kind)
    y, h, st, c, q = forward_and_check(cfg, bn, p, x, b, u, T, d)
    backward_and_check(cfg, bn, p, y, b, u, st, rnd, T, d, c, q)


@pytest.mark.parametrize("d", [32, 512, 768, 2048])
@pytest.mark.parametrize("pre", ["layer", None])
def test_many_steps_at_the_start_of_a_stack(d, pre):
    """Without a block: x alone is copied ahead."""
    T = three_steps(d)
    cfg, bn, p, x, _, _, rnd = make(T, d, "bf16", "f32", "layer", pre, "absent", ALL, seed=d)
    y, h, st, c, q = forward_and_check(cfg, bn, p, x, None, None, T, d)
    backward_and_check(cfg, bn, p, y, None, None, st, rnd, T, d, c, q)


@pytest.mark.parametrize("d", [64, 512, 1056, 2048])
@pytest.mark.parametrize("post", ["layer", None])
def test_many_steps_in_place(d, post):
    """y over x, and no h: the rows copied ahead are others than those that are written."""
    T = three_steps(d)
    cfg, bn, p, x, b, u, rnd = make(T, d, "bf16", "f32", post, "rms", "silu", ALL, seed=d)
    y, h = H.block_norm_fwd(cfg, bn, x, b, u)
    again = x.clone()
    y2, h2 = H.block_norm_fwd(cfg, bn, again, b, u, y=again)
    assert y2 is again and torch.equal(y2, y) and torch.equal(h2, h)
    y3, h3 = H.block_norm_fwd(cfg, bn, x, b, u, want_h=False)
    assert h3 is None and torch.equal(y3, y)


@pytest.mark.parametrize("T", [2, 3, 4, 8])
@pytest.mark.parametrize("d", [512, 768, 1024, 1056, 2048])
def test_two_steps_by_one_cta(T, d):
    """Two steps backward are left to one CTA, which adds its sums to the gradients itself (2 rows at 768 and
    1,056, which take one a step; 3 and 4 at 1,024 and 2,048; 8 at 512, two teams)."""
    for dt, io in TYPES:
        cfg, bn, p, x, b, u, rnd = make(T, d, dt, io, "layer", "rms", "silu", ALL, seed=T)
        y, h, st, c, q = forward_and_check(cfg, bn, p, x, b, u, T, d)
        backward_and_check(cfg, bn, p, y, b, u, st, rnd, T, d, c, q)

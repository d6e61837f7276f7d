"""Activation checkpoints in 8 bits (CUDA, through the C ABI) against the fp64 oracle.

What is held has one rounding, at a power-of-two scale: the bytes, scales and restored Pre, X and deviations are compared bit
for bit (the deviation is the fp32 difference O - mean, the restored O the fp32 sum).  G and Z take under 64 fp32 roundings
(u = 2^-24) of the magnitudes that enter, then half a step of the type they are written in (bf16 2^-8, fp32 2^-24)."""
import numpy as np
import pytest
import torch

from oracle import around_layers as A
from hstu_sequential_transducer_b200 import build
from hstu_sequential_transducer_b200 import hstu as H

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
FMT = {"int8": H.CKPT_INT8, "e4m3": H.CKPT_E4M3}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    H.lib()


def f64(t):
    return t.detach().double().cpu().numpy()


def make(T, d, dt, io, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.empty(*s, device=DEV).normal_(generator=g)
    cfg = H.make_config(d, d // 32, 64.0, H.HSTU_F32 if dt == "f32" else H.HSTU_BF16,
                        io_dtype=H.HSTU_F32 if io == "f32" else H.HSTU_BF16)
    n = H.saved_layout(cfg, T)[-1]
    saved = torch.full((max(n, 1),), 0x55, dtype=torch.uint8, device=DEV)
    v = H.saved_views(cfg, saved, T)
    v["pre"].copy_(rnd(T, 4 * d) * torch.exp(rnd(T, 1)))
    v["o"].copy_(rnd(T, d) * 0.05 + rnd(T, 1) * 0.1 + 0.4)
    if T:
        v["mean"].copy_(v["o"].mean(1))
        v["rstd"].copy_(1 / torch.sqrt(v["o"].var(1, unbiased=False) + 1e-5))
    if "xlow" in v:
        v["xlow"].copy_(rnd(T, d))
    gamma, beta = (1 + 0.1 * rnd(d)).to(H.torch_dtype(cfg.dtype)), (0.1 * rnd(d)).to(H.torch_dtype(cfg.dtype))
    return cfg, saved, v, gamma, beta


def parts(cfg, ckpt, T):
    off = H.checkpoint_layout(cfg, T)
    d = cfg.d_model
    x = d if cfg.io_dtype != cfg.dtype else 0
    w = [4 * d, d, x, 4 * d // 32, d // 32, x // 32]
    return [ckpt[off[i]:off[i] + T * w[i]].view(T, w[i]).cpu().numpy() for i in range(6)]


def decode(fmt, byte):
    if fmt == "int8":
        return byte.view(np.int8).astype(np.float64)
    mag = (byte & 127).astype(np.int64)
    assert np.all(mag < 127)
    return np.where(byte & 128, -1.0, 1.0) * A.E4M3[mag]


def round_trip(cfg, fmt, saved, T, gamma, beta):
    ckpt = torch.full((max(H.checkpoint_bytes(cfg, FMT[fmt], T), 1),), 0xAB, dtype=torch.uint8, device=DEV)
    H.checkpoint_save(cfg, FMT[fmt], saved, T, ckpt)
    back = torch.full_like(saved, 0xFF)
    H.checkpoint_restore(cfg, FMT[fmt], ckpt, T, gamma, beta, back)
    return ckpt, H.saved_views(cfg, back, T)


def check(cfg, fmt, v, ckpt, r, T, gamma, beta):
    d = cfg.d_model
    low = H.torch_dtype(cfg.dtype)
    half = 2.0 ** -8 if low == torch.bfloat16 else 2.0 ** -24
    dev = (v["o"] - v["mean"][:, None])
    src = [f64(v["pre"]), f64(dev)] + ([f64(v["xlow"])] if "xlow" in v else [])
    got = parts(cfg, ckpt, T)
    held = [A.hold(fmt, s) for s in src]
    for i, (q, k, _) in enumerate(held):
        np.testing.assert_array_equal(got[3 + i].astype(np.int64) - 127, k)
        np.testing.assert_array_equal(decode(fmt, got[i]), q)
    pre = held[0][2]
    np.testing.assert_array_equal(f64(r["pre"]), pre)
    np.testing.assert_array_equal(f64(r["o"]), (f64(v["mean"])[:, None].astype(np.float32) + held[1][2].astype(np.float32)).astype(np.float64))
    for n in ("mean", "rstd"):
        assert torch.equal(r[n], v[n])
    if "xlow" in v:
        np.testing.assert_array_equal(f64(r["xlow"]), held[2][2])
    s = 1 / (1 + np.exp(-pre))
    # exp's argument is rounded before it is scaled by log2 e: |pre| more roundings
    err = (64 + 2 * np.abs(pre)) * U * np.abs(pre * s)
    assert np.all(np.abs(f64(r["g"]) - pre * s) <= err + half * (np.abs(pre * s) + err) + 1e-37)
    ln = held[1][2] * f64(v["rstd"])[:, None] * (1 if gamma is None else f64(gamma)) 
    b = 0.0 if beta is None else f64(beta)
    gate = f64(r["g"])[:, :d]
    err = 64 * U * (np.abs(ln) + np.abs(b)) * np.abs(gate)
    want = (ln + b) * gate
    assert np.all(np.abs(f64(r["z"]) - want) <= err + half * (np.abs(want) + err) + 1e-37)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dt,io", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("T,d", [(1, 32), (3, 64), (130, 96), (77, 512), (19, 1056), (5, 2048)])
def test_round_trip(fmt, dt, io, T, d):
    cfg, saved, v, gamma, beta = make(T, d, dt, io, seed=T)
    ckpt, r = round_trip(cfg, fmt, saved, T, gamma, beta)
    check(cfg, fmt, v, ckpt, r, T, gamma, beta)
    assert H.checkpoint_bytes(cfg, FMT[fmt], T) <= (6.1875 * d + 8) * T + 8 * 256


@pytest.mark.parametrize("gamma,beta", [(True, False), (False, True), (False, False)])
def test_absent_affine(gamma, beta):
    T, d = 21, 128
    cfg, saved, v, g, b = make(T, d, "bf16", "f32")
    g, b = g if gamma else None, b if beta else None
    ckpt, r = round_trip(cfg, "int8", saved, T, g, b)
    check(cfg, "int8", v, ckpt, r, T, g, b)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_extreme_groups(fmt):
    """Zero groups, values at and next to the scale's borders, the largest and smallest magnitudes, ties."""
    T, d = 8, 64
    cfg, saved, v, gamma, beta = make(T, d, "f32", "f32")
    top = 127.0 if fmt == "int8" else 448.0
    p = v["pre"]
    p[0] = 0.0
    p[1, :32] = top
    p[1, 32:64] = float(np.nextafter(np.float32(top), np.float32(1e9)))
    p[2, :32] = torch.finfo(torch.float32).max
    p[2, 32:64] = -torch.finfo(torch.float32).max / 2
    p[3, :32] = 2.0 ** -126 * top
    p[3, 32:64] = 2.0 ** -140
    p[3, 64:96] = 2.0 ** -149
    p[4, :32] = torch.arange(32, device=DEV) + 0.5
    p[4, 0] = top
    p[5, :32] = -0.0
    ckpt, r = round_trip(cfg, fmt, saved, T, gamma, beta)
    got, want = parts(cfg, ckpt, T), A.hold(fmt, f64(p))
    np.testing.assert_array_equal(got[3].astype(np.int64) - 127, want[1])
    np.testing.assert_array_equal(decode(fmt, got[0]), want[0])
    np.testing.assert_array_equal(f64(r["pre"]), want[2])
    assert bool(torch.isfinite(r["g"]).all())


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_non_finite_groups(fmt):
    """A group with an infinity or NaN comes back as NaN; its neighbours are as they would be."""
    T, d = 6, 64
    cfg, saved, v, gamma, beta = make(T, d, "bf16", "f32")
    _, r0 = round_trip(cfg, fmt, saved, T, gamma, beta)
    keep = r0["pre"].clone()
    for row, col, bad in ((1, 5, float("nan")), (2, 70, float("inf")), (4, 255, float("-inf"))):
        v["pre"][row, col] = bad
    _, r = round_trip(cfg, fmt, saved, T, gamma, beta)
    hit = torch.zeros(T, 4 * d, dtype=torch.bool, device=DEV)
    for row, col in ((1, 0), (2, 64), (4, 224)):
        hit[row, col:col + 32] = True
    assert bool(torch.isnan(r["pre"][hit]).all()) and torch.equal(r["pre"][~hit], keep[~hit])
    assert bool(torch.isnan(r["g"][hit]).all())


def test_empty():
    cfg, saved, v, gamma, beta = make(0, 64, "bf16", "f32")
    round_trip(cfg, "int8", saved, 0, gamma, beta)


def test_offsets_past_32_bits():
    """A block whose Pre has more than 2^32 elements: the last rows are held as they are alone."""
    d = 1024
    T = (1 << 32) // (4 * d) + 5
    few, s1, v1, gamma, beta = make(4, d, "bf16", "bf16")
    _, want = round_trip(few, "int8", s1, 4, gamma, beta)
    saved = torch.zeros(H.saved_layout(few, T)[-1], dtype=torch.uint8, device=DEV)
    v = H.saved_views(few, saved, T)
    for n in ("pre", "o", "mean", "rstd"):
        v[n][-4:] = v1[n]
    _, r = round_trip(few, "int8", saved, T, gamma, beta)
    for n in ("pre", "g", "o", "z", "mean", "rstd"):
        assert torch.equal(r[n][-4:], want[n]), n


def test_other_stream_and_graph():
    T, d = 200, 256
    cfg, saved, v, gamma, beta = make(T, d, "bf16", "f32")
    ckpt, r = round_trip(cfg, "e4m3", saved, T, gamma, beta)
    side = torch.cuda.Stream()
    back, ck = torch.zeros_like(saved), torch.zeros_like(ckpt)
    torch.cuda.synchronize()
    H.checkpoint_save(cfg, H.CKPT_E4M3, saved, T, ck, stream=side)
    H.checkpoint_restore(cfg, H.CKPT_E4M3, ck, T, gamma, beta, back, stream=side)
    side.synchronize()
    r2 = H.saved_views(cfg, back, T)
    assert all(torch.equal(r[n], r2[n]) for n in r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        H.checkpoint_save(cfg, H.CKPT_E4M3, saved, T, ck)
        H.checkpoint_restore(cfg, H.CKPT_E4M3, ck, T, gamma, beta, back)
    v["pre"].mul_(-1)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(r2["pre"], -r["pre"])

"""The operators around the layers refuse what they cannot do before any launch, with no writes (CPU only; the pointers are
never followed)."""
import ctypes

import pytest
import torch

from hstu_sequential_transducer_b200 import build
from hstu_sequential_transducer_b200 import hstu as H

OK, INVALID, UNSUPPORTED, CUDA, WORKSPACE = range(5)
P1, P2, P3, P4, WS = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000


@pytest.fixture(scope="module")
def L():
    build.build()
    return H.lib()


def cfg(**kw):
    c = H.make_config(kw.pop("d", 64), kw.pop("heads", 2), 64.0, kw.pop("dtype", H.HSTU_BF16), io_dtype=kw.pop("io", H.HSTU_F32))
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def test_embedding_fwd(L):
    good = dict(table=P1, tt=0, V=10, dim=8, ts=8, ids=P2, ib=8, T=4, scale=1.0, out=P3, ot=0, width=8, os=8, low=None, ls=0)
    call = lambda **kw: L.hstu_embedding_fwd(*{**good, **kw}.values(), None)
    assert call(T=0) == OK
    assert call(T=0, table=None, ids=None, out=None) == OK
    for kw in (dict(table=None), dict(ids=None), dict(out=None), dict(T=-1), dict(V=0), dict(dim=0), dict(tt=2), dict(ot=-1), dict(ib=2),
               dict(width=7), dict(ts=7), dict(os=7), dict(low=P4, ls=7), dict(low=P4, ls=8, ot=1)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(table=P1 + 2), dict(ids=P2 + 4), dict(out=P3 + 1), dict(low=P4 + 1, ls=8), dict(V=1 << 31), dict(T=1 << 31),
               dict(dim=65537, ts=65537, width=65537, os=65537), dict(width=65537, os=65537), dict(tt=1, table=P1 + 1)):
        assert call(**kw) == UNSUPPORTED, kw


def test_embedding_bwd(L):
    ws = L.hstu_embedding_bwd_workspace_size(100, 10, 8)
    assert ws > 0
    assert L.hstu_embedding_bwd_workspace_size(0, 10, 8) == L.hstu_embedding_bwd_workspace_size(-1, 10, 8) == 0
    assert L.hstu_embedding_bwd_workspace_size(5, 0, 8) == L.hstu_embedding_bwd_workspace_size(1 << 31, 9, 8) == 0
    good = dict(dout=P1, dt=0, ds=8, ids=P2, ib=8, T=100, V=10, dim=8, scale=1.0, g=P3, gs=8, ws=WS, n=ws)
    call = lambda **kw: L.hstu_embedding_bwd(*{**good, **kw}.values(), None)
    assert call(T=0, ws=None, n=0) == OK
    for kw in (dict(dout=None), dict(ids=None), dict(g=None), dict(ws=None), dict(T=-1), dict(V=-1), dict(dim=0), dict(dt=3), dict(ib=1), dict(ds=7), dict(gs=7)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(dout=P1 + 2), dict(ids=P2 + 4), dict(g=P3 + 2), dict(ws=WS + 8), dict(V=1 << 31)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(n=ws - 1) == WORKSPACE
    good = dict(dout=P1, dt=0, ds=8, ids=P2, ib=4, T=100, V=10, dim=8, scale=1.0, rid=P3, rows=P4, rs=8, cnt=P1, ws=WS, n=ws)
    call = lambda **kw: L.hstu_embedding_bwd_rows(*{**good, **kw}.values(), None)
    for kw in (dict(rid=None), dict(rows=None), dict(cnt=None), dict(rs=7), dict(dim=0), dict(ids=None)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(rid=P3 + 4), dict(cnt=P1 + 4), dict(rows=P4 + 2)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(n=ws - 1) == WORKSPACE
    assert call(T=0, cnt=None) == INVALID


def test_block_norm(L):
    c = cfg()
    bn = lambda **kw: H.CBlockNorm(**{**dict(post_kind=1, pre_kind=1, gate_act=2), **kw})
    good = dict(cfg=c, bn=bn(), x=P1, b=P2, gate=P3, gs=64, T=4, y=P4, h=P4, st=P1)
    call = lambda **kw: L.hstu_block_norm_fwd(*[ctypes.byref(v) if isinstance(v, ctypes.Structure) else v for v in {**good, **kw}.values()], None)
    assert call(T=0) == OK
    for kw in (dict(cfg=None), dict(bn=None), dict(x=None), dict(y=None), dict(T=-1), dict(gs=63), dict(bn=bn(post_kind=3)),
               dict(bn=bn(pre_kind=-1)), dict(bn=bn(gate_act=3)), dict(bn=bn(reserved=1)), dict(cfg=cfg(num_heads=3))):
        assert call(**kw) == INVALID, kw
    for kw in (dict(x=P1 + 4), dict(b=P2 + 8), dict(gate=P3 + 2), dict(gs=68), dict(h=P4 + 2), dict(st=P1 + 4), dict(bn=bn(post_gamma=P1 + 2)),
               dict(bn=bn(pre_beta=P1 + 8)), dict(cfg=cfg(head_dim=48, d_model=96))):
        assert call(**kw) == UNSUPPORTED, kw
    # nothing to write: a success without a launch
    assert call(b=None, y=None, h=None, st=None) == OK
    ws = L.hstu_block_norm_bwd_workspace_size(ctypes.byref(c), 4)
    assert ws > 0 and L.hstu_block_norm_bwd_workspace_size(ctypes.byref(c), 0) == 0
    assert L.hstu_block_norm_bwd_workspace_size(ctypes.byref(cfg(num_heads=3)), 4) == 0
    gr = H.CBlockNormGrads(res_scale=P2)
    good = dict(cfg=c, bn=bn(), y=P1, b=P2, gate=P3, gs=64, st=P1, dy=P2, dh=P3, T=4, dx=P4, db=P1, dg=P2, dgs=64, gr=gr, ws=WS, n=ws)
    call = lambda **kw: L.hstu_block_norm_bwd(*[ctypes.byref(v) if isinstance(v, ctypes.Structure) else v for v in {**good, **kw}.values()], None)
    assert call(T=0, n=0) == OK
    for kw in (dict(y=None), dict(st=None), dict(T=-1), dict(gs=8), dict(dgs=8), dict(ws=None), dict(bn=bn(gate_act=-1))):
        assert call(**kw) == INVALID, kw
    for kw in (dict(dy=P2 + 4), dict(dh=P3 + 2), dict(dx=P4 + 8), dict(db=P1 + 2), dict(dg=P2 + 2), dict(dgs=65), dict(ws=WS + 4),
               dict(gr=H.CBlockNormGrads(pre_beta=P2 + 2))):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(n=ws - 1) == WORKSPACE


def test_checkpoint(L):
    c = cfg()
    off = H.checkpoint_layout(c, 100)
    assert all(o % 256 == 0 for o in off) and off[1] >= 100 * 256 and off[-1] >= 100 * (6 * 64 + 12 + 8)
    assert H.checkpoint_bytes(c, H.CKPT_INT8, 100) == off[-1]
    same = H.checkpoint_layout(cfg(io=H.HSTU_BF16), 100)
    assert same[H.CKPT_X + 1] == same[H.CKPT_X]             # X is held only where the saved block has it
    assert L.hstu_checkpoint_layout(ctypes.byref(c), -1, (ctypes.c_size_t * 9)()) == INVALID
    assert L.hstu_checkpoint_layout(ctypes.byref(c), 5, None) == INVALID
    save = lambda c=c, f=0, s=P1, T=4, k=P2: L.hstu_checkpoint_save(ctypes.byref(c), f, s, T, k, None)
    rest = lambda c=c, f=0, k=P2, g=P3, b=P3, T=4, s=P1: L.hstu_checkpoint_restore(ctypes.byref(c), f, k, g, b, T, s, None)
    assert save(T=0, s=None, k=None) == rest(T=0, s=None, k=None) == OK
    for st in (save(f=2), save(f=-1), save(s=None), save(k=None), save(T=-1), rest(f=2), rest(s=None), rest(k=None), rest(T=-1), save(c=cfg(dtype=5))):
        assert st == INVALID
    for st in (save(s=P1 + 8), save(k=P2 + 4), rest(g=P3 + 2), rest(b=P3 + 8), rest(s=P1 + 1)):
        assert st == UNSUPPORTED


def test_binding_refuses_wrong_tensors(L):
    """The Python calls check shapes, types, strides and devices before they call the library."""
    c = cfg()
    f = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t)
    ids = torch.zeros(4, dtype=torch.int64)
    bad = [lambda: H.embedding_fwd(f(3, 8), ids),                                           # not on a GPU
           lambda: H.embedding_fwd(f(3, 8), ids.to(torch.int16)),
           lambda: H.embedding_fwd(f(3, 8), torch.zeros(8, dtype=torch.int64)[::2]),
           lambda: H.embedding_fwd(f(3, 8, t=torch.float16), ids),
           lambda: H.embedding_fwd(f(8, 3).t(), ids),
           lambda: H.embedding_fwd(f(3, 8), ids, out=f(5, 8)),
           lambda: H.embedding_fwd(f(3, 8), ids, out=f(4, 8), low=f(4, 8)),
           lambda: H.embedding_bwd(f(5, 8), ids, f(3, 8)),
           lambda: H.embedding_bwd(f(4, 7), ids, f(3, 8)),
           lambda: H.embedding_bwd(f(4, 8), ids, f(3, 8, t=torch.bfloat16)),
           lambda: H.embedding_bwd_rows(f(4, 8), ids, 100, ids, f(3, 8), ids[:1]),
           lambda: H.embedding_bwd_rows(f(4, 8), ids, 100, ids.int(), f(4, 8), ids[:1]),
           lambda: H.block_norm_fwd(c, H.BlockNorm(post="batch"), f(4, 64), f(4, 64)),
           lambda: H.block_norm_fwd(c, H.BlockNorm(), f(4, 64), f(4, 64, t=torch.bfloat16)),
           lambda: H.block_norm_fwd(c, H.BlockNorm(post_gamma=f(64)), f(4, 64), f(4, 64)),
           lambda: H.block_norm_fwd(c, H.BlockNorm(), f(4, 64), f(4, 64), f(4, 64)),
           lambda: H.block_norm_bwd(c, H.BlockNorm(), None, f(4, 64), None, f(4, 4), dh=f(4, 64)),
           lambda: H.block_norm_bwd(c, H.BlockNorm(), f(4, 64), f(4, 64), None, f(4, 4), dgate=f(4, 64)),
           lambda: H.block_norm_bwd(c, H.BlockNorm(), f(4, 64), None, None, f(4, 4), db=f(4, 64)),
           lambda: H.checkpoint_save(c, 0, f(10, t=torch.uint8), 100, f(1 << 20, t=torch.uint8)),
           lambda: H.checkpoint_save(c, 0, f(1 << 22, t=torch.uint8), 100, f(10, t=torch.uint8)),
           lambda: H.checkpoint_restore(c, 0, f(1 << 20, t=torch.uint8), 100, f(64), None, f(1 << 22, t=torch.uint8))]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")


def test_joint_without_block_output():
    """Without b there is nothing to gate and no new y: a call that passes either is refused, not answered without it."""
    x = torch.zeros(4, 64)
    for kw in ({"gate": torch.zeros(4, 64, dtype=torch.bfloat16)}, {"y": torch.zeros(4, 64)}):
        with pytest.raises(ValueError, match="need b"):
            H.block_norm_fwd(cfg(), H.BlockNorm(), x, **kw)


def test_parameter_gradients_may_be_one_array_but_not_overlap(L):
    """Refused before any launch; the same array twice passes the checks as far as the workspace's."""
    c = cfg()
    bn = H.CBlockNorm(post_kind=1, pre_kind=2, gate_act=0)
    call = lambda **g: L.hstu_block_norm_bwd(ctypes.byref(c), ctypes.byref(bn), P1, P2, None, 0, P1, P2, P3, 4, P4, None, None, 0,
                                             ctypes.byref(H.CBlockNormGrads(**g)), WS, 0, None)
    assert call(post_gamma=P1, pre_gamma=P1 + 4) == INVALID
    assert call(pre_beta=P1, res_scale=P1 + 252) == INVALID
    assert call(post_gamma=P1, pre_gamma=P1) == WORKSPACE
    assert call(post_gamma=P1, pre_gamma=P1 + 256) == WORKSPACE

"""Cases of the operators around an HSTU stack's layers: the embedding lookup and its gradient, the norms before and
after a block with its gate and residual scale, and activation checkpoints in 8 bits.  Each has its plain form (elementary
torch operations), the library's call, and its definition in 64 bits."""
import functools
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-5


# ---------------------------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------------------------

def lookup(T, dim, V, *, width=0, table="f32", io="f32", low=True, ids="i64"):
    return {"op": "lookup", "T": T, "dim": dim, "V": V, "width": width or dim, "table": table, "io": io, "low": low and io == "f32", "ids": ids}


def grad(T, dim, V, *, width=0, io="f32", ids="i64", rows=False):
    return {"op": "grad_rows" if rows else "grad", "T": T, "dim": dim, "V": V, "width": width or dim, "io": io, "ids": ids}


def norms(T, d, *, dt="bf16", io="f32", post="layer", pre="layer", gate="silu", gate_cols=1, backward=False):
    return {"op": "norms_grad" if backward else "norms", "T": T, "d": d, "dt": dt, "io": io, "post": post, "pre": pre, "gate": gate, "gate_cols": gate_cols}


def checkpoint(T, d, *, dt="bf16", io="f32", fmt="int8"):
    return {"op": "checkpoint", "T": T, "d": d, "dt": dt, "io": io, "fmt": fmt}


def listed():
    return [
        # one request's microbatch of candidates: 16 users x 4 items, a bf16 table as served
        {"name": "lookup_request", **lookup(64, 512, 100_000, table="bf16")},
        # the training batch's rows (64 sequences, 287,928 events, d = 1,024) from an fp32 table, with the bf16 copy that the first layer reads
        {"name": "lookup_training_batch", **lookup(287_928, 1024, 200_000)},
        # the academic workload's table (3,706 items, 50 wide, rows of 64) and about as many events
        {"name": "lookup_grad_academic", **grad(14_001, 50, 3_706, width=64)},
        # the training batch's gradient: popular items repeat thousands of times
        {"name": "lookup_grad_training_batch", **grad(287_928, 1024, 200_000)},
        # a catalogue too large for a dense gradient: unique rows only, 32-bit ids, bf16 upstream gradient
        {"name": "lookup_grad_large_catalogue", **grad(131_071, 256, 20_000_000, io="bf16", ids="i32", rows=True)},
        # one token through the joint of two blocks
        {"name": "norms_single_token", **norms(1, 1024)},
        # 16 sequences of 8,192 tokens
        {"name": "norms_long_batch", **norms(131_072, 1024)},
        # fp32 layers with RMS norms and the gate taken from a wider projection, an odd number of tokens
        {"name": "norms_grad_rms_f32", **norms(10_007, 480, dt="f32", post="rms", pre="rms", gate="sigmoid", gate_cols=4, backward=True)},
        {"name": "norms_grad_long_batch", **norms(131_072, 1024, backward=True)},
        # the academic workload's size
        {"name": "checkpoint_academic", **checkpoint(14_001, 64)},
        # the long-history workload's width with a bf16 residual stream, in e4m3
        {"name": "checkpoint_long_history_e4m3", **checkpoint(40_003, 512, io="bf16", fmt="e4m3")},
        {"name": "checkpoint_long_batch", **checkpoint(131_072, 1024)},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["lookup", "grad", "grad_rows", "norms", "norms_grad", "checkpoint"])
    dt, io = rng.choice([("bf16", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
    if op in ("lookup", "grad", "grad_rows"):
        dim = rng.choice([spread(1, 1024), 2 * spread(4, 512), 64, 128, 256, 512, 1024])
        width = dim if rng.random() < 0.7 else dim + rng.randint(0, 64)
        T = spread(1, 131_072)
        V = spread(2, min(20_000_000, (200_000 * 1024) // dim))
        ids = rng.choice(["i64", "i64", "i32"])
        if op == "lookup":
            return lookup(T, dim, V, width=width, table=rng.choice(["f32", "bf16"]), io=io, low=rng.random() < 0.7, ids=ids)
        return grad(T, dim, V, width=width, io=io, ids=ids, rows=op == "grad_rows")
    head = rng.choice([32, 64, 128])
    d = head * rng.randint(1, min(16, 2048 // head))
    T = spread(1, 131_072 * 1024 // max(d, 1024))
    if op == "checkpoint":
        return checkpoint(T, d, dt=dt, io=io, fmt=rng.choice(["int8", "e4m3"]))
    return norms(T, d, dt=dt, io=io, post=rng.choice(["layer", "rms"]), pre=rng.choice(["layer", "rms"]), gate=rng.choice(["silu", "sigmoid", "none"]),
                 gate_cols=rng.choice([1, 4]), backward=op == "norms_grad")


# ---------------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------------

def normal(gen, shape, dtype, std=1.0, mean=0.0):
    x = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(mean, std, generator=gen)
    return x if dtype == torch.float32 else x.to(dtype)


def item_ids(gen, T, V, dtype):
    """Popularity k^-1.1 over the catalogue, popular items anywhere in it, one position in a hundred padding (-1)."""
    mass = torch.arange(1, V + 1, dtype=torch.float64, device="cuda").pow_(-1.1).cumsum_(0)
    u = torch.rand(T, dtype=torch.float64, device="cuda", generator=gen)
    rank = torch.searchsorted(mass, u * mass[-1]).clamp_(max=V - 1)
    step = next(p for p in (1_000_003, 7_368_787, 15_485_863) if V % p)
    ids = (rank * step) % V
    ids[torch.rand(T, device="cuda", generator=gen) < 0.01] = -1
    return ids.to(dtype)


def saved_offsets(c):
    """Where the parts of a layer's saved block lie: Pre, G, O, Z, mean, rstd and the operand copy of x, each on 256 bytes."""
    T, d, es = c["T"], c["d"], SIZE[c["dt"]]
    sizes = [("pre", T * 4 * d * es), ("g", T * 4 * d * es), ("o", T * d * 4), ("z", T * d * es), ("mean", T * 4), ("rstd", T * 4), ("xlow", T * d * es if c["io"] != c["dt"] else 0)]
    at, offs = 0, {}
    for name, n in sizes:
        offs[name] = (at, n)
        at = -(-(at + n) // 256) * 256
    return offs, at


def saved_views(c, block):
    offs, _ = saved_offsets(c)
    d, dt = c["d"], DT[c["dt"]]
    wide = {"pre": 4 * d, "g": 4 * d, "o": d, "z": d, "xlow": d}
    out = {}
    for name, (at, n) in offs.items():
        if n:
            v = block[at:at + n].view(torch.float32 if name in ("o", "mean", "rstd") else dt)
            out[name] = v.view(c["T"], wide[name]) if name in wide else v
    return out


def norm_params(gen, c):
    d, dt = c["d"], DT[c["dt"]]
    return {"post_gamma": normal(gen, d, dt, 0.1, 1.0), "post_beta": normal(gen, d, dt, 0.1) if c["post"] == "layer" else None, "res_scale": normal(gen, d, dt, 0.1, 0.5),
            "pre_gamma": normal(gen, d, dt, 0.1, 1.0), "pre_beta": normal(gen, d, dt, 0.1) if c["pre"] == "layer" else None}


GRADS = ("post_gamma", "post_beta", "res_scale", "pre_gamma", "pre_beta")


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    T = c["T"]
    if c["op"] in ("lookup", "grad", "grad_rows"):
        s["ids"] = item_ids(gen, T, c["V"], torch.int64 if c["ids"] == "i64" else torch.int32)
        io = DT[c["io"]]
        if c["op"] == "lookup":
            s["table"] = normal(gen, (c["V"], c["dim"]), DT[c["table"]], 0.02)
            s["out"] = torch.empty(T, c["width"], dtype=io, device="cuda")
            s["low"] = torch.empty(T, c["width"], dtype=torch.bfloat16, device="cuda") if c["low"] else None
        else:
            s["dx"] = normal(gen, (T, c["width"]), io)
            cap = min(T, c["V"])
            if c["op"] == "grad":
                s["dtable"] = torch.zeros(c["V"], c["dim"], device="cuda")
            else:
                s["rows"] = torch.zeros(cap, c["dim"], device="cuda")
                s["row_ids"] = torch.zeros(cap, dtype=torch.int64, device="cuda")
                s["count"] = torch.zeros(1, dtype=torch.int64, device="cuda")
        return s
    d, dt, io = c["d"], DT[c["dt"]], DT[c["io"]]
    if c["op"] == "checkpoint":
        offs, n = saved_offsets(c)
        s["saved"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
        s["back"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        v = saved_views(c, s["saved"])
        v["pre"].copy_(normal(gen, (T, 4 * d), dt))
        # rows of O have a mean several times their spread
        v["o"].copy_(normal(gen, (T, d), torch.float32, 0.05) + normal(gen, (T, 1), torch.float32, 0.1, 0.4))
        v["mean"].copy_(v["o"].mean(1))
        v["rstd"].copy_((v["o"].var(1, unbiased=False) + EPS).rsqrt())
        if "xlow" in v:
            v["xlow"].copy_(normal(gen, (T, d), dt))
        s["gamma"], s["beta"] = normal(gen, d, dt, 0.1, 1.0), normal(gen, d, dt, 0.1)
        return s
    s["x"] = normal(gen, (T, d), io)
    s["b"] = normal(gen, (T, d), io, 0.5, 0.1)
    wide = normal(gen, (T, d * c["gate_cols"]), dt) if c["gate"] != "none" else None
    s["gate"] = wide[:, :d] if wide is not None else None
    s["params"] = norm_params(gen, c)
    if c["op"] == "norms":
        s["y"], s["h"] = torch.empty(T, d, dtype=io, device="cuda"), torch.empty(T, d, dtype=dt, device="cuda")
        s["stats"] = torch.empty(T, 4, device="cuda")
        return s
    # what the forward left for the backward: y and each row's statistics
    y, stats = joint(c, s["params"], s["x"].float(), s["b"].float(), s["gate"])[:2]
    s["y"], s["stats"] = y.to(io), stats.float().contiguous()
    s["dy"], s["dh"] = normal(gen, (T, d), io), normal(gen, (T, d), io)
    s["dx"] = torch.empty(T, d, dtype=io, device="cuda")
    s["db"] = torch.empty(T, d, dtype=dt, device="cuda")
    s["dgate"] = torch.empty(T, d, dtype=dt, device="cuda") if wide is not None else None
    s["flat"] = torch.zeros(len(GRADS), d, device="cuda")
    s["grads"] = {n: s["flat"][i] for i, n in enumerate(GRADS) if s["params"][n] is not None}
    return s


# ---------------------------------------------------------------------------------------------------------------------
# Plain forms (32 bits)
# ---------------------------------------------------------------------------------------------------------------------

def plain_lookup(c, s):
    ids = s["ids"].long()
    fine = (ids >= 0) & (ids < c["V"])
    rows = s["table"][ids.clamp(0, c["V"] - 1)].float() * SCALE(c) * fine[:, None]
    if c["width"] > c["dim"]:
        rows = torch.cat([rows, rows.new_zeros(c["T"], c["width"] - c["dim"])], 1)
    return {"out": rows.to(DT[c["io"]]), "low": rows.to(torch.bfloat16) if c["low"] else None}


def SCALE(c):
    return float(np.float32(math.sqrt(c["dim"])))


def plain_grad(c, s):
    ids = s["ids"].long()
    fine = (ids >= 0) & (ids < c["V"])
    dx = s["dx"][:, :c["dim"]][fine].float()
    if c["op"] == "grad":
        s["dtable"].zero_()
        s["dtable"].index_add_(0, ids[fine], dx * SCALE(c))
        return {"dtable": s["dtable"]}
    uniq, where = torch.unique(ids[fine], sorted=True, return_inverse=True)
    n = uniq.numel()
    s["row_ids"][:n] = uniq
    s["rows"][:n] = torch.zeros(n, c["dim"], device="cuda").index_add_(0, where, dx) * SCALE(c)
    s["count"].fill_(n)
    return {"row_ids": s["row_ids"], "rows": s["rows"], "count": s["count"]}


def row_norm(kind, x):
    """(normalised rows, mean, 1 / spread)"""
    mean = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    x = x - mean
    r = 1.0 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
    return x * r, mean, r


def activate(kind, gate):
    """act(gate) and its derivative, in the gate's own precision."""
    if kind == "sigmoid":
        a = 1.0 / (1.0 + torch.exp(-gate))
        return a, a * (1.0 - a)
    if kind == "silu":
        a = 1.0 / (1.0 + torch.exp(-gate))
        return gate * a, a * (1.0 + gate * (1.0 - a))
    return gate, torch.ones_like(gate)


def affine(x, gamma, beta):
    x = x * gamma.to(x.dtype)
    return x if beta is None else x + beta.to(x.dtype)


def joint(c, p, x, b, gate):
    """y (rounded as it is stored), the rows' statistics and h, in the precision of x."""
    n, m1, r1 = row_norm(c["post"], b)
    v = affine(n, p["post_gamma"], p["post_beta"])
    if gate is not None:
        v = v * activate(c["gate"], gate.to(v.dtype))[0]
    y = (x + p["res_scale"].to(v.dtype) * v).to(DT[c["io"]]).to(x.dtype)
    n2, m2, r2 = row_norm(c["pre"], y)
    return y, torch.cat([m1, r1, m2, r2], 1), affine(n2, p["pre_gamma"], p["pre_beta"])


def plain_norms(c, s):
    y, stats, h = joint(c, s["params"], s["x"].float(), s["b"].float(), s["gate"])
    return {"y": y.to(DT[c["io"]]), "h": h.to(DT[c["dt"]]), "stats": stats}


def norm_backward(kind, n, r, dn):
    """Gradient of the rows before a norm from the one after it: n the normalised rows, r one over their spread."""
    g = dn - n * (dn * n).mean(1, keepdim=True)
    if kind == "layer":
        g = g - dn.mean(1, keepdim=True)
    return g * r


def plain_norms_grad(c, s):
    f = {k: s[k].float() for k in ("y", "b", "dy", "dh")}
    p, (m1, r1, m2, r2) = s["params"], s["stats"].split(1, 1)
    n2 = (f["y"] - m2) * r2
    dx = f["dy"] + norm_backward(c["pre"], n2, r2, f["dh"] * p["pre_gamma"].float())
    n1 = (f["b"] - m1) * r1
    v = affine(n1, p["post_gamma"], p["post_beta"])
    dv = dx * p["res_scale"].float()
    dgate = None
    act = 1.0
    if s["gate"] is not None:
        act, slope = activate(c["gate"], s["gate"].float())
        dgate = (dv * v * slope).to(DT[c["dt"]])
    dp = dv * act
    db = norm_backward(c["post"], n1, r1, dp * p["post_gamma"].float())
    sums = {"post_gamma": (dp * n1).sum(0), "post_beta": dp.sum(0), "res_scale": (dx * v * act).sum(0), "pre_gamma": (f["dh"] * n2).sum(0), "pre_beta": f["dh"].sum(0)}
    return {"dx": dx.to(DT[c["io"]]), "db": db.to(DT[c["dt"]]), "dgate": dgate, "grads": {n: sums[n] for n in s["grads"]}}


def pow2(e):
    """2^e in 32 bits for whole e in [-126, 127], exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def eight_bits(fmt, x):
    """The values that blocks of 32 stand for once they are held in 8 bits with a power of two as their scale: the smallest
    that keeps the block's largest value within the format's (127 whole steps, or e4m3's 448)."""
    t = x.reshape(x.shape[0], -1, 32)
    m, e = torch.frexp(t.abs().amax(2, keepdim=True))
    if fmt == "int8":
        e = torch.where(m <= 127 / 128, e - 7, e - 6).clamp(min=-126)
        return (torch.round(t * pow2(-e)) * pow2(e)).reshape(x.shape)
    e = torch.where(m <= 448 / 512, e - 9, e - 8).clamp(min=-126)
    t = t * pow2(-e)
    step = torch.frexp(t)[1].clamp(min=-5) - 4
    return (torch.round(t * pow2(-step)) * pow2(step) * pow2(e)).reshape(x.shape)


def plain_checkpoint(c, s):
    v, dt, d = saved_views(c, s["saved"]), DT[c["dt"]], c["d"]
    pre = eight_bits(c["fmt"], v["pre"].float())
    g = (pre / (1.0 + torch.exp(-pre))).to(dt)
    mean, rstd = v["mean"][:, None], v["rstd"][:, None]
    spread = eight_bits(c["fmt"], v["o"] - mean)
    z = affine(spread * rstd, s["gamma"], s["beta"]) * g[:, :d].float()
    out = {"pre": pre.to(dt), "g": g, "o": mean + spread, "z": z.to(dt), "mean": v["mean"].clone(), "rstd": v["rstd"].clone()}
    if "xlow" in v:
        out["xlow"] = eight_bits(c["fmt"], v["xlow"].float()).to(dt)
    return out


# ---------------------------------------------------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------------------------------------------------

@functools.lru_cache(maxsize=None)
def config(d, dt, io):
    from hstu_sequential_transducer_b200 import hstu as H
    return H.make_config(d, d // 32, 8192.0, H.HSTU_BF16 if dt == "bf16" else H.HSTU_F32, ln_eps=EPS, io_dtype=H.HSTU_BF16 if io == "bf16" else H.HSTU_F32)


def block_norm(H, c, s):
    """The module's parameters as the library takes them; made at the first call and kept, as a model keeps them."""
    if "bn" not in s:
        s["bn"] = H.BlockNorm(post=c["post"], pre=c["pre"], gate_act=c["gate"], **s["params"])
        if "grads" in s:
            s["bn_grads"] = H.BlockNormGrads(**s["grads"])
    return s["bn"]


def own_pass(c, s):
    from hstu_sequential_transducer_b200 import hstu as H
    if c["op"] == "lookup":
        H.embedding_fwd(s["table"], s["ids"], scale=SCALE(c), out=s["out"], low=s["low"])
        return {"out": s["out"], "low": s["low"]}
    if c["op"] == "grad":
        s["dtable"].zero_()
        H.embedding_bwd(s["dx"], s["ids"], s["dtable"], scale=SCALE(c))
        return {"dtable": s["dtable"]}
    if c["op"] == "grad_rows":
        H.embedding_bwd_rows(s["dx"], s["ids"], c["V"], s["row_ids"], s["rows"], s["count"], scale=SCALE(c))
        return {"row_ids": s["row_ids"], "rows": s["rows"], "count": s["count"]}
    cfg = config(c["d"], c["dt"], c["io"])
    if c["op"] == "norms":
        H.block_norm_fwd(cfg, block_norm(H, c, s), s["x"], s["b"], s["gate"], y=s["y"], h=s["h"], stats=s["stats"])
        return {"y": s["y"], "h": s["h"], "stats": s["stats"]}
    if c["op"] == "norms_grad":
        s["flat"].zero_()
        bn = block_norm(H, c, s)
        H.block_norm_bwd(cfg, bn, s["y"], s["b"], s["gate"], s["stats"], s["dy"], s["dh"], dx=s["dx"], db=s["db"], dgate=s["dgate"], grads=s["bn_grads"])
        return {"dx": s["dx"], "db": s["db"], "dgate": s["dgate"], "grads": s["grads"]}
    fmt = H.CKPT_INT8 if c["fmt"] == "int8" else H.CKPT_E4M3
    if "ckpt" not in s:
        s["ckpt"] = torch.empty(H.checkpoint_bytes(cfg, fmt, c["T"]), dtype=torch.uint8, device="cuda")
    H.checkpoint_save(cfg, fmt, s["saved"], c["T"], s["ckpt"])
    H.checkpoint_restore(cfg, fmt, s["ckpt"], c["T"], s["gamma"], s["beta"], s["back"])
    return saved_views(c, s["back"])


PLAIN = {"lookup": plain_lookup, "grad": plain_grad, "grad_rows": plain_grad, "norms": plain_norms, "norms_grad": plain_norms_grad, "checkpoint": plain_checkpoint}


def run(state):
    c = state["case"]
    return own_pass(c, state) if own else PLAIN[c["op"]](c, state)


# ---------------------------------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------------

def unique_items(c):
    """How many different items T draws meet, on average."""
    p = np.arange(1, c["V"] + 1, dtype=np.float64) ** -1.1
    p /= p.sum()
    return float(np.sum(-np.expm1(0.99 * c["T"] * np.log1p(-np.minimum(p, 1 - 1e-12)))))


def work(case):
    c = case
    T = c["T"]
    if c["op"] in ("lookup", "grad", "grad_rows"):
        ids, U, row = T * (8 if c["ids"] == "i64" else 4), unique_items(c), T * c["width"]
        if c["op"] == "lookup":
            return {"bytes": ids + U * c["dim"] * SIZE[c["table"]] + row * SIZE[c["io"]] + (row * 2 if c["low"] else 0), "flops": T * c["dim"]}
        rows = T * c["dim"] * SIZE[c["io"]]
        wrote = c["V"] * c["dim"] * 4 if c["op"] == "grad" else U * (c["dim"] * 4 + 8)
        return {"bytes": ids + rows + wrote, "flops": T * c["dim"]}
    d, es, io = c["d"], SIZE[c["dt"]], SIZE[c["io"]]
    gate = es if c["op"] != "checkpoint" and c["gate"] != "none" else 0
    if c["op"] == "norms":
        return {"bytes": T * (d * (2 * io + gate + io + es) + 16), "flops": 16 * T * d}
    if c["op"] == "norms_grad":
        return {"bytes": T * (d * (4 * io + gate + io + es + gate) + 16), "flops": 40 * T * d}
    x = es if c["io"] != c["dt"] else 0
    block = T * (d * (8 * es + 4 + es + x) + 8)
    return {"bytes": T * (d * (4 * es + 4 + x) + 8) + block, "flops": 30 * T * d}


# ---------------------------------------------------------------------------------------------------------------------
# Definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------------

def exact(case, seed):
    c = case
    s = prepare(c, seed)
    f8 = torch.float64
    T = c["T"]
    if c["op"] in ("lookup", "grad", "grad_rows"):
        ids, dim, scale = s["ids"].long(), c["dim"], SCALE(c)
        ok = ((ids >= 0) & (ids < c["V"])).nonzero().flatten()
        if c["op"] == "lookup":
            out = torch.zeros(T, c["width"], dtype=f8, device="cuda")
            out[ok, :dim] = scale * s["table"][ids[ok]].to(f8)
            return {"out": out, "low": out if c["low"] else None}
        order = ok[torch.sort(ids[ok], stable=True).indices]
        if c["op"] == "grad":
            dtable = torch.zeros(c["V"], dim, dtype=f8, device="cuda")
            dtable.index_put_((ids[order],), scale * s["dx"][order, :dim].to(f8), accumulate=True)
            return {"dtable": dtable}
        sorted_ids = ids[order]
        head = torch.ones_like(sorted_ids, dtype=torch.bool)
        head[1:] = sorted_ids[1:] != sorted_ids[:-1]
        n = int(head.sum())
        rows = torch.zeros(s["rows"].shape, dtype=f8, device="cuda")
        rows.index_put_((head.long().cumsum(0) - 1,), scale * s["dx"][order, :dim].to(f8), accumulate=True)
        row_ids = torch.zeros_like(s["row_ids"])
        row_ids[:n] = sorted_ids[head]
        return {"row_ids": row_ids, "rows": rows, "count": torch.tensor([n])}
    p = s.get("params", {})
    w = {n: (t.to(f8) if t is not None else None) for n, t in p.items()}

    def statistics(kind, x):
        mu = x.sum(1) / x.shape[1] if kind == "layer" else x.new_zeros(x.shape[0])
        return mu, ((x - mu[:, None]).pow(2).sum(1) / x.shape[1] + EPS).pow(-0.5)

    def scaled(n, gamma, beta):
        return n * gamma + (0.0 if beta is None else beta)

    def gated(kind, u):
        sg = torch.sigmoid(u)
        return {"silu": (u * sg, sg + u * sg * (1 - sg)), "sigmoid": (sg, sg * (1 - sg)), "none": (u, torch.ones_like(u))}[kind]

    if c["op"] == "norms":
        b, x = s["b"].to(f8), s["x"].to(f8)
        m1, r1 = statistics(c["post"], b)
        v = scaled((b - m1[:, None]) * r1[:, None], w["post_gamma"], w["post_beta"])
        del b
        if s["gate"] is not None:
            v = v * gated(c["gate"], s["gate"].to(f8))[0]
        y = x + w["res_scale"] * v
        del x, v
        # h is the norm of y as it is stored
        stored = y.to(DT[c["io"]]).to(f8)
        m2, r2 = statistics(c["pre"], stored)
        return {"y": y, "h": scaled((stored - m2[:, None]) * r2[:, None], w["pre_gamma"], w["pre_beta"]), "stats": torch.stack([m1, r1, m2, r2], 1)}
    if c["op"] == "norms_grad":
        m1, r1, m2, r2 = (t[:, None] for t in s["stats"].to(f8).unbind(1))
        d = c["d"]

        def back(kind, n, r, up):
            along = (up * n).sum(1, keepdim=True) / d
            level = up.sum(1, keepdim=True) / d if kind == "layer" else 0.0
            return r * (up - level - n * along)

        dh = s["dh"].to(f8)
        n2 = (s["y"].to(f8) - m2) * r2
        dx = s["dy"].to(f8) + back(c["pre"], n2, r2, dh * w["pre_gamma"])
        sums = {"pre_gamma": (dh * n2).sum(0), "pre_beta": dh.sum(0)}
        del dh, n2
        n1 = (s["b"].to(f8) - m1) * r1
        v = scaled(n1, w["post_gamma"], w["post_beta"])
        a, da = gated(c["gate"], s["gate"].to(f8)) if s["gate"] is not None else (1.0, None)
        dgate = dx * w["res_scale"] * v * da if da is not None else None
        del da
        sums["res_scale"] = (dx * v * a).sum(0)
        del v
        dp = dx * w["res_scale"] * a
        sums["post_beta"], sums["post_gamma"] = dp.sum(0), (dp * n1).sum(0)
        return {"dx": dx, "db": back(c["post"], n1, r1, dp * w["post_gamma"]), "dgate": dgate, "grads": {n: sums[n] for n in s["grads"]}}

    top, mantissa, lowest = {"int8": (127.0, None, None), "e4m3": (448.0, 3, -6)}[c["fmt"]]

    def power(k):
        return ((k.long() + 1023) << 52).view(f8)

    def held(x):
        """x, a part of the block, through 8 bits: per 32 values the smallest 2^k (k >= -126) with max |x| <= top * 2^k."""
        x = x.to(f8).view(x.shape[0], -1, 32)
        peak = x.abs().max(2, keepdim=True).values
        k = torch.ceil(torch.log2(peak / top)).clamp(-126, 127)
        # the logarithm is rounded: put right where it is off by one
        k = torch.where(power(k) * top < peak, k + 1, k)
        k = torch.where((power(k - 1) * top >= peak) & (k > -126), k - 1, k)
        q = x / power(k)
        if mantissa is None:
            q = torch.round(q)
        else:
            ulp = power((torch.frexp(q)[1] - 1).clamp(min=lowest) - mantissa)
            q = torch.round(q / ulp) * ulp
        return (q * power(k)).view(x.shape[0], -1)

    v, d = saved_views(c, s["saved"]), c["d"]
    mean, rstd = v["mean"].to(f8)[:, None], v["rstd"].to(f8)[:, None]
    out = {"pre": held(v["pre"]), "mean": v["mean"].to(f8), "rstd": v["rstd"].to(f8)}
    out["g"] = out["pre"] * torch.sigmoid(out["pre"])
    # the difference from the mean is taken, and held, in 32 bits
    dev = held((v["o"] - v["mean"][:, None]))
    out["o"] = mean + dev
    out["z"] = (dev * rstd * s["gamma"].to(f8) + s["beta"].to(f8)) * out["g"][:, :d].to(DT[c["dt"]]).to(f8)
    if "xlow" in v:
        out["xlow"] = held(v["xlow"])
    return out

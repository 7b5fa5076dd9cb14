"""Cases of the sequence-block operators: scaled lookup and its row gradient, the
root-mean-square norm with the residual's addition and its backward pass, and
jagged attention with its backward pass.

`run` computes a case either in plain form (elementary torch operations in 32
bits, rounded once at the end) or, where `own` is true, by the library's calls.
Sizes follow the repository's workloads: tables of 100K x 64 f32, 1M x 64 f32
and 10M x 128 bf16, UIH lengths lognormal (5, 1.2), (6, 1.4), (6.5, 1.5) and
(7, 1.6), up to 64 candidates a sample; model widths are generic.
"""
import math
import random

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "bf16": 2, "e4m3": 1}
EPS = 1e-6


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # one user's history scored alone: a few hundred IDs against a small table
        {"name": "lookup-one-user-f32", "op": "lookup", "T": 257, "R": 100_000, "D": 64, "table": "f32", "out": "f32"},
        # a rank's whole batch of the mid-size table
        {"name": "lookup-batch-bf16", "op": "lookup", "T": 2_000_033, "R": 10_000_000, "D": 128, "table": "bf16",
         "out": "bf16"},
        # the gradient of a few users' histories
        {"name": "grad-few-users-f32", "op": "grad", "T": 2_049, "R": 100_000, "D": 64, "dout": "f32", "grad": "f32"},
        # a rank's whole batch, hot rows repeated many thousand times
        {"name": "grad-batch-bf16", "op": "grad", "T": 2_000_033, "R": 10_000_000, "D": 128, "dout": "bf16",
         "grad": "f32"},
        # one user's rows into an 8-bit projection
        {"name": "norm-one-user-8bit", "op": "norm", "T": 257, "D": 256, "x": "bf16", "y": "e4m3", "res": True},
        # a rank's batch at the width of a mid-size block, 8-bit output
        {"name": "norm-batch-8bit", "op": "norm", "T": 400_003, "D": 512, "x": "bf16", "y": "e4m3", "res": True},
        # the embedding width in f32, a few samples
        {"name": "norm-bwd-few-f32", "op": "norm_bwd", "T": 515, "D": 64, "x": "f32", "res": True},
        {"name": "norm-bwd-batch-bf16", "op": "norm_bwd", "T": 400_003, "D": 512, "x": "bf16", "res": True},
        # a few short histories with candidates
        {"name": "attn-few-users", "op": "attn", "S": 8, "mu": 5.0, "sigma": 1.2, "lmax": 512, "cand": 8, "Hq": 4,
         "Hkv": 4, "Dh": 64, "causal": True},
        # long histories, shared key/value heads
        {"name": "attn-long-histories", "op": "attn", "S": 16, "mu": 7.0, "sigma": 1.6, "lmax": 4096, "cand": 64,
         "Hq": 8, "Hkv": 2, "Dh": 128, "causal": True},
        {"name": "attn-bwd-few-users", "op": "attn_bwd", "S": 8, "mu": 5.0, "sigma": 1.2, "lmax": 512, "cand": 8,
         "Hq": 4, "Hkv": 4, "Dh": 64, "causal": True},
        {"name": "attn-bwd-long-histories", "op": "attn_bwd", "S": 16, "mu": 6.5, "sigma": 1.5, "lmax": 4096,
         "cand": 32, "Hq": 8, "Hkv": 2, "Dh": 128, "causal": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lookup", "grad", "norm", "norm_bwd", "attn", "attn_bwd"])
    if op in ("lookup", "grad"):
        c = {"op": op, "T": _log(rng, 1, 2_000_000), "R": _log(rng, 1_000, 10_000_000), "D": rng.choice([32, 64, 128])}
        if op == "lookup":
            c["table"], c["out"] = rng.choice(["f32", "bf16"]), rng.choice(["f32", "bf16"])
        else:
            c["dout"], c["grad"] = rng.choice(["f32", "bf16"]), rng.choice(["f32", "bf16"])
        return c
    if op in ("norm", "norm_bwd"):
        D = 8 * _log(rng, 8, 256)
        c = {"op": op, "T": _log(rng, 1, 204_800_000 // (2 * D)), "D": D, "x": rng.choice(["f32", "bf16"]),
             "res": rng.random() < 0.7}
        if op == "norm":
            c["y"] = rng.choice([c["x"], "e4m3"])
        return c
    lmax = _log(rng, 32, 4096)
    Hkv = rng.choice([1, 2, 4])
    Hq = Hkv * rng.choice([1, 2, 4]) if Hkv < 4 else rng.choice([4, 8])
    causal = rng.random() < 0.8
    S = max(1, min(_log(rng, 1, 64), (16 if causal else 8) * 4096 * 4096 // (lmax * lmax)))
    return {"op": op, "S": S, "mu": round(rng.uniform(4.0, 7.0), 2), "sigma": round(rng.uniform(0.8, 1.6), 2),
            "lmax": lmax, "cand": rng.choice([0, 8, 32, 64]), "Hq": Hq, "Hkv": Hkv, "Dh": rng.choice([64, 128]),
            "causal": causal}


# ------------------------------------------------------------------- inputs

def _lengths(c):
    """UIH lengths and candidate counts of a case's samples (the case's own: every seed has the same sizes)."""
    r = random.Random("%(S)d %(mu)s %(sigma)s %(lmax)d %(cand)d" % c)
    uih = [min(c["lmax"] - c["cand"], max(0, round(r.lognormvariate(c["mu"], c["sigma"])))) if c["lmax"] > c["cand"]
           else r.randint(0, c["lmax"] // 2) for _ in range(c["S"])]
    uih[0] = max(1, c["lmax"] - c["cand"])  # the longest history is always there
    cand = [r.randint(1, c["cand"]) if c["cand"] else 0 for _ in range(c["S"])]
    if c["S"] > 2:
        uih[1], cand[1] = 0, 0  # a user without history
    cand = [min(b, max(0, c["lmax"] - a)) for a, b in zip(uih, cand)]
    return uih, cand


def _ids(T, R, g):
    """Zipf-like IDs (log-uniform ranks), scattered over the rows."""
    rank = torch.exp(torch.rand(T, generator=g, device="cuda", dtype=torch.float64) * math.log(R + 1)).long() - 1
    A = 0x9E3779B97F4A7C15 % R | 1
    while math.gcd(A, R) != 1:
        A += 1
    return rank.clamp_(0, R - 1) * A % R


def _normal(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = c["op"]
    s = {"c": c, "op": op, "err": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if op == "lookup":
        s["table"] = _normal(g, c["R"], c["D"], dtype=DT[c["table"]], std=0.01)
        s["ids"] = _ids(c["T"], c["R"], g)
        s["scale"] = math.sqrt(c["D"])
        s["out"] = torch.empty(c["T"], c["D"], dtype=DT[c["out"]], device="cuda")
    elif op == "grad":
        cap = min(c["T"], c["R"])
        s["ids"] = _ids(c["T"], c["R"], g)
        s["dout"] = _normal(g, c["T"], c["D"], dtype=DT[c["dout"]])
        s["scale"] = math.sqrt(c["D"])
        s["rows"] = torch.zeros(cap, dtype=torch.int64, device="cuda")
        s["grads"] = torch.zeros(cap, c["D"], dtype=DT[c["grad"]], device="cuda")
        s["count"] = torch.zeros(1, dtype=torch.int64, device="cuda")
    elif op in ("norm", "norm_bwd"):
        T, D, dt = c["T"], c["D"], DT[c["x"]]
        level = torch.exp(torch.randn(T, 1, generator=g, device="cuda"))  # rows of very different sizes
        s["gamma"] = 1 + 0.1 * _normal(g, D)
        if op == "norm":
            s["x"] = (_normal(g, T, D) * level).to(dt)
            s["res"] = (_normal(g, T, D) * level).to(dt) if c["res"] else None
            s["sum"] = torch.empty_like(s["x"]) if c["res"] else None
            s["y"] = torch.empty(T, D, dtype=DT[c["y"]], device="cuda")
            s["y_scale"] = torch.empty(T, dtype=torch.float32, device="cuda") if c["y"] == "e4m3" else None
            s["rstd"] = torch.empty(T, dtype=torch.float32, device="cuda")
        else:
            s["h"] = (_normal(g, T, D) * level).to(dt)
            s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS)
            s["dy"] = _normal(g, T, D, dtype=dt)
            s["dsum"] = _normal(g, T, D, dtype=dt) if c["res"] else None
            s["dh"] = torch.empty_like(s["h"])
            s["dgamma"] = torch.empty(D, dtype=torch.float32, device="cuda")
    else:
        uih, cand = _lengths(c)
        L = [a + b for a, b in zip(uih, cand)]
        T, Hq, Hkv, Dh = sum(L), c["Hq"], c["Hkv"], c["Dh"]
        s["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(L)]), dtype=torch.int64, device="cuda")
        s["cand"] = torch.tensor(cand, dtype=torch.int32, device="cuda") if c["cand"] else None
        s["lmax"], s["scale"] = max(L), 1.0 / math.sqrt(Dh)
        # one projection's output holds q, k and v side by side
        qkv = _normal(g, T, Hq + 2 * Hkv, Dh, dtype=torch.bfloat16)
        s["q"], s["k"], s["v"] = qkv.split([Hq, Hkv, Hkv], dim=1)
        s["out"] = torch.empty(T, Hq, Dh, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(Hq, T, dtype=torch.float32, device="cuda")
        if op == "attn_bwd":
            s["out"], s["lse"] = _plain_attn(s)
            s["dout"] = _normal(g, T, Hq, Dh, dtype=torch.bfloat16)
            dqkv = torch.empty(T, Hq + 2 * Hkv, Dh, dtype=torch.bfloat16, device="cuda")
            s["dq"], s["dk"], s["dv"] = dqkv.split([Hq, Hkv, Hkv], dim=1)
    return s


# ------------------------------------------------------------------- plain forms

def _plain_lookup(s):
    return (s["table"][s["ids"]].float() * s["scale"]).to(s["out"].dtype)


def _plain_grad(s):
    T, R = s["ids"].numel(), s["rows"].numel()
    key, order = torch.sort(s["ids"], stable=True)
    head = torch.ones(T, dtype=torch.bool, device="cuda")
    head[1:] = key[1:] != key[:-1]
    at = torch.cumsum(head, 0) - 1
    rows = torch.zeros(R, dtype=torch.int64, device="cuda")
    rows.scatter_(0, at, key)
    g = torch.zeros(R, s["dout"].shape[1], dtype=torch.float32, device="cuda")
    g.index_add_(0, at, s["dout"][order].float())
    return {"rows": rows, "grads": (g * s["scale"]).to(s["grads"].dtype), "count": (at[-1:] + 1)}


def _plain_norm(s):
    h = s["x"].float()
    out = {}
    if s["res"] is not None:
        out["sum"] = (h + s["res"].float()).to(s["x"].dtype)
        h = out["sum"].float()
    rstd = 1.0 / torch.sqrt((h * h).mean(1) + EPS)
    y = h * rstd[:, None] * s["gamma"]
    if s["y_scale"] is not None:
        scale = y.abs().amax(1) / 448.0
        out["y_scale"] = scale
        y = y / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None]
    out["y"], out["rstd"] = y.to(s["y"].dtype), rstd
    return out


def _plain_norm_bwd(s):
    n = s["h"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    w = dy * s["gamma"]
    dh = s["rstd"][:, None] * (w - n * (w * n).mean(1, keepdim=True))
    if s["dsum"] is not None:
        dh = dh + s["dsum"].float()
    return {"dh": dh.to(s["h"].dtype), "dgamma": (dy * n).sum(0)}


def _padded(s):
    """Places of the samples' rows in a padded [S, lmax] batch, and which keys a row sees."""
    off, lm = s["offsets"], s["lmax"]
    L = off[1:] - off[:-1]
    i = torch.arange(lm, device="cuda")
    idx = torch.minimum(off[:-1, None] + i, off[-1] - 1)
    ok = i < L[:, None]
    uih = L - s["cand"] if s["cand"] is not None else L
    see = (i[None, None, :] < uih[:, None, None]) | (i[None, :, None] == i[None, None, :])
    if s["c"]["causal"]:
        see = see & (i[None, None, :] <= i[None, :, None])
    see = see & ok[:, None, :]
    t = torch.arange(s["q"].shape[0], device="cuda")
    smp = torch.searchsorted(off, t, right=True) - 1
    return idx, see[:, None, None], smp * lm + (t - off[smp])


def _heads(x, idx, Hkv):
    """[T, H, Dh] -> [S, Hkv, H / Hkv, lmax, Dh] in 32 bits."""
    S, lm = idx.shape
    return x.float()[idx].view(S, lm, Hkv, -1, x.shape[2]).permute(0, 2, 3, 1, 4)


def _flat(x, at, H):
    """[S, Hkv, G, lmax, Dh] -> [T, H, Dh]."""
    return x.permute(0, 3, 1, 2, 4).reshape(-1, H, x.shape[-1])[at]


def _plain_probs(s, idx, see):
    Hkv = s["k"].shape[1]
    q, k = _heads(s["q"], idx, Hkv), _heads(s["k"], idx, Hkv)
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"]).masked_fill_(~see, -math.inf)
    m = x.amax(-1, keepdim=True).clamp_(min=-1e30)  # rows past a sample's end may see nothing
    p = x.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    return q, k, p.div_(z.clamp(min=1e-30)), (m + torch.log(z))[..., 0]


def _plain_attn(s):
    T, Hq, _ = s["q"].shape
    if T == 0:
        return s["out"], s["lse"]
    Hkv = s["k"].shape[1]
    idx, see, at = _padded(s)
    _, _, p, lse = _plain_probs(s, idx, see)
    o = torch.matmul(p, _heads(s["v"], idx, Hkv))
    lse = lse.permute(1, 2, 0, 3).reshape(Hq, -1)[:, at]
    return _flat(o, at, Hq).to(torch.bfloat16), lse


def _plain_attn_bwd(s):
    Hq, Hkv = s["q"].shape[1], s["k"].shape[1]
    idx, see, at = _padded(s)
    q, k, p, _ = _plain_probs(s, idx, see)
    ok = torch.zeros(idx.numel(), 1, device="cuda")
    ok[at] = 1.0
    do = _heads(s["dout"], idx, Hkv) * ok.view(idx.shape[0], 1, 1, idx.shape[1], 1)
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2, keepdim=True)
    ds = torch.matmul(do, _heads(s["v"], idx, Hkv).transpose(-1, -2))
    ds.sub_((ds * p).sum(-1, keepdim=True)).mul_(p)
    del p
    dq = torch.matmul(ds, k).mul_(s["scale"])
    dk = torch.matmul(ds.transpose(-1, -2), q).mul_(s["scale"]).sum(2, keepdim=True)
    return {"dq": _flat(dq, at, Hq).to(torch.bfloat16), "dk": _flat(dk, at, Hkv).to(torch.bfloat16),
            "dv": _flat(dv, at, Hkv).to(torch.bfloat16)}


# ------------------------------------------------------------------- one pass

def run(s):
    op = s["op"]
    if not own:
        if op == "attn":
            out, lse = _plain_attn(s)
            return {"out": out, "lse": lse}
        return {"lookup": _plain_lookup, "grad": _plain_grad, "norm": _plain_norm, "norm_bwd": _plain_norm_bwd,
                "attn_bwd": _plain_attn_bwd}[op](s)
    from jagged_embedding_gb300 import binding as B
    if op == "lookup":
        B.fs_emb_lookup_scaled(s["table"], s["ids"], s["scale"], out=s["out"], err=s["err"])
        return s["out"]
    if op == "grad":
        if "ws" not in s:  # a training loop keeps its workspace
            s["ws"] = B.workspace(B.emb_grad_rows_workspace_size(s["c"]["T"], s["c"]["R"], s["c"]["D"]), "cuda")
        B.fs_emb_grad_rows(s["ids"], s["dout"], s["c"]["R"], s["scale"], rows=s["rows"], row_grads=s["grads"],
                           count=s["count"], err=s["err"], ws=s["ws"])
        return {"rows": s["rows"], "grads": s["grads"], "count": s["count"]}
    if op == "norm":
        B.fs_rmsnorm(s["x"], s["gamma"], EPS, res=s["res"], sum_out=s["sum"], y=s["y"], y_scale=s["y_scale"],
                     rstd=s["rstd"])
        return {k: s[k] for k in ("sum", "y", "y_scale", "rstd") if s[k] is not None}
    if op == "norm_bwd":
        if "ws" not in s:
            s["ws"] = B.workspace(B.rmsnorm_backward_workspace_size(s["c"]["T"], s["c"]["D"]), "cuda")
        B.fs_rmsnorm_backward(s["dy"], s["h"], s["gamma"], s["rstd"], dsum=s["dsum"], dh=s["dh"],
                              dgamma=s["dgamma"], ws=s["ws"])
        return {"dh": s["dh"], "dgamma": s["dgamma"]}
    causal = s["c"]["causal"]
    if "ws" not in s:
        T, Hq, Dh = s["q"].shape
        s["ws"] = B.workspace(B.jagged_attn_workspace_size(T, s["c"]["S"], Hq, s["k"].shape[1], Dh), "cuda")
    if op == "attn":
        B.fs_jagged_attn(s["q"], s["k"], s["v"], s["offsets"], s["scale"], causal=causal, cand_len=s["cand"],
                         out=s["out"], lse=s["lse"], err=s["err"], ws=s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    B.fs_jagged_attn_backward(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], s["offsets"], s["scale"],
                              causal=causal, cand_len=s["cand"], dq=s["dq"], dk=s["dk"], dv=s["dv"], err=s["err"],
                              ws=s["ws"])
    return {"dq": s["dq"], "dk": s["dk"], "dv": s["dv"]}


# ------------------------------------------------------------------- work and exact values

def _distinct(T, R):
    """Expected distinct rows among T log-uniform ranks of [0, R)."""
    edge = np.unique(np.concatenate([np.arange(1, min(R, 4096) + 1), np.geomspace(1, R + 1, 4096)]).astype(np.float64))
    lo, hi = edge[:-1], edge[1:]
    n = hi - lo  # rows of a stretch, each about as likely
    p = np.log(hi / lo) / math.log(R + 1) / n
    return float(np.sum(n * -np.expm1(T * np.log1p(-np.minimum(p, 0.999)))))


def _pairs(c):
    """Visible (row, key) pairs of one head."""
    n = 0
    for u, b in zip(*_lengths(c)):
        n += (u * (u + 1) // 2 if c["causal"] else u * u) + b * (u + 1)
    return n


def work(c):
    op = c["op"]
    if op == "lookup":
        b = c["T"] * (8 + c["D"] * SIZE[c["out"]]) + _distinct(c["T"], c["R"]) * c["D"] * SIZE[c["table"]]
        return {"bytes": b, "flops": c["T"] * c["D"]}
    if op == "grad":
        b = c["T"] * (8 + c["D"] * SIZE[c["dout"]]) + _distinct(c["T"], c["R"]) * (8 + c["D"] * SIZE[c["grad"]])
        return {"bytes": b, "flops": c["T"] * c["D"]}
    if op == "norm":
        per = c["D"] * (SIZE[c["x"]] * (3 if c["res"] else 1) + SIZE[c["y"]]) + 4 + (4 if c["y"] == "e4m3" else 0)
        return {"bytes": c["T"] * per + 4 * c["D"], "flops": 5 * c["T"] * c["D"]}
    if op == "norm_bwd":
        return {"bytes": c["T"] * (c["D"] * SIZE[c["x"]] * (4 if c["res"] else 3) + 4) + 8 * c["D"],
                "flops": 9 * c["T"] * c["D"]}
    T = sum(map(sum, _lengths(c)))
    rows = T * c["Dh"] * 2
    if op == "attn":
        return {"bytes": rows * 2 * (c["Hq"] + c["Hkv"]) + 4 * T * c["Hq"], "flops": 4 * c["Dh"] * c["Hq"] * _pairs(c)}
    return {"bytes": rows * (4 * c["Hq"] + 4 * c["Hkv"]) + 4 * T * c["Hq"], "flops": 10 * c["Dh"] * c["Hq"] * _pairs(c)}


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    f8 = torch.float64
    if op == "lookup":
        return torch.index_select(s["table"], 0, s["ids"]).to(f8) * s["scale"]
    if op == "grad":
        uniq, inv = torch.unique(s["ids"], return_inverse=True)
        n = uniq.numel()
        rows, g = torch.zeros_like(s["rows"]), torch.zeros(s["grads"].shape, dtype=f8, device="cuda")
        rows[:n] = uniq
        order = torch.argsort(inv)
        total = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), torch.bincount(inv, minlength=n).cumsum(0)])
        for a in range(0, c["D"], 32):  # a running sum in 64 bits, cut at the rows' ends
            run_ = s["dout"][order, a:a + 32].to(f8).cumsum(0)
            run_ = torch.cat([torch.zeros(1, run_.shape[1], dtype=f8, device="cuda"), run_])
            g[:n, a:a + 32] = (run_[total[1:]] - run_[total[:-1]]) * s["scale"]
        return {"rows": rows, "grads": g, "count": torch.tensor([n], device="cuda")}
    if op == "norm":
        h, out = s["x"].to(f8), {}
        if s["res"] is not None:
            out["sum"] = h + s["res"].to(f8)
            h = out["sum"].to(s["x"].dtype).to(f8)  # the sum is normed as it is stored
        out["rstd"] = (torch.linalg.vector_norm(h, dim=1) ** 2 / c["D"] + EPS) ** -0.5
        y = torch.einsum("td,t,d->td", h, out["rstd"], s["gamma"].to(f8))
        if s["y_scale"] is not None:
            out["y_scale"] = torch.linalg.vector_norm(y, ord=math.inf, dim=1) / 448
            y = y / out["y_scale"].clamp(min=1e-300)[:, None]
        out["y"] = y
        return out
    if op == "norm_bwd":
        h, r, dy, gm = s["h"].to(f8), s["rstd"].to(f8), s["dy"].to(f8), s["gamma"].to(f8)
        dot = torch.einsum("td,td,d->t", h, dy, gm)
        dh = torch.einsum("t,td,d->td", r, dy, gm) - h * (r ** 3 * dot / c["D"])[:, None]
        return {"dh": dh if s["dsum"] is None else dh + s["dsum"].to(f8), "dgamma": torch.einsum("t,td,td->d", r, h, dy)}
    return _exact_attn(c, s)


def _exact_attn(c, s):
    if c["Dh"] * c["Hq"] * sum((u + b) ** 2 for u, b in zip(*_lengths(c))) > 2e11:
        return None
    f8, Hq, Hkv = torch.float64, c["Hq"], c["Hkv"]
    names = ("out",) if c["op"] == "attn" else ("dq", "dk", "dv")
    r = {n: torch.zeros(s["q"].shape if n in ("out", "dq") else s["k"].shape, dtype=f8, device="cuda") for n in names}
    if c["op"] == "attn":
        r["lse"] = torch.zeros(s["lse"].shape, dtype=f8, device="cuda")
    a = 0
    for u, b in zip(*_lengths(c)):
        n = u + b
        w = torch.ones(n, n, dtype=torch.bool, device="cuda")
        w[:, u:] = False
        w |= torch.eye(n, dtype=torch.bool, device="cuda")
        w = w.tril() if c["causal"] else w
        for h in range(Hq if n else 0):
            z = slice(a, a + n)
            q, k, v = s["q"][z, h].to(f8), s["k"][z, h * Hkv // Hq].to(f8), s["v"][z, h * Hkv // Hq].to(f8)
            x = torch.where(w, q @ k.T * s["scale"], -math.inf)
            lse = torch.logsumexp(x, 1)
            p = torch.exp(x - lse[:, None])
            if c["op"] == "attn":
                r["out"][z, h], r["lse"][h, z] = p @ v, lse
                continue
            do = s["dout"][z, h].to(f8)
            dp = do @ v.T
            ds = p * (dp - (do * (p @ v)).sum(1, keepdim=True)) * s["scale"]
            r["dq"][z, h] = ds @ k
            r["dk"][z, h * Hkv // Hq] += ds.T @ q
            r["dv"][z, h * Hkv // Hq] += p.T @ do
        a += n
    return r

"""Workloads of the layer's norm and of the router's training side.

Four operators, as a trainer or a server runs them around the routed-expert
layer: the RMS norm with the residual's addition and an 8-bit output, its
backward (from the 16-bit sum or from the 8-bit checkpoint), the balance loss
with the experts' counts and its gradient, and the router's backward (top-k
softmax and the two products, from 16-bit tokens or from the checkpoint).

`own` false: `run` computes them in elementary torch operations.  `own` true:
through moe_routed_expert_router_amd.  Shapes: hidden size 4096, 384 experts,
6 picks, 1 / 32 / 8192 tokens are the layer's own workloads (decode, batched
decode, prefill); the others stand for odd and ragged batches.
"""
import math

import torch

own = False

EPS = 1e-6
ALPHA = 0.01
F32, BF16 = "f32", "bf16"
DT = {F32: torch.float32, BF16: torch.bfloat16}


# ------------------------------- the cases ---------------------------------
def _norm(name, T, H, x=BF16, res=BF16, q="none"):
    return {"name": name, "op": "norm", "T": T, "H": H, "x": x, "res": res, "q": q}


def _norm_bwd(name, T, H, src, dy=BF16, dres=BF16, dx=BF16):
    return {"name": name, "op": "norm_bwd", "T": T, "H": H, "src": src, "dy": dy, "dres": dres, "dx": dx}


def _balance(name, T, E, k, seqs=0, masked=False):
    return {"name": name, "op": "balance", "T": T, "E": E, "k": k, "seqs": seqs, "masked": masked}


def _route_bwd(name, T, H, E, k, src, renorm, dz_in, dx=BF16):
    return {"name": name, "op": "route_bwd", "T": T, "H": H, "E": E, "k": k, "src": src, "renorm": renorm,
            "dz_in": dz_in, "dx": dx}


def listed():
    return [
        # one decode token's pre-norm: latency
        _norm("norm_decode1", 1, 4096),
        # a batched decode step whose next product takes 8-bit tokens
        _norm("norm_decode32_q", 32, 4096, q="out"),
        # a prefill / training batch that keeps the 8-bit checkpoint
        _norm("norm_8k_ckpt", 8192, 4096, q="norm"),
        # fp32 layer output added to an fp32 residual stream, odd batch and width
        _norm("norm_f32_1031", 1031, 1408, x=F32, res=F32, q="out"),
        # training batch, backward from the stored sum
        _norm_bwd("norm_bwd_8k", 8192, 4096, "h"),
        # odd batch, backward from the 8-bit checkpoint, fp32 gradients
        _norm_bwd("norm_bwd_ckpt_777", 777, 2176, "ckpt", dy=F32, dres=F32, dx=F32),
        # loss and gradient of one small step
        _balance("balance_32", 32, 384, 6),
        # the whole training batch as one group
        _balance("balance_8k", 8192, 384, 6),
        # packed sequences of uneven length with padding, odd expert count
        _balance("balance_seqs_5003", 5003, 257, 8, seqs=17, masked=True),
        # router backward of a small step
        _route_bwd("route_bwd_32", 32, 4096, 384, 6, "x", True, True),
        # router backward of a training batch
        _route_bwd("route_bwd_8k", 8192, 4096, 384, 6, "x", True, True),
        # odd batch from the 8-bit checkpoint, softmax over all experts, fp32 dx
        _route_bwd("route_bwd_ckpt_2051", 2051, 4096, 384, 6, "ckpt", False, True, dx=F32),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    T = _log_int(rng, 1, 8191)
    H = 128 * _log_int(rng, 1, 32)
    E = _log_int(rng, 8, 384)
    k = rng.randint(1, min(8, E))
    ty = lambda: rng.choice((F32, BF16))  # noqa: E731
    op = rng.choice(("norm", "norm_bwd", "balance", "route_bwd"))
    if op == "norm":
        c = _norm("", T, H, ty(), ty(), rng.choice(("none", "out", "norm")))
    elif op == "norm_bwd":
        c = _norm_bwd("", T, H, rng.choice(("h", "ckpt")), ty(), ty(), ty())
    elif op == "balance":
        c = _balance("", T, E, k, rng.choice((0, 0, _log_int(rng, 1, 64))), rng.random() < 0.5)
    else:
        c = _route_bwd("", T, H, E, k, rng.choice(("x", "ckpt")), rng.random() < 0.5, rng.random() < 0.5, ty())
    del c["name"]
    return c


# ------------------------------- the inputs --------------------------------
def _e4m3(v):
    """Values of |v| <= 448 rounded to e4m3 (half to even), in v's type."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6)))
    e = torch.where(torch.ldexp(torch.ones_like(v), e + 1) <= v.abs(), e + 1, e).clamp_min(-6)
    step = torch.ldexp(torch.ones_like(v), e - 3)
    return torch.round(v / step) * step


def _quantise(v):
    """(e4m3 codes, e8m0 scales) of rows in blocks of 32: the least power of
    two that brings the block's largest magnitude to 448 or below."""
    T, H = v.shape
    b = v.view(T, H // 32, 32)
    amax = b.abs().amax(2)
    e = torch.floor(torch.log2(amax.clamp_min(2.0 ** -140))) - 8
    e = torch.where(amax > 448 * torch.ldexp(torch.ones_like(amax), e), e + 1, e)
    e = torch.where(amax > 448 * torch.ldexp(torch.ones_like(amax), e), e + 1, e)
    e = e.clamp(-127, 127)
    q = _e4m3(torch.ldexp(b, -e[:, :, None])).view(T, H)
    return q.float().to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _values(codes, scales):
    T, H = codes.shape
    s = torch.ldexp(torch.ones_like(scales, dtype=torch.float32), scales.float() - 127)
    return (codes.float().view(T, H // 32, 32) * s[:, :, None]).view(T, H)


def _rnd(g, shape, dev, scale=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device=dev) * scale).to(dtype)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    T, op = case["T"], case["op"]
    st = {"case": case}
    if op == "norm":
        H = case["H"]
        st["x"] = _rnd(g, (T, H), dev, 0.5, DT[case["x"]])
        st["res"] = _rnd(g, (T, H), dev, 2.0, DT[case["res"]])
        st["weight"] = 1 + _rnd(g, (H,), dev, 0.1)
        st["res_out"] = torch.empty_like(st["res"])
        st["y"] = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
        st["rstd"] = torch.empty(T, device=dev)
        if case["q"] != "none":
            st["codes"] = torch.empty((T, H), dtype=torch.uint8, device=dev)
            st["scales"] = torch.empty((T, H // 32), dtype=torch.uint8, device=dev)
    elif op == "norm_bwd":
        H = case["H"]
        h = _rnd(g, (T, H), dev, 2.0, DT[case["dres"]])
        st["rstd"] = (h.float().square().mean(1) + EPS).rsqrt()
        st["weight"] = 1 + _rnd(g, (H,), dev, 0.1)
        st["dy"] = _rnd(g, (T, H), dev, 1e-3, DT[case["dy"]])
        st["dres"] = _rnd(g, (T, H), dev, 1e-3, DT[case["dres"]])
        if case["src"] == "h":
            st["h"] = h
        else:
            st["codes"], st["scales"] = _quantise(h.float() * st["rstd"][:, None])
        st["dx"] = torch.empty((T, H), dtype=DT[case["dx"]], device=dev)
        st["dweight"] = torch.empty(H, device=dev)
    elif op == "balance":
        _routing(st, case, g, dev)
        E, S = case["E"], max(1, case["seqs"])
        st["offsets"] = st["mask"] = None
        if case["seqs"]:
            # cut points in the first nineteen twentieths: a padded tail, uneven and empty sequences
            cuts = torch.randint(0, T - T // 20 + 1, (S,), generator=g, device=dev).sort().values
            st["offsets"] = torch.cat([torch.zeros(1, device=dev), cuts]).int()
        if case["masked"]:
            st["mask"] = (torch.rand(T, generator=g, device=dev) > 0.1).to(torch.uint8)
        st["dloss"] = torch.ones(1, device=dev)
        st["loss"] = torch.empty(1, device=dev)
        st["counts"] = torch.empty((S, E), dtype=torch.int32, device=dev)
        st["n_valid"] = torch.empty(S + 1, dtype=torch.int32, device=dev)
        st["prob_mean"] = torch.empty((S, E), device=dev)
        st["dlogits"] = torch.empty((T, E), device=dev)
    else:
        _routing(st, case, g, dev)
        H, E, k = case["H"], case["E"], case["k"]
        x = _rnd(g, (T, H), dev, 1.0)
        if case["src"] == "x":
            st["x"] = x.bfloat16()
        else:
            st["codes"], st["scales"] = _quantise(x)
            st["weight"] = 1 + _rnd(g, (H,), dev, 0.1)
        st["wr"] = _rnd(g, (E, H), dev, H ** -0.5)
        st["dw"] = _rnd(g, (T, k), dev, 1e-2)
        st["dz_in"] = _rnd(g, (T, E), dev, 1e-4) if case["dz_in"] else None
        st["dx"] = torch.empty((T, H), dtype=DT[case["dx"]], device=dev)
        st["dwr"] = torch.empty((E, H), device=dev)
        st["db"] = torch.empty(E, device=dev)
    return st


def _routing(st, case, g, dev):
    """Logits with a Zipf-like prior over the experts, the picks and weights."""
    T, E, k = case["T"], case["E"], case["k"]
    rank = torch.randperm(E, generator=g, device=dev).float()
    st["z"] = _rnd(g, (T, E), dev, 1.0) - 0.5 * torch.log1p(rank)
    top = torch.topk(st["z"], k, dim=1)
    st["ids"] = top.indices.int()
    p = torch.softmax(top.values if case.get("renorm", True) else st["z"], 1)
    st["topw"] = p if case.get("renorm", True) else p.gather(1, top.indices)


# ------------------------------ the plain forms ----------------------------
def _plain_norm(st, case):
    wide = torch.float64 if case["q"] != "none" else torch.float32   # a rounding border decides a code
    h = (st["x"].float() + st["res"].float()).to(st["res"].dtype)
    hw = h.to(wide)
    r = 1 / torch.sqrt(hw.square().mean(1, keepdim=True) + EPS)
    n = hw * r
    y = n * st["weight"].to(wide)
    out = {"res_out": h, "y": y.to(torch.bfloat16), "rstd": r[:, 0].float()}
    if case["q"] != "none":
        codes, scales = _quantise(y if case["q"] == "out" else n)
        out["codes"], out["scales"] = codes, scales.view(torch.float8_e8m0fnu)
    return out


def _plain_norm_bwd(st, case):
    H = case["H"]
    r = st["rstd"][:, None]
    n = st["h"].float() * r if case["src"] == "h" else _values(st["codes"], st["scales"])
    dy = st["dy"].float()
    gw = dy * st["weight"]
    dh = r * (gw - n * ((gw * n).sum(1, keepdim=True) / H)) + st["dres"].float()
    return {"dx": dh.to(st["dx"].dtype), "dweight": (dy * n).sum(0)}


def _groups(st, case):
    """Group of each token, -1 for one that belongs to none."""
    T, S = case["T"], max(1, case["seqs"])
    t = torch.arange(T, device=st["z"].device)
    gid = torch.zeros_like(t)
    if st["offsets"] is not None:
        gid = (t[:, None] >= st["offsets"][None, 1:]).sum(1)
        gid = torch.where((t < st["offsets"][0]) | (gid >= S), -1, gid)
    if st["mask"] is not None:
        gid = torch.where(st["mask"] != 0, gid, -1)
    return gid, S


def _plain_balance(st, case):
    E, k = case["E"], case["k"]
    gid, S = _groups(st, case)
    ok = gid >= 0
    at = torch.where(ok, gid, S)   # row S collects the tokens of no group
    z = st["z"]
    p = torch.exp(z - z.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True)
    psum = torch.zeros((S + 1, E), device=z.device).index_add_(0, at, p)[:S]
    n = torch.zeros(S + 1, dtype=torch.int32, device=z.device).index_add_(0, at, torch.ones_like(at).int())[:S]
    flat = (at[:, None] * E + st["ids"]).reshape(-1)
    counts = torch.zeros((S + 1) * E, dtype=torch.int32, device=z.device)
    counts = counts.index_add_(0, flat, torch.ones_like(flat).int()).view(S + 1, E)[:S]
    live = (n > 0).sum().int()
    nn = n.clamp_min(1).float()[:, None]
    mean = psum / nn
    f = counts.float() * E / (k * nn)
    loss = ALPHA * (f * mean).sum() / live.clamp_min(1)
    a = st["dloss"] * ALPHA * f / (nn * live.clamp_min(1))
    at_t = a[gid.clamp_min(0)]
    dz = p * (at_t - (p * at_t).sum(1, keepdim=True))
    dz = torch.where(ok[:, None], dz, torch.zeros_like(dz))
    return {"loss": loss.view(1), "counts": counts, "n_valid": torch.cat([n, live.view(1)]), "prob_mean": mean,
            "dlogits": dz}


def _plain_route_bwd(st, case):
    z, w, dw = st["z"], st["topw"], st["dw"]
    ids = st["ids"].long()
    dot = (w * dw).sum(1, keepdim=True)
    if case["renorm"]:
        dz = torch.zeros_like(z).scatter_add_(1, ids, w * (dw - dot))
    else:
        p = torch.exp(z - z.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
        dz = p * (torch.zeros_like(z).scatter_add_(1, ids, dw) - dot)
    if st["dz_in"] is not None:
        dz = dz + st["dz_in"]
    x = st["x"].float() if case["src"] == "x" else _values(st["codes"], st["scales"]) * st["weight"]
    return {"dx": (dz @ st["wr"]).to(st["dx"].dtype), "dwr": dz.t() @ x, "db": dz.sum(0)}


# --------------------------- the framework's calls --------------------------
def _handle(st, case):
    """What a user's program keeps: the layer's shape and a workspace."""
    if "shape" not in st:
        import moe_routed_expert_router_amd as moe
        st["moe"] = moe
        st["shape"] = moe.shape(case.get("H", 128), 128, case.get("E", 8), case.get("k", 1))
        n = moe.moe_train_workspace_bytes(st["shape"], case["T"], max(1, case.get("seqs", 0)))
        st["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return st["moe"], st["shape"], st["ws"]


def _own_norm(st, case):
    moe, s, _ = _handle(st, case)
    kind = {"none": moe.MOE_Q_NONE, "out": moe.MOE_Q_OUTPUT, "norm": moe.MOE_Q_NORMALIZED}[case["q"]]
    codes, scales = st.get("codes"), st.get("scales")
    moe.moe_rms_norm(s, st["x"], st["res"], st["weight"], EPS, st["res_out"], st["y"], kind, codes, scales,
                     st["rstd"])
    out = {"res_out": st["res_out"], "y": st["y"], "rstd": st["rstd"]}
    if codes is not None:
        out["codes"], out["scales"] = codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)
    return out


def _own_norm_bwd(st, case):
    moe, s, ws = _handle(st, case)
    moe.moe_rms_norm_backward(s, st["dy"], st["dres"], st.get("h"), st.get("codes"), st.get("scales"), st["rstd"],
                              st["weight"], None, st["dx"], st["dweight"], ws)
    return {"dx": st["dx"], "dweight": st["dweight"]}


def _own_balance(st, case):
    moe, s, ws = _handle(st, case)
    moe.moe_balance_loss(s, st["z"], st["ids"], st["mask"], st["offsets"], ALPHA, st["loss"], st["counts"],
                         st["n_valid"], st["prob_mean"], ws)
    moe.moe_balance_loss_backward(s, st["z"], st["mask"], st["offsets"], ALPHA, st["dloss"], st["counts"],
                                  st["n_valid"], st["dlogits"])
    return {n: st[n] for n in ("loss", "counts", "n_valid", "prob_mean", "dlogits")}


def _own_route_bwd(st, case):
    moe, s, ws = _handle(st, case)
    moe.moe_route_backward(s, st.get("x"), st.get("codes"), st.get("scales"), st.get("weight"), st["wr"],
                           case["renorm"], st["z"], st["ids"], st["topw"], st["dw"], st["dz_in"], None,
                           st["dx"], st["dwr"], st["db"], ws)
    return {"dx": st["dx"], "dwr": st["dwr"], "db": st["db"]}


PLAIN = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "balance": _plain_balance, "route_bwd": _plain_route_bwd}
OWN = {"norm": _own_norm, "norm_bwd": _own_norm_bwd, "balance": _own_balance, "route_bwd": _own_route_bwd}


def run(state):
    case = state["case"]
    return (OWN if own else PLAIN)[case["op"]](state, case)


# ----------------------------- the 64-bit values ----------------------------
def exact(case, seed):
    """The operators' definitions in 64 bits."""
    st = prepare(case, seed)
    d = lambda n: st[n].to(torch.float64)  # noqa: E731
    if case["op"] == "norm":
        h = (d("x") + d("res")).to(torch.float32).to(st["res"].dtype)
        hd = h.double()
        r = (torch.linalg.vector_norm(hd, dim=1).pow(2) / case["H"] + EPS).pow(-0.5)
        y = torch.einsum("th,t,h->th", hd, r, d("weight"))
        out = {"res_out": hd, "y": y, "rstd": r}
        if case["q"] != "none":
            out["codes"], out["scales"] = _mx_by_table(y if case["q"] == "out" else hd * r[:, None])
        return out
    if case["op"] == "norm_bwd":
        r = d("rstd")[:, None]
        n = d("h") * r if case["src"] == "h" else _mx_values(st["codes"], st["scales"])
        dn = d("dy") * d("weight")
        proj = torch.matmul(dn.unsqueeze(1), n.unsqueeze(2)).squeeze(2) / case["H"]
        return {"dx": d("dres") + r * dn - r * proj * n, "dweight": torch.einsum("th,th->h", d("dy"), n)}
    logp = torch.log_softmax(d("z"), 1)
    if case["op"] == "balance":
        T, E, k, S = case["T"], case["E"], case["k"], max(1, case["seqs"])
        off = [0, T] if st["offsets"] is None else st["offsets"].tolist()
        keep = torch.ones(T, dtype=torch.bool, device="cuda") if st["mask"] is None else st["mask"].bool()
        z = d("z").requires_grad_()
        p = torch.softmax(z, 1)
        n, counts, mean, losses = [], [], [], []
        for i in range(S):
            m = keep[off[i]:off[i + 1]]
            ids, pp = st["ids"][off[i]:off[i + 1]][m], p[off[i]:off[i + 1]][m]
            n.append(len(ids))
            counts.append(torch.bincount(ids.reshape(-1).long(), minlength=E))
            mean.append(pp.mean(0) if n[-1] else pp.sum(0))
            losses.append((counts[-1].double() / max(n[-1], 1) * E / k * mean[-1]).sum())
        live = sum(v > 0 for v in n)
        loss = ALPHA * sum(losses) / max(live, 1)
        dz, = torch.autograd.grad(loss, z)
        return {"loss": loss.detach().view(1), "counts": torch.stack(counts).int(),
                "n_valid": torch.tensor(n + [live], dtype=torch.int32, device="cuda"),
                "prob_mean": torch.stack(mean).detach(), "dlogits": dz}
    E = case["E"]
    if case["renorm"]:
        soft = d("topw")
        jac = torch.diag_embed(soft) - soft[:, :, None] * soft[:, None, :]
        u = (jac @ d("dw")[:, :, None])[:, :, 0]
        dz = torch.zeros((case["T"], E), dtype=torch.float64, device="cuda")
        dz.scatter_add_(1, st["ids"].long(), u)
    else:
        p = logp.exp()
        pick = torch.zeros_like(p).scatter_add_(1, st["ids"].long(), d("dw"))
        dz = p * pick - p * (d("topw") * d("dw")).sum(1, keepdim=True)
    if st["dz_in"] is not None:
        dz += d("dz_in")
    x = d("x") if case["src"] == "x" else _mx_values(st["codes"], st["scales"]) * d("weight")
    return {"dx": dz @ d("wr"), "dwr": (x.t() @ dz).t().contiguous(), "db": dz.sum(0)}


def _mx_values(codes, scales):
    e = torch.repeat_interleave(scales.double() - 127, 32, 1)
    return codes.to(torch.float64) * torch.pow(torch.full_like(e, 2.0), e)


def _mx_by_table(v):
    """Codes (as the values they stand for) and scales of v by a search in the
    table of e4m3's values: the nearest, an even code where two are as near."""
    bits = torch.arange(127, device=v.device)
    ex, man = bits // 8, bits % 8
    table = torch.where(ex == 0, man.double() * 2.0 ** -9, (8 + man).double() * torch.pow(2.0, ex.double() - 10))
    b = v.reshape(v.shape[0], -1, 32)
    top = b.abs().amax(2)
    grid = torch.pow(torch.full((255,), 2.0, dtype=torch.float64, device=v.device),
                     torch.arange(-127, 128, device=v.device).double())
    s = torch.searchsorted(448 * grid, top).clamp(max=254)
    u = b.abs() / grid[s][:, :, None]
    hi = torch.searchsorted(table, u.reshape(-1)).clamp(1, 126).view(u.shape)
    lo = hi - 1
    dl, dh = u - table[lo], table[hi] - u
    c = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    q = torch.copysign(table[c], b).view(v.shape)
    return q, grid[s]


def work(case):
    T, op = case["T"], case["op"]
    size = {F32: 4, BF16: 2}
    if op == "norm":
        n = T * case["H"]
        b = n * (size[case["x"]] + 2 * size[case["res"]] + 2 + (33 / 32 if case["q"] != "none" else 0))
        return {"bytes": b + 4 * (T + case["H"]), "flops": 6 * n}
    if op == "norm_bwd":
        n = T * case["H"]
        b = n * (size[case["dy"]] + size[case["dres"]] + size[case["dx"]]
                 + (size[case["dres"]] if case["src"] == "h" else 33 / 32))
        return {"bytes": b + 4 * (T + 2 * case["H"]), "flops": 12 * n}
    E, k = case["E"], case["k"]
    if op == "balance":
        S = max(1, case["seqs"])
        b = 4 * T * (2 * E + k) + 8 * S * E + (T if case["masked"] else 0) + 4 * S
        return {"bytes": b, "flops": 12 * T * E}
    H = case["H"]
    b = T * H * (2 if case["src"] == "x" else 33 / 32) + 8 * E * H + 12 * T * k + T * H * size[case["dx"]] + 4 * E
    b += 4 * T * E * ((not case["renorm"]) + bool(case["dz_in"]))
    return {"bytes": b, "flops": 4 * T * H * E}

"""The norm and the router's training side on the GPU against the float64 oracle.

Tolerances are sums of rounding bounds, written beside their use: U = 2^-24 is
half a step of fp32, UB = 2^-8 of bf16 (relative to the value); a sum of n
terms added in any order is off by at most n U times the sum of magnitudes.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_routed_expert_router_amd as moe  # noqa: E402
from oracle import train as ot  # noqa: E402

U, UB = 2.0 ** -24, 2.0 ** -8
EPS = 1e-6
F32, B16 = torch.float32, torch.bfloat16


def f64(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def rnd(seed, shape, scale=1.0, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def new_ws(s, T, n_seq=1):
    return torch.empty(moe.moe_train_workspace_bytes(s, T, n_seq), dtype=torch.uint8, device="cuda").fill_(0xA5)


def close(got, want, bound):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    bad = np.abs(got - want)[ok] > np.broadcast_to(bound, want.shape)[ok]
    worst = np.max(np.abs(got - want)[ok] / np.maximum(np.broadcast_to(bound, want.shape)[ok], 1e-300), initial=0.0)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside, worst {worst:.3g} x the bound"


# --------------------------------- norm ------------------------------------
class Norm:
    def __init__(self, T, H, xt, rt, kind, res=True, seed=0, x=None):
        self.s = moe.shape(H, 128, 8, 2)
        self.x = rnd(seed, (T, H), 0.7, xt) if x is None else x
        self.res = rnd(seed + 1, (T, H), 2.0, rt) if res else None
        self.w = 1 + rnd(seed + 2, (H,), 0.2)
        self.ro = torch.full((T, H), 7.0, dtype=rt, device="cuda")
        self.y = torch.full((T, H), 7.0, dtype=B16, device="cuda")
        self.r = torch.full((T,), 7.0, device="cuda")
        self.kind = kind
        q = kind != moe.MOE_Q_NONE
        self.c = torch.full((T, H), 9, dtype=torch.uint8, device="cuda") if q else None
        self.sc = torch.full((T, H // 32), 9, dtype=torch.uint8, device="cuda") if q else None

    def run(self, stream=None, eps=EPS):
        moe.moe_rms_norm(self.s, self.x, self.res, self.w, eps, self.ro, self.y, self.kind, self.c, self.sc, self.r,
                         stream)

    def check(self, eps=EPS):
        torch.cuda.synchronize()
        h, r, n, y = ot.rms_norm(f64(self.x), f64(self.res), f64(self.w), float(np.float32(eps)),
                                 self.ro.dtype == B16, True)
        assert np.array_equal(f64(self.ro), h)
        close(self.r, r, np.abs(r) * (U + 1e-12))
        # r, h r, weight: three fp32 roundings, then the store
        close(self.y, y, np.abs(y) * (UB + 4 * U))
        if self.c is not None:
            c, sc = ot.mx8_encode(y if self.kind == moe.MOE_Q_OUTPUT else n)
            assert np.array_equal(self.sc.cpu().numpy(), sc)
            assert np.array_equal(self.c.cpu().numpy(), c)


@pytest.mark.parametrize("kind", [moe.MOE_Q_NONE, moe.MOE_Q_OUTPUT, moe.MOE_Q_NORMALIZED])
@pytest.mark.parametrize("T,H", [(1, 4096), (3, 128), (5, 1152), (2, 2176), (7, 640), (9, 1024), (2, 16384), (1, 16512),
                                 (2, 65536)])
@pytest.mark.parametrize("xt,rt", [(B16, B16), (F32, F32), (F32, B16), (B16, F32)])
def test_norm(T, H, xt, rt, kind):
    c = Norm(T, H, xt, rt, kind, seed=T + H)
    c.run()
    c.check()


@pytest.mark.parametrize("kind", [moe.MOE_Q_NONE, moe.MOE_Q_OUTPUT])
def test_norm_without_residual(kind):
    c = Norm(4, 384, F32, B16, kind, res=False)
    c.run()   # residual_out given: h rounded to its type
    c.check()
    y = torch.empty_like(c.y)
    moe.moe_rms_norm(c.s, c.x, None, c.w, EPS, None, y)   # neither: h = x as it is
    torch.cuda.synchronize()
    _, _, _, want = ot.rms_norm(f64(c.x), None, f64(c.w), float(np.float32(EPS)), False, False)
    close(y, want, np.abs(want) * (UB + 4 * U))


def test_norm_in_place():
    a, b = Norm(9, 512, B16, B16, moe.MOE_Q_NORMALIZED), Norm(9, 512, B16, B16, moe.MOE_Q_NORMALIZED)
    a.run()
    b.ro, b.y = b.res, b.x
    b.run()
    torch.cuda.synchronize()
    for n in ("ro", "y", "c", "sc", "r"):
        assert torch.equal(getattr(a, n), getattr(b, n)), n


def test_norm_magnitudes():
    """Squares beyond fp32's range, tiny rows, zero rows, non-finite rows."""
    H = 256
    x = rnd(5, (6, H), 1.0, B16)
    x[0] *= 2.0 ** 120
    x[1] *= 2.0 ** -120
    x[2] = 0
    x[3, 7] = float("inf")
    x[4, 9] = float("nan")
    c = Norm(6, H, B16, B16, moe.MOE_Q_OUTPUT, res=False, x=x)
    c.run()
    torch.cuda.synchronize()
    got = f64(c.y)
    with np.errstate(all="ignore"):
        h, r, n, y = ot.rms_norm(f64(x), None, f64(c.w), float(np.float32(EPS)), True, True)
        codes, sc = ot.mx8_encode(y)
    close(c.y, y, np.abs(y) * (UB + 4 * U) + 2.0 ** -133)
    assert np.array_equal(c.sc.cpu().numpy(), sc)
    rows = [0, 2, 5]   # row 1: values near fp32's least, row 3, 4: non-finite
    assert np.array_equal(c.c.cpu().numpy()[rows], codes[rows])
    assert np.isnan(got[3, 7]) and np.all(np.isnan(got[4])) and np.all(got[2] == 0)
    assert np.all(np.isnan(ot.mx8_decode(c.c.cpu().numpy(), c.sc.cpu().numpy())[4]))


# ----------------------------- norm backward --------------------------------
@pytest.mark.parametrize("src", ["h16", "h32", "ckpt"])
@pytest.mark.parametrize("T,H", [(1, 4096), (5, 1152), (700, 256), (1300, 128), (3, 16512), (513, 2176)])
@pytest.mark.parametrize("dyt,drt,dxt", [(B16, B16, B16), (F32, None, F32), (F32, B16, F32), (B16, F32, B16)])
def test_norm_backward(T, H, src, dyt, drt, dxt):
    s = moe.shape(H, 128, 8, 2)
    w = 1 + rnd(1, (H,), 0.2)
    dy = rnd(2, (T, H), 1e-2, dyt)
    dres = None if drt is None else rnd(3, (T, H), 1e-2, drt)
    h = codes = sc = None
    x = rnd(4, (T, H), 1.5, F32 if src == "h32" else B16)
    r = (x.float().square().mean(1) + EPS).rsqrt()
    if src == "ckpt":
        codes = torch.empty((T, H), dtype=torch.uint8, device="cuda")
        sc = torch.empty((T, H // 32), dtype=torch.uint8, device="cuda")
        moe.moe_rms_norm(s, x, None, w, EPS, None, None, moe.MOE_Q_NORMALIZED, codes, sc, r)
        torch.cuda.synchronize()
        n = ot.mx8_decode(codes.cpu().numpy(), sc.cpu().numpy())
    else:
        h = x
        n = f64(h) * f64(r)[:, None]
    mask = None
    if T > 4:
        mask = torch.ones(T, dtype=torch.uint8, device="cuda")
        mask[T // 2] = mask[T - 1] = 0
        dy[T // 2] = float("nan")
        if h is not None:
            h[T - 1] = float("inf")
    dx = torch.full((T, H), 7.0, dtype=dxt, device="cuda")
    dwt = torch.full((H,), 7.0, device="cuda")
    moe.moe_rms_norm_backward(s, dy, dres, h, codes, sc, r, w, mask, dx, dwt, new_ws(s, T))
    torch.cuda.synchronize()
    m = None if mask is None else mask.cpu().numpy()
    wx, ww = ot.rms_norm_backward(f64(dy), f64(dres), n, f64(r), f64(w), m)
    keep = np.ones(T, bool) if m is None else m.astype(bool)
    g, nn = np.abs(np.where(keep[:, None], f64(dy), 0) * f64(w)), np.abs(np.where(keep[:, None], n, 0))
    S = (g * nn).sum(1, keepdims=True)
    # a lane adds at most 64 terms, then 6 levels of the wave and 16 waves;
    # n, g, their product: 3 roundings; mean, product, difference, sum: 4
    gam = (64 + 6 + 16 + 3) * U
    b = f64(r)[:, None] * (6 * U * (g + nn * S / H) + nn * S / H * gam)
    b = b + 2 * U * np.abs(wx) + (0 if dres is None else U * np.abs(np.where(keep[:, None], f64(dres), 0)))
    close(dx, wx, b + (UB if dxt == B16 else U) * (np.abs(wx) + b))
    # ceil(T / 512) terms in a block, 64 rows in a chain, 3 levels; 2 per term
    A = (np.abs(np.where(keep[:, None], f64(dy), 0)) * nn).sum(0)
    close(dwt, ww, (-(-T // 512) + 64 + 3 + 2) * U * A)


def test_norm_backward_parts_and_in_place():
    """dx alone, dweight alone and dx over dy give the same bits as together."""
    T, H = 40, 768
    s = moe.shape(H, 128, 8, 2)
    w, dy, dres, h = 1 + rnd(1, (H,), 0.2), rnd(2, (T, H)), rnd(3, (T, H)), rnd(4, (T, H))
    r = (h.square().mean(1) + EPS).rsqrt()
    ws = new_ws(s, T)
    dx, dw = torch.empty_like(dy), torch.empty(H, device="cuda")
    moe.moe_rms_norm_backward(s, dy, dres, h, None, None, r, w, None, dx, dw, ws)
    dx1, dw1 = torch.empty_like(dy), torch.empty(H, device="cuda")
    moe.moe_rms_norm_backward(s, dy, dres, h, None, None, r, w, None, dx1, None, ws)
    moe.moe_rms_norm_backward(s, dy, dres, h, None, None, r, w, None, None, dw1, ws)
    for t in (dy, dres, h):
        u = {id(q): q.clone() for q in (dy, dres, h)}
        a, b, c = u[id(dy)], u[id(dres)], u[id(h)]
        moe.moe_rms_norm_backward(s, a, b, c, None, None, r, w, None, u[id(t)], dw1, ws)
        torch.cuda.synchronize()
        assert torch.equal(u[id(t)], dx) and torch.equal(dw1, dw)
    assert torch.equal(dx1, dx)


# ------------------------------- balance ------------------------------------
def routing(seed, T, E, k, neg=False):
    z = rnd(seed, (T, E)) - 0.5 * torch.log1p(torch.arange(E, device="cuda").float())
    if neg and T > 2:
        z[:, E // 2] = float("-inf")
        z[1] = float("-inf")
    ids = torch.topk(z, k, dim=1).indices.int()
    return z, ids


def balance(s, z, ids, mask, off, alpha, dloss=None, ws=None):
    T, E = z.shape
    S = 1 if off is None else off.numel() - 1
    o = {"loss": torch.full((1,), 7.0, device="cuda"), "counts": torch.full((S, E), -1, dtype=torch.int32, device="cuda"),
         "n_valid": torch.full((S + 1,), -1, dtype=torch.int32, device="cuda"),
         "prob_mean": torch.full((S, E), 7.0, device="cuda"), "dlogits": torch.full((T, E), 7.0, device="cuda")}
    moe.moe_balance_loss(s, z, ids, mask, off, alpha, o["loss"], o["counts"], o["n_valid"], o["prob_mean"],
                         new_ws(s, T, S) if ws is None else ws)
    moe.moe_balance_loss_backward(s, z, mask, off, alpha, dloss, o["counts"], o["n_valid"], o["dlogits"])
    return o


def check_balance(o, z, ids, mask, off, alpha, k, up=1.0):
    torch.cuda.synchronize()
    E = z.shape[1]
    zz, m = f64(z), None if mask is None else mask.cpu().numpy()
    ref = ot.balance_loss(zz, ids.cpu().numpy(), E, k, alpha, m, None if off is None else off.cpu().numpy())
    assert np.array_equal(o["counts"].cpu().numpy(), ref["counts"])
    assert np.array_equal(o["n_valid"].cpu().numpy(), ref["n_valid"])
    fin = zz[np.isfinite(zz)]
    D = fin.max() - fin.min() if fin.size else 0.0
    # a probability: exp of a rounded difference (D U) and expf's own two
    # steps, the same in the sum, 16 + 8 terms to add, reciprocal, product
    p = (2 * D + 40) * U
    # chunk: up to 128 terms per wave, 3 levels; then up to 128 chunks in a chain, 3 levels; division
    close(o["prob_mean"], ref["prob_mean"], ref["prob_mean"] * (p + 264 * U) + 1e-38)
    close(o["loss"], np.array([ref["loss"]]), abs(ref["loss"]) * (p + 270 * U))
    with np.errstate(all="ignore"):
        pr = ot.softmax(zz)
    off_l = [0, len(zz)] if off is None else off.tolist()
    a = np.zeros_like(zz)
    for g in range(len(off_l) - 1):
        n, live = ref["n_valid"][g], ref["n_valid"][-1]
        if n:
            a[off_l[g]:off_l[g + 1]] = alpha * up / live / n * ref["counts"][g] * E / (k * n)
    scale = pr * (np.abs(a) + (pr * np.abs(a)).sum(1, keepdims=True))
    close(o["dlogits"], ref["dlogits"] * up, scale * (2 * p + 40 * U) + 1e-38)


@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (4, 8, 2), (32, 384, 6), (33, 257, 8), (100, 1, 1), (129, 1024, 32),
                                   (2000, 65, 3), (257, 384, 6)])
def test_balance(T, E, k):
    s = moe.shape(128, 128, E, k)
    z, ids = routing(T + E, T, E, k, neg=E > 8)
    check_balance(balance(s, z, ids, None, None, 0.02), z, ids, None, None, 0.02, k)


@pytest.mark.parametrize("cuts", [[0, 5, 5, 40, 77], [3, 3, 64, 70], [0, 1, 2, 3, 4], [80, 80], [0, 0, 0], [31, 32, 33, 96, 100]])
@pytest.mark.parametrize("masked", [False, True])
def test_balance_sequences(cuts, masked):
    T, E, k = 100, 70, 4
    s = moe.shape(128, 128, E, k)
    z, ids = routing(9, T, E, k, neg=True)
    ids[7, 1] = ids[7, 0]           # listed twice: counted twice
    ids[8, 0], ids[9, 2] = -1, E    # outside [0, E): not counted
    mask = None
    if masked:
        mask = (rnd(3, (T,)) > 0).to(torch.uint8)
        mask[10] = 0
        z[10] = float("nan")        # masked: no part in anything
        mask[64:70] = 0
    off = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    dloss = torch.tensor([2.5], device="cuda")
    o = balance(s, z, ids, mask, off, 0.05, dloss)
    torch.cuda.synchronize()
    rows = [t for t in range(T) if t < cuts[0] or t >= cuts[-1] or (mask is not None and not mask[t])]
    assert torch.all(o["dlogits"][rows] == 0)
    if masked:
        z = torch.where(torch.isnan(z), torch.zeros_like(z), z)
    check_balance(o, z, ids, mask, off, 0.05, k, 2.5)


def test_balance_many_sequences_and_bool_mask():
    T, E, k = 3000, 40, 2
    s = moe.shape(128, 128, E, k)
    z, ids = routing(1, T, E, k)
    off = torch.cat([torch.zeros(1), torch.randint(0, T, (899,), generator=torch.Generator().manual_seed(1)).sort().values,
                     torch.tensor([T])]).int().cuda()
    mask = rnd(2, (T,)) > -1
    check_balance(balance(s, z, ids, mask, off, 0.01), z, ids, mask, off, 0.01, k)


def test_balance_bad_offsets_stay_inside():
    """Offsets that decrease or leave [0, T] give some numbers, from inside the arrays only."""
    T, E, k = 64, 16, 2
    s = moe.shape(128, 128, E, k)
    z, ids = routing(1, T, E, k)
    for cuts in ([0, 500, 10, -7, 64], [1 << 30, -(1 << 30), 5], [60, 40, 20, 0]):
        o = balance(s, z, ids, None, torch.tensor(cuts, dtype=torch.int32, device="cuda"), 0.01)
        torch.cuda.synchronize()
        assert torch.all(o["counts"] >= 0) and torch.all(torch.isfinite(o["dlogits"]))


@pytest.mark.parametrize("T", [20, 200])
def test_balance_nonfinite_rows(T):
    """NaN and +inf reach the loss, their sequence's means and their own rows;
    -inf is a probability of 0 and a row of nothing else counts as a token."""
    E, k = 70, 3
    s = moe.shape(128, 128, E, k)
    for bad in (float("nan"), float("inf")):
        z, ids = routing(4, T, E, k)
        z[3, 5] = bad
        off = torch.tensor([0, T // 2, T], dtype=torch.int32, device="cuda")
        for o in (None, off):
            r = balance(s, z, ids, None, o, 0.1)
            torch.cuda.synchronize()
            assert torch.isnan(r["loss"]).all() and torch.isnan(r["prob_mean"][0]).all()
            assert torch.isnan(r["dlogits"][3]).all()
            assert torch.isfinite(r["dlogits"][4:]).all() and torch.isfinite(r["prob_mean"][1:]).all()
            assert r["counts"].sum().item() == T * k
    z = torch.full((T, E), float("-inf"), device="cuda")
    r = balance(s, z, ids, None, None, 0.1)
    torch.cuda.synchronize()
    assert r["loss"].item() == 0 and torch.all(r["dlogits"] == 0) and r["n_valid"].tolist() == [T, 1]


@pytest.mark.parametrize("E", [40, 257, 1024])
@pytest.mark.parametrize("T", [300, 1000])
def test_balance_one_group_in_parts(T, E):
    """One group added up by several blocks: non-finite parts from any of
    them, the largest sum there is (every pick the same expert, probability
    1), and the same workspace call after call."""
    k = 32
    s = moe.shape(128, 128, E, k)
    z, ids = routing(9, T, E, k)
    ws = new_ws(s, T)
    ws.fill_(0xFF)
    good = balance(s, z, ids, None, None, 0.1, ws=ws)
    check_balance(good, z, ids, None, None, 0.1, k)
    for bad in (float("nan"), float("inf")):
        for e in (0, E - 1):
            y = z.clone()
            y[T - 2, e] = bad
            r = balance(s, y, ids, None, None, 0.1, ws=ws)
            torch.cuda.synchronize()
            assert torch.isnan(r["loss"]).all() and r["n_valid"].tolist() == [T, 1]
            assert torch.equal(r["counts"], good["counts"])
    y = torch.zeros((T, E), device="cuda")
    y[:, E - 1] = 200.0   # the others' exp is 0
    r = balance(s, y, torch.full_like(ids, E - 1), None, None, 0.25, ws=ws)
    torch.cuda.synchronize()
    assert r["loss"].item() == 0.25 * E and r["counts"][0, E - 1].item() == T * k
    again = balance(s, z, ids, None, None, 0.1, ws=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(good[n], again[n]) for n in good)


def test_balance_in_place():
    s = moe.shape(128, 128, 40, 3)
    z, ids = routing(2, 300, 40, 3)
    o = balance(s, z, ids, None, None, 0.1)
    dz = z.clone()
    moe.moe_balance_loss_backward(s, dz, None, None, 0.1, None, o["counts"], o["n_valid"], dz)
    torch.cuda.synchronize()
    assert torch.equal(dz, o["dlogits"])


def test_balance_empty():
    s = moe.shape(128, 128, 8, 2)
    z, ids = torch.empty((0, 8), device="cuda"), torch.empty((0, 2), dtype=torch.int32, device="cuda")
    o = balance(s, z, ids, None, None, 0.5)
    torch.cuda.synchronize()
    assert o["loss"].item() == 0 and torch.all(o["counts"] == 0) and o["n_valid"].tolist() == [0, 0]
    z, ids = routing(1, 6, 8, 2)
    o = balance(s, z, ids, torch.zeros(6, dtype=torch.uint8, device="cuda"), None, 0.5)
    torch.cuda.synchronize()
    assert o["loss"].item() == 0 and torch.all(o["dlogits"] == 0) and o["n_valid"].tolist() == [0, 0]


# ---------------------------- router backward -------------------------------
class Route:
    def __init__(self, T, H, E, k, src="x", renorm=True, dw=True, dz=True, mask=False, dxt=B16, seed=0):
        self.T, self.H, self.E, self.k, self.renorm = T, H, E, k, renorm
        self.s = moe.shape(H, 128, E, k)
        self.z, self.ids = routing(seed, T, E, k)
        top = self.z.gather(1, self.ids.long())
        self.w = torch.softmax(top, 1) if renorm else torch.softmax(self.z, 1).gather(1, self.ids.long())
        self.dw = rnd(seed + 1, (T, k), 0.1) if dw else None
        self.dz = rnd(seed + 2, (T, E), 0.01) if dz else None
        self.wr = rnd(seed + 3, (E, H), H ** -0.5)
        self.x = self.c = self.sc = self.qw = None
        x = rnd(seed + 4, (T, H), 1.0, B16)
        if src == "x":
            self.x, self.xv = x, f64(x)
        else:
            kind = moe.MOE_Q_OUTPUT if src == "q_out" else moe.MOE_Q_NORMALIZED
            self.c = torch.empty((T, H), dtype=torch.uint8, device="cuda")
            self.sc = torch.empty((T, H // 32), dtype=torch.uint8, device="cuda")
            w = 1 + rnd(seed + 5, (H,), 0.2)
            moe.moe_rms_norm(self.s, x, None, w, EPS, None, None, kind, self.c, self.sc)
            self.qw = None if src == "q_out" else w
            torch.cuda.synchronize()
            self.xv = ot.mx8_decode(self.c.cpu().numpy(), self.sc.cpu().numpy())
            if self.qw is not None:
                self.xv = self.xv * f64(w)
        self.mask = None
        if mask:
            self.mask = (rnd(seed + 6, (T,)) > -0.5).to(torch.uint8)
            self.mask[T - 1] = 0
            if self.x is not None:
                self.x[T - 1] = float("nan")
                self.xv = np.where(np.isnan(self.xv), 0, self.xv)
                self.xv[T - 1] = 0
            if self.dw is not None:
                self.dw[T - 1] = float("nan")
        self.dx = torch.full((T, H), 7.0, dtype=dxt, device="cuda")
        self.dwr = torch.full((E, H), 7.0, device="cuda")
        self.db = torch.full((E,), 7.0, device="cuda")
        self.ws = new_ws(self.s, T)

    def run(self, stream=None, dx=True, dwr=True, db=True):
        moe.moe_route_backward(self.s, self.x, self.c, self.sc, self.qw, self.wr, self.renorm, self.z, self.ids, self.w,
                               self.dw, self.dz, self.mask, self.dx if dx else None, self.dwr if dwr else None,
                               self.db if db else None, self.ws, stream)

    def check(self):
        torch.cuda.synchronize()
        T, E, k = self.T, self.E, self.k
        m = None if self.mask is None else self.mask.cpu().numpy()
        ids = self.ids.cpu().numpy()
        dz = ot.route_dlogits(f64(self.z), ids, f64(self.w), f64(self.dw), self.renorm, f64(self.dz), E, m)
        keep = np.ones(T, bool) if m is None else m.astype(bool)
        # bound of dz's error: magnitudes of the terms times their roundings
        # (dot over k picks, products, the k + 1 additions into one logit)
        err = np.zeros((T, E))
        if self.dw is not None:
            w, d = np.abs(f64(self.w)), np.abs(np.where(keep[:, None], f64(self.dw), 0))
            ok = (ids >= 0) & (ids < E)
            d = np.where(ok, d, 0)
            dot = (w * d).sum(1, keepdims=True)
            if self.renorm:
                t, j = np.nonzero(ok)
                np.add.at(err, (t, ids[t, j]), (w * (d + dot))[t, j] * (k + 12) * U)
            else:
                z = f64(self.z)
                D = z.max() - z.min()
                g = np.repeat(dot, E, 1)
                t, j = np.nonzero(ok)
                np.add.at(g, (t, ids[t, j]), d[t, j])
                err += ot.softmax(z) * g * (2 * D + 40 + k + 12) * U
        if self.dz is not None:
            err += 2 * U * np.abs(f64(self.dz))
        err = np.where(keep[:, None], err + 2 * U * np.abs(dz), 0)
        wx, ww, wb = ot.route_backward(dz, np.where(keep[:, None], self.xv, 0), f64(self.wr), m)
        W, X, Z = np.abs(f64(self.wr)), np.abs(np.where(keep[:, None], self.xv, 0)), np.abs(dz)
        Ep = -(-E // 32) * 32
        # dx above 96 tokens: fp16 terms of factors scaled per row (dz) and
        # column (Wr) to a largest magnitude of 2^14 or more.  A term leaves
        # 2^-11 of the value, two leave 2^-22, and what is under half of fp16's
        # least step, 2^-25, i.e. 2^-39 of the largest.  bf16 out: one term,
        # |zw - z1 w1| <= (2 2^-11 + 2^-22) |z||w|.  fp32 out: hi hi + hi lo +
        # lo hi: 2 2^-22 left of the factors and lo lo <= 2^-22.  Up to 96 tokens
        # the products are fp32's.  The accumulation rounds once for each of
        # nprod Ep additions (2 U: a matrix core may truncate).
        one = self.dx.dtype == B16
        split, nprod = (2.001 * 2.0 ** -11, 1) if one else (3 * 2.0 ** -22, 3)
        floor = 2.0 ** -38 * (Z.max(1, keepdims=True) * W.sum(0) + Z.sum(1, keepdims=True) * W.max(0))
        if T <= 96:
            split, nprod, floor = U, 1, (Ep + 32) * 2.0 ** -150
        b = err @ W + (split + 2 * U * nprod * (Ep + 32)) * (Z @ W) + floor
        # and half the least step that the stored type has: 2^-133 (bf16),
        # 2^-149 (fp32); in the unscaled fp32 sums every addition may lose that
        close(self.dx, wx, b + (UB if one else U) * (np.abs(wx) + b) + (2.0 ** -134 if one else 2.0 ** -150))
        n = 3 * (-(-T // 32) * 32) + 16
        close(self.dwr, ww, err.T @ X + (2.0 ** -24 + 2 * U * n + 2 * U) * (Z.T @ X))
        close(self.db, wb, err.sum(0) + (8 + T / 32 / 8 + 14) * U * Z.sum(0))


@pytest.mark.parametrize("src,renorm,dxt", [("x", True, B16), ("x", False, F32), ("q_norm", True, F32), ("q_out", False, B16)])
@pytest.mark.parametrize("T,H,E,k", [(1, 128, 8, 2), (4, 256, 8, 2), (33, 384, 40, 3), (130, 128, 257, 8), (64, 640, 1, 1),
                                     (300, 1024, 130, 4), (40, 256, 1024, 32), (96, 256, 33, 2), (97, 384, 40, 3), (128, 256, 64, 2),
                                     (140, 256, 1024, 32), (161, 896, 385, 6), (256, 128, 8, 2)])
def test_route_backward(T, H, E, k, src, renorm, dxt):
    c = Route(T, H, E, k, src, renorm, mask=T > 4, dxt=dxt, seed=T)
    c.run()
    c.check()


@pytest.mark.parametrize("src,dxt", [("x", B16), ("q_norm", F32)])
@pytest.mark.parametrize("T,H,E,k", [(2100, 4224, 40, 3), (2100, 4224, 257, 8), (400, 2176, 65, 2)])
def test_route_backward_many_tiles(T, H, E, k, src, dxt):
    """More dx tiles than compute units and hidden tiles that do not divide by
    the eight XCDs (17 in groups of three, 9 in groups of two)."""
    c = Route(T, H, E, k, src, True, mask=True, dxt=dxt, seed=E)
    c.run()
    c.check()
    got = c.dx.clone()
    c.dx.fill_(7.0)
    c.run(dwr=False)
    torch.cuda.synchronize()
    assert torch.equal(c.dx, got)


@pytest.mark.parametrize("T", [1500, 2081])
def test_route_backward_split_tokens(T):
    """Enough tokens that dw_router is summed in parts."""
    c = Route(T, 256, 96, 4, "x", True, mask=True)
    c.run()
    c.check()
    # the worst-case bound grows with the tokens; roundings of either sign
    # stay within six times its square root
    dz = ot.route_dlogits(None, c.ids.cpu().numpy(), f64(c.w), f64(c.dw), True, f64(c.dz), c.E, c.mask.cpu().numpy())
    X = np.where(c.mask.cpu().numpy().astype(bool)[:, None], c.xv, 0)
    rms = np.sqrt(np.square(np.where(np.isnan(dz), 0, dz)).T @ np.square(X))
    err = np.abs(f64(c.dwr) - np.where(np.isnan(dz), 0, dz).T @ X)
    assert np.all(err <= 6 * U * np.sqrt(3 * T) * rms * np.sqrt(T) + 40 * U * rms)


@pytest.mark.parametrize("dw,dz", [(True, False), (False, True)])
def test_route_backward_one_gradient(dw, dz):
    c = Route(50, 256, 24, 3, "x", True, dw=dw, dz=dz)
    c.run()
    c.check()


@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_dropped_and_repeated_ids(renorm):
    c = Route(37, 128, 24, 3, "x", renorm)
    c.ids[3, 1], c.ids[4, 0], c.ids[5, 2] = -1, 24, 1 << 30
    c.ids[6, 1] = c.ids[6, 0]
    c.ids[7] = -1
    c.run()
    c.check()


@pytest.mark.parametrize("T", [90, 150])
@pytest.mark.parametrize("dxt", [B16, F32])
def test_route_backward_magnitudes(dxt, T):
    """Rows of dz and columns of Wr over many decades, within and between rows:
    the scaling keeps every row's own precision."""
    c = Route(T, 256, 72, 3, "x", True, dw=False, dxt=dxt)
    g = torch.Generator().manual_seed(3)
    c.dz *= 10.0 ** (torch.rand((T, 1), generator=g) * 40 - 30).cuda()
    c.dz[:45] *= 10.0 ** -(torch.rand((45, 72), generator=g) * 9).cuda()
    c.dz[3] = 0
    c.wr *= 10.0 ** (torch.rand((1, 256), generator=g) * 20 - 15).cuda()
    c.wr[:, :128] *= 10.0 ** -(torch.rand((72, 128), generator=g) * 9).cuda()
    c.wr[:, 5] = 0
    c.run()
    c.check()


@pytest.mark.parametrize("T", [70, 140])
def test_route_backward_nonfinite_rows(T):
    """A non-finite entry makes its own row (or column) non-finite and no other."""
    for dxt in (B16, F32):
        c = Route(T, 256, 40, 3, "x", True, dw=False, dxt=dxt)
        c.dz[4, 7] = float("inf")
        c.dz[40, 0] = float("nan")
        c.wr[9, 200] = float("-inf")
        c.run()
        torch.cuda.synchronize()
        bad = ~torch.isfinite(c.dx)
        want = torch.zeros_like(bad)
        want[4] = want[40] = True
        want[:, 200] = True
        assert torch.equal(bad, want)
        bad = ~torch.isfinite(c.dwr)
        want = torch.zeros_like(bad)
        want[7] = want[0] = True
        assert torch.equal(bad, want)
        assert not torch.isfinite(c.db[[0, 7]]).any() and torch.isfinite(c.db[1:7]).all()


def test_route_backward_parts():
    """Each output alone has the bits it has with the others."""
    c = Route(70, 256, 40, 3)
    c.run()
    torch.cuda.synchronize()
    want = [t.clone() for t in (c.dx, c.dwr, c.db)]
    for i in range(3):
        for t in (c.dx, c.dwr, c.db):
            t.fill_(3.0)
        c.ws.fill_(0xFF)
        c.run(dx=i == 0, dwr=i == 1, db=i == 2)
        torch.cuda.synchronize()
        for j, t in enumerate((c.dx, c.dwr, c.db)):
            assert torch.equal(t, want[j]) if i == j else torch.all(t == 3.0)


def test_empty_batch_writes_zero_sums():
    s = moe.shape(256, 128, 8, 2)
    e16, e32 = torch.empty((0, 256), dtype=B16, device="cuda"), torch.empty((0, 8), device="cuda")
    dw, dwr, db = (torch.full(n, 7.0, device="cuda") for n in ((256,), (8, 256), (8,)))
    w = torch.ones(256, device="cuda")
    moe.moe_rms_norm(s, e16, None, w, EPS, None, e16)
    moe.moe_rms_norm_backward(s, e16, None, e16, None, None, torch.empty(0, device="cuda"), w, None, e16, dw, None)
    moe.moe_route_backward(s, e16, None, None, None, torch.empty((8, 256), device="cuda"), True, None, None, None, None,
                           e32, None, None, dwr, db, None)
    torch.cuda.synchronize()
    assert torch.all(dw == 0) and torch.all(dwr == 0) and torch.all(db == 0)


# ------------------------------ the largest sizes ---------------------------
def test_elements_past_32_bits():
    """2^20 tokens: the tensors' last elements are past 2^32 (x, dx) and their
    bytes past it (logits); the last rows and the sums over all of them."""
    T, H, E, k = 1 << 20, 4224, 8, 2
    s = moe.shape(H, 128, E, k)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty((T, H), dtype=B16, device="cuda").normal_(generator=g)
    w = 1 + rnd(1, (H,), 0.2)
    y = torch.empty_like(x)
    codes = torch.empty((T, H), dtype=torch.uint8, device="cuda")
    sc = torch.empty((T, H // 32), dtype=torch.uint8, device="cuda")
    r = torch.empty(T, device="cuda")
    moe.moe_rms_norm(s, x, None, w, EPS, None, y, moe.MOE_Q_NORMALIZED, codes, sc, r)
    rows = [0, 1, T // 2 + 1, T - 2, T - 1]
    h, wr, n, wy = ot.rms_norm(f64(x[rows]), None, f64(w), float(np.float32(EPS)), False, False)
    close(y[rows], wy, np.abs(wy) * (UB + 4 * U))
    c0, s0 = ot.mx8_encode(n)
    assert np.array_equal(codes[rows].cpu().numpy(), c0) and np.array_equal(sc[rows].cpu().numpy(), s0)
    # backward of the norm, dx over y's memory
    dw = torch.empty(H, device="cuda")
    ws = new_ws(s, T)
    moe.moe_rms_norm_backward(s, x, None, None, codes, sc, r, w, None, y, dw, ws)
    dx, _ = ot.rms_norm_backward(f64(x[rows]), None, ot.mx8_decode(c0, s0), f64(r[rows]), f64(w))
    close(y[rows], dx, np.abs(dx) * UB + 1e-4)
    # the router's backward: every token has the same two picks' gradient
    dz = torch.full((T, E), 0.0, device="cuda")
    dz[:, 3] = 1.0
    dz[T - 1, 5] = 2.0
    wrt = rnd(2, (E, H), 0.1)
    dwr, db = torch.empty((E, H), device="cuda"), torch.empty(E, device="cuda")
    moe.moe_route_backward(s, x, None, None, None, wrt, True, None, None, None, None, dz, None, y, dwr, db, ws)
    torch.cuda.synchronize()
    want = f64(dz[rows]) @ f64(wrt)
    close(y[rows], want, np.abs(want) * UB + 3e-3 * (np.abs(f64(dz[rows])) @ np.abs(f64(wrt))))
    total = sum(x[i:i + 65536].double().sum(0) for i in range(0, T, 65536)).cpu().numpy()
    # 2^20 values of order 1 in fp32: a random walk of roundings of sums of
    # order 2^10, 2^15 additions in a chain each
    assert np.max(np.abs(f64(dwr[3]) - total)) < 0.05
    assert np.array_equal(f64(dwr[5]), 2 * f64(x[T - 1])) and torch.all(dwr[[0, 1, 2, 4, 6, 7]] == 0)
    assert db.tolist() == [0, 0, 0, float(T), 0, 2, 0, 0]
    del x, y, codes, sc, ws, dz
    # logits of 4 GB
    E = 1024
    s = moe.shape(128, 128, E, 1)
    z = torch.empty((T, E), device="cuda").normal_(generator=g)
    ids = torch.full((T, 1), 7, dtype=torch.int32, device="cuda")
    o = balance(s, z, ids, None, None, 1.0)
    torch.cuda.synchronize()
    assert o["counts"][0, 7].item() == T and o["counts"].sum().item() == T
    p = sum(torch.softmax(z[i:i + 65536].double(), 1).sum(0) for i in range(0, T, 65536)) / T
    assert torch.max(torch.abs(o["prob_mean"][0].double() - p) / p).item() < 1e-5
    assert abs(o["loss"].item() - E * p[7].item()) < 1e-5 * E * p[7].item()
    t = T - 1
    pr = torch.softmax(z[t].double(), 0)
    a = torch.zeros(E, dtype=torch.float64, device="cuda")
    a[7] = E / T
    want = pr * (a - (pr * a).sum())
    assert torch.max(torch.abs(o["dlogits"][t].double() - want)).item() < 1e-5 * a[7].item()


# ------------------------------ in use together -----------------------------
class Chain:
    """norm -> route -> balance loss, then back: balance, router, norm (from
    the checkpoint), as a trainer of the router and the norm runs them."""

    def __init__(self, T=96, H=256, E=24, k=3, seed=0):
        self.T, self.H, self.E, self.k = T, H, E, k
        self.s = moe.shape(H, 128, E, k)
        self.x, self.res = rnd(seed, (T, H), 0.5, B16), rnd(seed + 1, (T, H), 2.0, B16)
        self.wn, self.wr = 1 + rnd(seed + 2, (H,), 0.2), rnd(seed + 3, (E, H), H ** -0.5)
        self.dtw, self.dres = rnd(seed + 4, (T, k), 0.1), rnd(seed + 5, (T, H), 0.01)
        e = lambda *n, d=F32: torch.empty(n, dtype=d, device="cuda")  # noqa: E731
        self.h, self.y, self.r = e(T, H, d=B16), e(T, H, d=B16), e(T)
        self.c, self.sc = e(T, H, d=torch.uint8), e(T, H // 32, d=torch.uint8)
        self.ids, self.w, self.z = e(T, k, d=torch.int32), e(T, k), e(T, E)
        self.loss, self.cnt, self.nv = e(1), e(1, E, d=torch.int32), e(2, d=torch.int32)
        self.pm, self.dz, self.dx = e(1, E), e(T, E), e(T, H)
        self.dwr, self.db, self.dh, self.dwn = e(E, H), e(E), e(T, H), e(H)
        self.ws = new_ws(self.s, T)
        self.lws = torch.empty(moe.moe_workspace_bytes(self.s, T), dtype=torch.uint8, device="cuda")

    OUT = ("h", "y", "c", "sc", "ids", "w", "z", "loss", "cnt", "nv", "dz", "dx", "dwr", "db", "dh", "dwn")

    def run(self, stream=None):
        s = self.s
        moe.moe_rms_norm(s, self.x, self.res, self.wn, EPS, self.h, self.y, moe.MOE_Q_NORMALIZED, self.c, self.sc,
                         self.r, stream)
        moe.moe_route(s, self.y, self.wr, None, True, self.ids, self.w, self.z, self.lws, stream)
        moe.moe_balance_loss(s, self.z, self.ids, None, None, 0.1, self.loss, self.cnt, self.nv, self.pm, self.ws,
                             stream)
        moe.moe_balance_loss_backward(s, self.z, None, None, 0.1, None, self.cnt, self.nv, self.dz, stream)
        moe.moe_route_backward(s, None, self.c, self.sc, self.wn, self.wr, True, self.z, self.ids, self.w, self.dtw,
                               self.dz, None, self.dx, self.dwr, self.db, self.ws, stream)
        moe.moe_rms_norm_backward(s, self.dx, self.dres, None, self.c, self.sc, self.r, self.wn, None, self.dh,
                                  self.dwn, self.ws, stream)

    def outs(self):
        return {n: getattr(self, n).clone() for n in self.OUT}


def test_chain_matches_the_formulas():
    c = Chain()
    c.run()
    torch.cuda.synchronize()
    # each step against the oracle on the step's own inputs
    n = ot.mx8_decode(c.c.cpu().numpy(), c.sc.cpu().numpy())
    z, ids = f64(c.z), c.ids.cpu().numpy()
    ref = ot.balance_loss(z, ids, c.E, c.k, 0.1)
    rel = lambda a, b: np.linalg.norm(f64(a) - b) / np.linalg.norm(b)  # noqa: E731
    assert rel(c.loss, np.array([ref["loss"]])) < 1e-5 and rel(c.dz, ref["dlogits"]) < 1e-5
    dz = ot.route_dlogits(z, ids, f64(c.w), f64(c.dtw), True, f64(c.dz), c.E)
    dx, dwr, db = ot.route_backward(dz, n * f64(c.wn), f64(c.wr))
    assert rel(c.dx, dx) < 1e-5 and rel(c.dwr, dwr) < 1e-5 and rel(c.db, db) < 1e-5
    dh, dwn = ot.rms_norm_backward(f64(c.dx), f64(c.dres), n, f64(c.r), f64(c.wn))
    assert rel(c.dh, dh) < 1e-5 and rel(c.dwn, dwn) < 1e-5


def test_chain_gradient_against_differences():
    """The chain's gradients of the router weight and of the norm's weight
    along a direction, against differences of the whole loss in float64 (from
    the stored h; the picks and the counts held, as the gradient holds them).
    The checkpoint replaces n by values within half a step of e4m3 (2^-4), so
    the gradients agree to that, in the norm over a random direction: 2^-4."""
    c = Chain(T=200)
    c.run()
    torch.cuda.synchronize()
    h, r, ids = f64(c.h), f64(c.r), c.ids.cpu().numpy().astype(np.int64)
    wn, wr, cnt = f64(c.wn), f64(c.wr), f64(c.cnt)[0]
    f = cnt * c.E / (c.k * c.T)

    def loss(wn, wr):
        z = (h * r[:, None] * wn) @ wr.T
        top = np.take_along_axis(z, ids, 1)
        p = np.exp(top - top.max(1, keepdims=True))
        return 0.1 * (f * ot.softmax(z).mean(0)).sum() + (f64(c.dtw) * p / p.sum(1, keepdims=True)).sum()

    e = 1e-5
    for got, i in ((f64(c.dwn), 0), (f64(c.dwr), 1)):
        d = got / np.linalg.norm(got)
        a = (wn + e * d, wr) if i == 0 else (wn, wr + e * d)
        b = (wn - e * d, wr) if i == 0 else (wn, wr - e * d)
        assert abs((loss(*a) - loss(*b)) / (2 * e) - np.linalg.norm(got)) <= 2.0 ** -4 * np.linalg.norm(got)


def test_chain_on_another_stream_and_twice():
    a, b = Chain(seed=1), Chain(seed=2)
    a.run()
    b.run()
    torch.cuda.synchronize()
    wa, wb = a.outs(), b.outs()
    for t in (a, b):
        for n in Chain.OUT:
            getattr(t, n).zero_()
        t.ws.fill_(0x77)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        a.run(sa)          # two at once, each with its own workspace
        with torch.cuda.stream(sb):
            b.run()
    torch.cuda.synchronize()
    for n in Chain.OUT:
        assert torch.equal(getattr(a, n), wa[n]), n
        assert torch.equal(getattr(b, n), wb[n]), n


def test_chain_graph_replay():
    c = Chain(T=300, H=512, E=72, k=4)
    c.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    st = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=st):
        c.run(st)
    for i in range(4):
        c.x.copy_(rnd(50 + i, (c.T, c.H), 0.5, B16))
        c.run()                     # eager, the program's own
        torch.cuda.synchronize()
        want = c.outs()
        for n in Chain.OUT:
            getattr(c, n).zero_()
        c.ws.fill_(i)
        g.replay()
        torch.cuda.synchronize()
        for n in Chain.OUT:
            assert torch.equal(getattr(c, n), want[n]), (i, n)


# --------------------------------- refusals ---------------------------------
def refuse(status, f, *a, **k):
    with pytest.raises(moe.MoeError) as e:
        f(*a, **k)
    assert e.value.status == status, e.value


def test_refusals():
    T, H, E, k = 8, 256, 16, 2
    s = moe.shape(H, 128, E, k)
    c = Norm(T, H, B16, B16, moe.MOE_Q_OUTPUT)
    bad, arg = moe.MOE_ERR_MISALIGNED, moe.MOE_ERR_INVALID_ARG
    big = torch.zeros(T * H + 8, dtype=B16, device="cuda")
    refuse(bad, moe.moe_rms_norm, s, big[1:1 + T * H].view(T, H), None, c.w, EPS, c.ro, c.y)
    refuse(arg, moe.moe_rms_norm, s, c.x, c.res, c.w, -1.0, c.ro, c.y)
    refuse(arg, moe.moe_rms_norm, s, c.x, c.res, c.w, float("nan"), c.ro, c.y)
    refuse(arg, moe.moe_rms_norm, s, c.x, c.res, c.w, EPS, None, None)
    refuse(arg, moe.moe_rms_norm, s, c.x, c.res, c.w, EPS, c.ro, c.y, 5)
    refuse(arg, moe.moe_rms_norm, s, c.x, c.res, c.w, EPS, c.ro, c.y, moe.MOE_Q_OUTPUT, None, c.sc)
    refuse(arg, moe.moe_rms_norm, s, c.x, c.res, c.w, EPS, c.ro, c.ro)                # two outputs in one
    refuse(arg, moe.moe_rms_norm, s, c.x, c.res, c.w, EPS, c.ro, c.res)               # y over the residual
    two = torch.zeros(T * H + 64, dtype=B16, device="cuda")
    refuse(arg, moe.moe_rms_norm, s, two[:T * H].view(T, H), None, c.w, EPS, None, two[64:].view(T, H))
    refuse(moe.MOE_ERR_NOT_DEVICE_ACCESSIBLE, moe.moe_rms_norm, s, c.x.cpu(), c.res, c.w, EPS, c.ro, c.y)
    with pytest.raises(TypeError):
        moe.moe_rms_norm(s, c.x.half(), c.res, c.w, EPS, c.ro, c.y)
    with pytest.raises(ValueError):
        moe.moe_rms_norm(s, c.x, c.res[:4], c.w, EPS, c.ro, c.y)
    with pytest.raises(ValueError):
        moe.moe_rms_norm(s, torch.zeros((H, T), dtype=B16, device="cuda").t(), c.res, c.w, EPS, c.ro, c.y)
    with pytest.raises(TypeError):
        moe.moe_rms_norm(s, c.x, c.res, c.w, EPS, c.ro.float(), c.y)
    torch.cuda.synchronize()
    assert torch.all(c.ro == 7) and torch.all(c.y == 7)

    # in place twice: y and residual_out both over x
    refuse(arg, moe.moe_rms_norm, s, c.x, c.res, c.w, EPS, c.x, c.x)

    dy, r, dw = rnd(1, (T, H)), torch.ones(T, device="cuda"), torch.full((H,), 7.0, device="cuda")
    ws = new_ws(s, T, 3)
    refuse(moe.MOE_ERR_WORKSPACE_TOO_SMALL, moe.moe_rms_norm_backward, s, dy, None, c.x, None, None, r, c.w, None, None,
           dw, ws[:256])
    refuse(bad, moe.moe_rms_norm_backward, s, dy, None, c.x, None, None, r, c.w, None, None, dw,
           torch.empty(moe.moe_train_workspace_bytes(s, T) + 256, dtype=torch.uint8, device="cuda")[16:])
    refuse(arg, moe.moe_rms_norm_backward, s, dy, None, c.x, c.c, c.sc, r, c.w, None, None, dw, ws)   # two sources
    refuse(arg, moe.moe_rms_norm_backward, s, dy, None, None, None, None, r, c.w, None, None, dw, ws)  # none
    refuse(arg, moe.moe_rms_norm_backward, s, dy, None, c.x, None, None, r, c.w, None, None, None, ws)
    refuse(arg, moe.moe_rms_norm_backward, s, dy, None, c.x, None, None, r, c.w, None, None, c.w, ws)

    z, ids = routing(1, T, E, k)
    loss, cnt, nv = torch.full((1,), 7.0, device="cuda"), torch.zeros((1, E), dtype=torch.int32, device="cuda"), \
        torch.zeros(2, dtype=torch.int32, device="cuda")
    refuse(arg, moe.moe_balance_loss, s, z, ids, None, None, float("inf"), loss, cnt, nv, None, ws)
    refuse(moe.MOE_ERR_WORKSPACE_TOO_SMALL, moe.moe_balance_loss, s, z, ids, None, None, 1.0, loss, cnt, nv, None, None)
    refuse(moe.MOE_ERR_UNSUPPORTED_SHAPE, moe.moe_balance_loss, s, z, ids, None,
           torch.zeros(1, dtype=torch.int32, device="cuda"), 1.0, loss, cnt[:0], nv[:1], None, ws)
    with pytest.raises(ValueError):
        moe.moe_balance_loss(s, z, ids, None, torch.zeros(4, dtype=torch.int32, device="cuda"), 1.0, loss, cnt, nv,
                             None, ws)
    wr, dx = rnd(2, (E, H)), torch.full((T, H), 7.0, device="cuda")
    w = torch.softmax(z, 1).gather(1, ids.long())
    refuse(arg, moe.moe_route_backward, s, c.x, None, None, None, wr, True, None, ids, w, w, None, None, None, None,
           None, ws)
    refuse(arg, moe.moe_route_backward, s, c.x, c.c, c.sc, None, wr, True, None, ids, w, w, None, None, dx, wr, None, ws)
    refuse(arg, moe.moe_route_backward, s, c.x, None, None, None, wr, True, None, ids, w, w, None, None, dx, wr, None, ws)
    refuse(arg, moe.moe_route_backward, s, c.x, None, None, None, wr, False, None, ids, w, w, None, None, dx, None, None,
           ws)                                                                        # logits are needed
    with pytest.raises(ValueError):
        moe.moe_route_backward(s, c.x, None, None, None, wr, True, None, ids, w, None, None, None, dx, None, None, ws)
    torch.cuda.synchronize()
    assert torch.all(dx == 7) and torch.all(dw == 7) and loss.item() == 7

"""The norm and the router's training side without a GPU: sizes, and the
argument errors raised before any launch."""
import ctypes

import pytest

moe = pytest.importorskip("moe_routed_expert_router_amd",
                          reason="libmoe.so not built (python moe_routed_expert_router_amd/build.py)")


def test_train_workspace_bytes():
    s = moe.shape(4096, 2048, 384, 6)
    w1, w8192 = moe.moe_train_workspace_bytes(s, 1, 1), moe.moe_train_workspace_bytes(s, 8192, 1)
    assert 0 < w1 < w8192
    assert moe.moe_train_workspace_bytes(s, 0, 1) > 0
    assert moe.moe_train_workspace_bytes(s, 8192, 32768) >= w8192
    for bad in ((s, -1, 1), (s, 1, 0), (s, 1, 32769), (moe.shape(100, 128, 8, 2), 1, 1)):
        assert moe.moe_train_workspace_bytes(*bad) == 0


@pytest.mark.parametrize("H", [128, 1024, 1152, 4096, 16512, 65536])
@pytest.mark.parametrize("E", [1, 8, 257, 1024])
def test_train_workspace_serves_fewer_tokens(H, E):
    s = moe.shape(H, 128, E, 1)
    near = {m + d for m in (32, 96, 128, 512, 1024, 2048, 4096, 32768, 65536, 1 << 20) for d in (-1, 0, 1)}
    ts = sorted(t for t in near | set(range(0, 3000, 37)) | {8192, 12345, 100000, 777777} if t <= 1 << 20)
    for n_seq in (1, 64, 32768):
        w = [moe.moe_train_workspace_bytes(s, t, n_seq) for t in ts]
        assert w == sorted(w)


def test_train_entries_reject_before_any_launch():
    lib, s = moe.lib, moe.shape(256, 128, 8, 2)
    p, bad = ctypes.byref(s), moe.shape(100, 128, 8, 2)
    arg, shp = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED_SHAPE
    fake = 4096   # an address that no check may dereference

    def norm(sh=p, T=4, xd=1, x=None, rd=1, eps=1e-6, y=fake, q=0):
        return lib.moe_rms_norm(sh, T, xd, x, rd, fake, fake, eps, None, y, q, None, None, None, None)

    assert norm() == arg and "x is NULL" in moe.moe_last_error()
    assert norm(sh=ctypes.byref(bad)) == shp and norm(T=-1) == shp and norm(T=(1 << 20) + 1) == shp
    assert norm(xd=2) == arg and norm(rd=7) == arg and norm(q=3) == arg and norm(y=None) == arg
    for e in (-1e-6, float("nan"), float("inf")):
        assert norm(eps=e) == arg and "eps" in moe.moe_last_error()
    assert norm(T=0) == moe.MOE_OK
    assert norm(x=8) == moe.MOE_ERR_MISALIGNED

    nb = lib.moe_rms_norm_backward
    assert nb(p, 4, 1, None, 1, None, 1, fake, None, None, fake, fake, None, 1, fake, None, None, 0, None) \
        == moe.MOE_ERR_WORKSPACE_TOO_SMALL
    assert nb(p, 4, 1, None, 1, None, 1, fake, None, None, fake, fake, None, 1, None, None, None, 0, None) == arg
    assert nb(p, 4, 1, None, 1, None, 1, fake, fake, fake, fake, fake, None, 1, fake, None, fake, 1 << 30, None) == arg
    assert "both" in moe.moe_last_error()
    assert nb(p, 4, 9, None, 1, None, 1, fake, None, None, fake, fake, None, 1, fake, None, fake, 1 << 30, None) == arg
    assert nb(p, 4, 1, None, 1, None, 1, fake, None, None, fake, fake, None, 1, fake, None, fake, 1 << 30, None) == arg
    assert "dy is NULL" in moe.moe_last_error()
    assert nb(p, 0, 1, None, 1, None, 1, None, None, None, None, None, None, 1, fake, None, None, 0, None) == moe.MOE_OK

    bl = lib.moe_balance_loss
    assert bl(p, 4, None, None, None, None, 2, 1.0, None, None, None, None, fake, 1 << 30, None) == arg
    assert bl(p, 4, None, None, None, None, 0, 1.0, None, None, None, None, fake, 1 << 30, None) == shp
    assert bl(p, 4, None, None, None, None, 1, float("nan"), None, None, None, None, fake, 1 << 30, None) == arg
    assert bl(p, 4, None, None, None, None, 1, 1.0, None, None, None, None, fake, 16, None) \
        == moe.MOE_ERR_WORKSPACE_TOO_SMALL
    assert bl(p, 4, None, None, None, None, 1, 1.0, None, None, None, None, fake, 1 << 30, None) == arg
    assert "logits is NULL" in moe.moe_last_error()
    bb = lib.moe_balance_loss_backward
    assert bb(p, 4, None, None, None, 1, 1.0, None, None, None, None, None) == arg
    assert bb(p, 0, None, None, None, 1, 1.0, None, None, None, None, None) == moe.MOE_OK

    def rb(T=4, x=None, c=None, dw=None, dz=None, dx=fake, dwr=None, dxd=1, ws=1 << 40):
        return lib.moe_route_backward(p, T, x, c, None, None, None, 1, None, None, None, dw, dz, None, dxd, dx, dwr,
                                      None, fake, ws, None)

    assert rb(dz=fake, dx=None) == arg and "no output" in moe.moe_last_error()
    assert rb() == arg and "no gradient" in moe.moe_last_error()
    assert rb(dz=fake, x=fake, c=fake) == arg and "both" in moe.moe_last_error()
    assert rb(dz=fake, dxd=5) == arg
    assert rb(dz=fake, ws=1) == moe.MOE_ERR_WORKSPACE_TOO_SMALL
    assert rb(dz=fake) == arg and "w_router is NULL" in moe.moe_last_error()
    assert rb(dz=fake, dx=None, dwr=fake) == arg and "q_codes is NULL" in moe.moe_last_error()
    assert rb(T=0, dx=fake) == moe.MOE_OK

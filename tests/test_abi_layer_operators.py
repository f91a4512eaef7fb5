"""Host-side refusals of the layer's dense operators: a negative status and
nothing enqueued (no HIP call is made on these paths)."""

import ctypes

NULL = None
FAKE = 0x10000  # 16-byte aligned, never dereferenced
FAR = 1 << 40   # steps between buffers that must not overlap


def _close(lib, **kw):
    a = dict(z=FAKE, z_rows=8, rows=FAKE, k=2, w=NULL, x=FAR, gate=NULL, wp=FAKE, wn=FAKE,
             scale=1.0, eps=1e-6, T=4, H=64, dt=1, y=2 * FAR, h=3 * FAR)
    a.update(kw)
    return lib.moe_combine_norm(*a.values(), NULL, NULL, NULL)


def test_combine_norm_rejects(built_lib):
    f = lambda **kw: _close(built_lib, **kw)  # noqa: E731
    assert f(T=0) == 0                                  # nothing to do
    assert f(dt=2) == -3
    assert f(T=-1) == -2 and f(H=0) == -2 and f(k=9) == -2 and f(k=-1) == -2
    assert f(T=2 ** 30) == -2                           # T * k
    assert f(H=16392) == -2 and f(H=8196, dt=0) == -2   # rows over 32 KiB
    assert f(eps=0.0) == -2 and f(eps=float("nan")) == -2 and f(eps=float("inf")) == -2
    assert f(scale=float("inf")) == -2
    assert f(H=60) == -4 and f(H=66, dt=0) == -4        # rows of whole 16 bytes
    assert f(x=NULL) == -1 and f(rows=NULL) == -1 and f(wp=NULL) == -1 and f(z=NULL) == -1
    assert f(y=NULL, h=NULL) == -1 and f(wn=NULL) == -1
    assert f(x=FAR + 8) == -4 and f(y=2 * FAR + 2) == -4 and f(wp=FAKE + 4) == -4
    assert f(y=FAR) == -2 and f(h=FAR + 64) == -2       # over x
    assert f(y=FAKE) == -2                              # over z
    assert f(h=2 * FAR + 128) == -2                     # y and h


def _grad(lib, **kw):
    a = dict(dy=FAKE, dh=FAKE, z=FAR, z_rows=8, rows=FAKE, k=2, w=FAKE, y=FAKE, gate=NULL, wp=FAKE,
             wn=FAKE, scale=1.0, eps=1e-6, T=4, H=64, dt=1, dx=2 * FAR, dz=3 * FAR, dw=FAKE,
             dg=FAKE, dwp=FAKE, dwn=FAKE, nv=NULL, err=NULL, ws=4 * FAR, n=1 << 20)
    a.update(kw)
    return lib.moe_combine_norm_backward(*a.values(), NULL)


def test_combine_norm_backward_rejects(built_lib):
    f = lambda **kw: _grad(built_lib, **kw)  # noqa: E731
    assert f(dt=7) == -3 and f(T=-1) == -2 and f(H=16392) == -2 and f(eps=-1.0) == -2
    assert f(dy=NULL, dh=NULL) == -1 and f(dx=NULL) == -1 and f(dz=NULL) == -1
    assert f(y=NULL) == -1 and f(wn=NULL) == -1 and f(dwn=NULL) == -1 and f(dwp=NULL) == -1
    assert f(w=NULL) == -1                              # d_row_weight without row_weight
    assert f(ws=NULL) == -1 and f(n=16) == -5 and f(ws=4 * FAR + 4) == -4
    assert f(dz=3 * FAR + 4) == -4
    assert f(dx=FAKE) == -2 and f(dx=FAR) == -2 and f(dz=FAR) == -2 and f(dx=3 * FAR) == -2


def test_combine_norm_workspace(built_lib):
    n = ctypes.c_size_t()
    q = built_lib.moe_combine_norm_backward_workspace_size
    assert q(4, 64, 1, ctypes.byref(n)) == 0 and n.value >= 2 * 64 * 4
    assert q(0, 64, 1, ctypes.byref(n)) == 0 and n.value >= 2 * 64 * 4
    big = ctypes.c_size_t()
    assert q(1 << 20, 64, 1, ctypes.byref(big)) == 0
    assert n.value < big.value <= 4096 * 2 * 64 * 4     # bounded by the launch, not by T
    assert q(4, 64, 1, NULL) == -1 and q(-1, 64, 1, ctypes.byref(n)) == -2
    assert q(4, 60, 1, ctypes.byref(n)) == -4 and q(4, 64, 5, ctypes.byref(n)) == -3


def _ffn(lib, **kw):
    a = dict(x=FAKE, R=8, H=64, F=32, E=2, first=FAKE, count=FAKE, w_in=FAKE, w_down=FAKE, dt=1,
             act=0, gu=FAR, a=2 * FAR, y=3 * FAR)
    a.update(kw)
    return lib.moe_expert_ffn(*a.values(), NULL, NULL)


def test_expert_ffn_rejects(built_lib):
    f = lambda **kw: _ffn(built_lib, **kw)  # noqa: E731
    assert f(R=0) == 0                                  # nothing to do
    assert f(dt=2) == -3 and f(act=2) == -3 and f(act=-1) == -3
    assert f(R=-1) == -2 and f(R=2 ** 31) == -2 and f(H=0) == -2 and f(F=0) == -2
    assert f(E=0) == -2 and f(E=257) == -2
    assert f(H=2 ** 15, F=2 ** 14) == -2                # one expert's w_in passes 2^31 bytes
    assert f(H=2 ** 21 + 8, F=8) == -2 and f(H=8, F=2 ** 20 + 8) == -2
    assert f(H=60) == -4 and f(F=36) == -4 and f(H=66, dt=0) == -4
    for n in ("x", "first", "count", "w_in", "w_down", "a", "y"):
        assert f(**{n: NULL}) == -1, n
    for n in ("x", "w_in", "w_down", "gu", "a", "y"):
        assert f(**{n: 5 * FAR + 8}) == -4, n
    assert f(y=FAKE) == -2 and f(a=FAKE) == -2 and f(gu=FAKE) == -2  # over an input
    assert f(y=2 * FAR) == -2 and f(a=FAR + 64) == -2                # over each other


def _ffn_grad(lib, **kw):
    a = dict(dy=FAKE, x=FAKE, R=8, H=64, F=32, E=2, first=FAKE, count=FAKE, w_in=FAKE, w_down=FAKE,
             gu=FAKE, a=FAKE, dt=1, act=0, dx=FAR, dwi=2 * FAR, dwd=3 * FAR, err=NULL, ws=4 * FAR,
             n=8 * 64 * 2 + 256)
    a.update(kw)
    return lib.moe_expert_ffn_backward(*a.values(), NULL)


def test_expert_ffn_backward_rejects(built_lib):
    f = lambda **kw: _ffn_grad(built_lib, **kw)  # noqa: E731
    assert f(dt=2) == -3 and f(act=2) == -3 and f(R=-1) == -2 and f(E=257) == -2
    assert f(H=60) == -4 and f(F=36) == -4
    for n in ("dy", "x", "first", "count", "w_in", "w_down", "gu", "a", "dx", "dwi", "dwd", "ws"):
        assert f(**{n: NULL}) == -1, n
    assert f(ws=4 * FAR + 8) == -4 and f(dx=FAR + 4) == -4
    assert f(n=8 * 64 * 2 - 1) == -5
    for n in ("dx", "dwi", "dwd", "ws"):
        assert f(**{n: FAKE}) == -2, n                  # over an input
    assert f(dwd=2 * FAR + 16) == -2 and f(ws=FAR) == -2


def test_expert_ffn_workspace(built_lib):
    n = ctypes.c_size_t()
    q = built_lib.moe_expert_ffn_backward_workspace_size
    assert q(100, 64, 32, 2, 1, ctypes.byref(n)) == 0 and n.value >= 100 * 64 * 2
    assert q(100, 64, 32, 2, 0, ctypes.byref(n)) == 0 and n.value >= 100 * 64 * 4
    assert q(0, 64, 32, 2, 1, ctypes.byref(n)) == 0 and n.value == 0
    # few experts with many rows: shares of both weight gradients, one at a time
    assert q(100000, 64, 32, 2, 1, ctypes.byref(n)) == 0
    assert 100000 * 64 * 2 < n.value <= 100000 * 64 * 2 + 256 + 256 * 2 * 64 * 64 * 4
    assert q(100, 64, 32, 2, 1, NULL) == -1 and q(-1, 64, 32, 2, 1, ctypes.byref(n)) == -2
    assert q(100, 64, 36, 2, 1, ctypes.byref(n)) == -4 and q(100, 64, 32, 2, 9, ctypes.byref(n)) == -3
    assert q(100, 64, 32, 0, 1, ctypes.byref(n)) == -2


def test_expert_ffn_most_rows(built_lib):
    """Row counts are rounded up to whole tiles in 32 bits: the last 511
    counts are refused (a missing pointer tells an accepted size)."""
    n = ctypes.c_size_t()
    size = built_lib.moe_expert_ffn_backward_workspace_size
    most = 2 ** 31 - 512
    assert _ffn(built_lib, R=most, x=NULL) == -1 and _ffn(built_lib, R=most + 1, x=NULL) == -2
    assert _ffn_grad(built_lib, R=most, x=NULL) == -1 and _ffn_grad(built_lib, R=most + 1, x=NULL) == -2
    assert size(most, 8, 8, 1, 1, ctypes.byref(n)) == 0 and n.value >= most * 32
    assert size(2 ** 31 - 1, 8, 8, 1, 1, ctypes.byref(n)) == -2


def test_expert_ffn_outputs_over_the_counts(built_lib):
    """expert_first and expert_count are inputs too."""
    at = 6 * FAR
    for n in ("first", "count"):
        for out in ("gu", "a", "y"):
            assert _ffn(built_lib, **{n: at + 4, out: at}) == -2, (n, out)
        for out in ("dx", "dwi", "dwd", "ws"):
            assert _ffn_grad(built_lib, **{n: at + 4, out: at}) == -2, (n, out)


def test_combine_norm_workspace_over_rows(built_lib):
    """The workspace shares no bytes with a row buffer."""
    at = 6 * FAR
    for n in ("dy", "dh", "y", "z", "dx", "dz"):
        assert _grad(built_lib, ws=at, **{n: at + 64}) == -2, n


def test_combine_norm_gate_gradient_over_the_gate(built_lib):
    """Waves of a token's block read its gate after another has written."""
    at = 6 * FAR
    assert _grad(built_lib, gate=at, dg=at) == -2 and _grad(built_lib, gate=at + 12, dg=at) == -2

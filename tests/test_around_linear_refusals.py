"""Layer norm, the product with an epilogue, its backward and gradient clipping
refuse bad arguments before anything is launched (these calls never reach the
GPU, so they run on a host without one)."""
import ctypes

import pytest
import torch

import fp8_quantized_lora_amd as fq

EINVAL, OK = 1, 0
P = 1 << 20          # 16-byte aligned fake addresses, never dereferenced
Q, R, S = 1 << 21, 1 << 22, 1 << 23
MIS = P + 1          # no element's alignment
BIG = 1 << 40
NAN, INF = float("nan"), float("inf")


def refused(f, ok, changes):
    for idx, val in changes:
        a = list(ok)
        a[idx] = val
        assert f(*a) == EINVAL, (f.__name__, idx, val)


def test_layer_norm_fwd():
    f = fq.load().layer_norm_fwd
    #     x  xt w  b  T  d   eps   y  yt mean rstd stream
    ok = [P, 0, Q, R, 4, 64, 1e-5, S, 1, P, Q, None]
    refused(f, ok, [(0, None), (0, MIS), (7, None), (7, MIS), (7, P), (1, 2), (8, -1), (2, MIS),
                    (3, MIS), (9, MIS), (10, MIS), (4, -1), (4, (1 << 30) + 1), (5, 0), (5, -8),
                    (5, (1 << 24) + 1), (6, -1e-5), (6, NAN), (6, INF)])
    assert f(None, 0, None, None, 0, 64, 1e-5, None, 0, None, None, None) == OK      # T = 0


def test_layer_norm_bwd():
    f = fq.load().layer_norm_bwd
    ws = fq.layer_norm_bwd_workspace_bytes(2000, 64)
    assert ws >= 2 * 64 * 4
    assert fq.layer_norm_bwd_workspace_bytes(-1, 64) == 0
    assert fq.layer_norm_bwd_workspace_bytes(4, 0) == 0
    assert fq.layer_norm_bwd_workspace_bytes(4, 64) == 0       # few rows need none
    #     dy gt x  xt w  mu rs T     d   dx dw db ws n   stream
    ok = [P, 0, Q, 1, R, S, S, 2000, 64, P, Q, R, S, ws, None]
    refused(f, ok, [(0, None), (0, MIS), (2, None), (2, MIS), (5, None), (6, None), (4, MIS),
                    (9, MIS), (9, Q), (10, MIS), (10, R), (11, MIS), (1, 5), (3, 2), (7, -1),
                    (8, 0), (8, (1 << 24) + 1), (12, None), (12, P + 16), (13, ws - 1)])


def test_linear_act_fwd():
    f = fq.load().melded_linear_fwd_act
    assert fq.melded_linear_fwd_act_workspace_bytes(8, 32, 48) == 0
    assert fq.melded_linear_fwd_act_workspace_bytes(8, 33, 48) == 0
    nb = fq.melded_linear_fwd_act_workspace_bytes(64, 13824, 5120)
    assert nb >= 2 * 64 * 5120 * 4                              # split over d_in
    #     xq sx wq sw b  act res T  di  do  t  y  z  ws n  stream
    ok = [P, P, Q, P, R, 2, S, 64, 13824, 5120, 1, P, Q, R, nb, None]
    refused(f, ok, [(13, None), (13, P + 16), (14, nb - 1)])
    ok = [P, P, Q, P, R, 2, S, 8, 32, 48, 1, P, Q, None, 0, None]
    refused(f, ok, [(0, None), (0, MIS), (1, None), (1, P + 2), (2, None), (3, None), (4, MIS),
                    (5, -1), (5, 5), (6, MIS), (7, -1), (8, 24), (9, 40), (10, 2), (11, None),
                    (11, MIS), (12, MIS), (12, P), (12, S), (7, 1 << 31)])
    # more 256 x 256 tiles than a 32-bit grid holds
    assert f(P, P, Q, P, None, 0, None, 1 << 30, 32, 1 << 30, 1, R, None, None, 0,
             None) == EINVAL
    assert f(None, P, Q, P, None, 0, None, 0, 32, 48, 1, None, None, None, 0, None) == OK  # T = 0
    assert f(P, P, None, P, None, 0, None, 4, 32, 0, 1, None, None, None, 0, None) == OK   # d_out


def test_linear_act_bwd():
    f = fq.load().linear_act_bwd
    ws = fq.linear_act_bwd_workspace_bytes(1000, 48)
    assert ws >= 48 * 4 and fq.linear_act_bwd_workspace_bytes(8, -1) == 0
    assert fq.linear_act_bwd_workspace_bytes(8, 48) == 0        # few rows need none
    #     dy gt z  zt act T    d   dz db ws n   stream
    ok = [P, 0, Q, 1, 2, 1000, 48, R, S, P, ws, None]
    refused(f, ok, [(0, None), (0, MIS), (2, None), (2, MIS), (7, MIS), (7, Q),
                    (1, 2), (3, 2), (4, -1), (4, 5), (5, -1), (6, -1), (6, (1 << 24) + 1),
                    (8, MIS), (9, None), (9, P + 16), (10, ws - 1)])
    assert f(None, 0, None, 0, 2, 8, 0, None, None, None, 0, None) == OK             # d_out = 0
    assert f(P, 0, Q, 1, 2, 8, 48, None, None, None, 0, None) == EINVAL              # no output


def arrays(ptrs, n, t):
    k = len(ptrs)
    return ((ctypes.c_void_p * k)(*ptrs), (ctypes.c_int64 * k)(*n), (ctypes.c_int32 * k)(*t))


def test_grad_calls():
    lib = fq.load()
    ws = fq.grad_norm_workspace_bytes(2)
    assert ws > 0 and fq.grad_norm_workspace_bytes(-1) == 0
    assert fq.grad_norm_workspace_bytes(fq.GRAD_MAX_TENSORS + 1) == 0

    def both(ptrs=(P, Q), n=(100, 100), t=(0, 1), norm=S, w=R, nb=ws, count=2, max_norm=1.0,
             eps=1e-6, out=None):
        g, nn, tt = arrays(ptrs, n, t)
        o = None if out is None else arrays(out, n, t)[0]
        return (lib.grad_norm(count, g, nn, tt, norm, w, nb, None),
                lib.grad_clip(count, g, nn, tt, max_norm, eps, o, norm, w, nb, None))

    for bad in (dict(ptrs=(P, None)), dict(ptrs=(P + 2, Q)), dict(ptrs=(P, Q + 1)),
                dict(n=(100, -1)), dict(n=(100, BIG + 1)), dict(n=(BIG, BIG)), dict(t=(0, 2)),
                dict(norm=None), dict(norm=S + 2), dict(w=None), dict(w=R + 16),
                dict(nb=ws - 1), dict(count=-1), dict(count=fq.GRAD_MAX_TENSORS + 1)):
        assert both(**bad) == (EINVAL, EINVAL), bad
    g, nn, tt = arrays((P, Q), (100, 100), (0, 1))
    assert lib.grad_norm(2, None, nn, tt, S, R, ws, None) == EINVAL
    assert lib.grad_norm(2, g, None, tt, S, R, ws, None) == EINVAL
    assert lib.grad_norm(2, g, nn, None, S, R, ws, None) == EINVAL
    for bad in (dict(max_norm=-1.0), dict(max_norm=NAN), dict(eps=-1e-6), dict(eps=NAN),
                dict(eps=INF), dict(out=(P, None)), dict(out=(P + 2, Q)),
                dict(ptrs=(P, P), t=(0, 0)),                      # one tensor twice
                dict(ptrs=(P, P + 396), t=(0, 0)),                # overlapping by one element
                dict(out=(Q, P)),                                 # another input's memory
                dict(out=(P + 4, R)), dict(out=(R, R + 100))):
        assert both(**bad)[1] == EINVAL, bad


def test_overlaps_are_refused():
    """One element of an output in another tensor of the call, in the workspace or
    in its own input but not at its start."""
    lib = fq.load()
    at = [(i + 1) << 24 for i in range(10)]                 # far apart
    x, w, b, mu, rs, dy, o, dw, db, ws = at
    T, d = 2000, 64
    big = T * d * 4
    fwd = [x, 0, w, b, T, d, 1e-5, o, 0, mu, rs, None]
    refused(lib.layer_norm_fwd, fwd,
            [(7, x), (7, x + big - 4), (7, x - big + 4), (7, w), (7, b + 4 * d - 4),
             (7, mu + 4 * T - 4), (9, rs - 4 * T + 4), (9, x + 4), (9, w), (10, x), (10, mu)])
    nb = fq.layer_norm_bwd_workspace_bytes(T, d)
    bwd = [dy, 0, x, 0, w, mu, rs, T, d, o, dw, db, ws, nb, None]
    refused(lib.layer_norm_bwd, bwd,
            [(9, x), (9, dy + 4), (9, dy - 4), (9, w), (9, mu), (9, rs), (9, dw), (9, ws),
             (10, db + 4), (10, db), (10, dy), (10, w), (11, ws + nb - 4), (11, x), (12, dy),
             (12, x)])
    xq, sx, wq, sw, b, res, y, z, ws = at[:9]
    T, d_in, d_out = 64, 13824, 5120
    nb, big = fq.melded_linear_fwd_act_workspace_bytes(T, d_in, d_out), T * d_out * 2
    act = [xq, sx, wq, sw, b, 2, res, T, d_in, d_out, 1, y, z, ws, nb, None]
    refused(lib.melded_linear_fwd_act, act,
            [(11, res + 2), (11, res - 2), (11, z + big - 2), (11, xq + T * d_in - 2),
             (11, wq - 2 + d_in * d_out), (11, sx), (11, sw), (11, b), (11, ws), (12, res),
             (12, xq), (12, ws - 2), (12, b - big + 2), (13, xq), (13, wq), (13, res)])
    dy, z, dz, db, ws = at[:5]
    T, d = 1000, 48
    nb = fq.linear_act_bwd_workspace_bytes(T, d)
    ok = [dy, 0, z, 1, 2, T, d, dz, db, ws, nb, None]
    refused(lib.linear_act_bwd, ok,
            [(7, z), (7, z + T * d * 2 - 4), (7, dy + 4), (7, db), (7, ws), (8, dy), (8, z),
             (8, ws), (8, dz + 4), (9, dy), (9, z)])
    g0, g1, norm, ws, o0, o1 = at[:6]
    nb = fq.grad_norm_workspace_bytes(2)
    g, n, t = arrays((g0, g1), (100, 100), (0, 1))
    out = arrays((o0, o1), (100, 100), (0, 1))[0]
    for r, w in ((g0 + 396, ws), (g1, ws), (ws + nb - 4, ws), (norm, g0 & ~255), (norm, g1)):
        assert lib.grad_norm(2, g, n, t, r, w, nb, None) == EINVAL
        assert lib.grad_clip(2, g, n, t, 1.0, 0.0, out, r, w, nb, None) == EINVAL
    for r, w in ((o0, ws), (o1 + 196, ws), (norm, o1)):
        assert lib.grad_clip(2, g, n, t, 1.0, 0.0, out, r, w, nb, None) == EINVAL


def test_binding_refuses_before_the_library():
    x = torch.zeros((4, 64))
    w, s, q = torch.zeros(64), torch.zeros(4), torch.zeros((4, 64), dtype=torch.uint8)
    one = torch.ones(1)
    bad = pytest.raises(fq.FalqError)
    with bad:
        fq.layer_norm_fwd(x.half(), w, w, x)                      # type
    with bad:
        fq.layer_norm_fwd(x, w[:32], w, x.clone())                # shape
    with bad:
        fq.layer_norm_fwd(x, w, w, x.clone(), mean=torch.zeros(5))
    with bad:
        fq.layer_norm_fwd(x, w, w, x.clone())                     # not on the GPU
    with bad:
        fq.layer_norm_bwd(x, x, w, s, s, x.bfloat16())            # dx has dy's type
    with bad:
        fq.layer_norm_bwd(x[:3], x, w, s, s, x.clone())
    with bad:
        fq.melded_linear_fwd_act(q, one, q, one, torch.zeros((4, 4)), act="tanh")
    with bad:
        fq.melded_linear_fwd_act(q, one, q, one, torch.zeros((4, 5)))
    with bad:
        fq.melded_linear_fwd_act(q, one, q, one, torch.zeros((4, 4)),
                                 residual=torch.zeros((4, 4), dtype=torch.bfloat16))
    with bad:
        fq.melded_linear_fwd_act(q, one, q, torch.ones(2), torch.zeros((4, 4)))
    with bad:
        fq.linear_act_bwd(x, None, x.clone(), act="gelu")
    with bad:
        fq.linear_act_bwd(x, x[:2], x.clone(), act="gelu")
    with bad:
        fq.linear_act_bwd(x, x, x.bfloat16(), act="gelu")
    with bad:
        fq.layer_norm_fwd(x[0], w, w, x[0].clone())               # one dimension
    with bad:
        fq.grad_norm([x], one)                                    # not on the GPU
    with bad:
        fq.grad_clip([x], 1.0, torch.ones(2))
    with bad:
        fq.grad_clip([x.half()], 1.0, one)

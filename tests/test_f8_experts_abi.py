"""CPU-side checks of the e4m3 products' and the experts' C entry points and of their
binding: sizes and the refusals, none of which reaches a device."""
import ctypes

import pytest
import torch

import quantized_gemv_argmax_amd as qg

OK, ENULL, ESHAPE, EALIGN, EWS, EDEV, EUNSUP = range(7)
A, B, C, D, E, F, G = (0x1000000000 * i for i in range(1, 8))  # device addresses that nothing dereferences


@pytest.fixture(scope="module")
def L():
    return qg.lib()


def no_gpu():
    return not torch.cuda.is_available()


def test_sizes(L):
    assert L.qg_f8_bytes(16, 128, 1) == 4096
    assert L.qg_f8_bytes(33, 129, 3) == 3 * 2 * 2 * 4096
    assert L.qg_f8_bytes(152064, 3584, 1) == 152064 * 3584
    for m, k, e in [(0, 64, 1), (16, 0, 1), (4194304, 64, 1), (16, 131073, 1), (16, 64, 0), (16, 64, 1025), (4194303, 131072, 1024)]:
        assert L.qg_f8_bytes(m, k, e) == 0
    for m, k, n, t in [(0, 64, 4, 0), (16, 0, 4, 0), (16, 64, 0, 0), (16, 64, 4194304, 0), (65537, 64, 65537, 0), (16, 64, 4, 3)]:
        assert L.qgemm_f8_workspace_bytes(m, k, n, t) == 0
    f = L.logits_expert_select_workspace_bytes
    assert f(5000, 60, 4) >= 60 * -(-5000 // 32) * 4
    for n, e, k in [(0, 8, 2), (5000, 0, 1), (5000, 1025, 2), (5000, 8, 9), (5000, 64, 33), (5000, 8, 0), (4194304, 8, 1), (2100000, 8, 2)]:
        assert f(n, e, k) == 0


def refuser(f, good):
    def bad(*pairs):
        a = list(good)
        for i, v in pairs:
            a[i] = v
        return f(*a)
    return bad


def test_pack_validation(L):
    #       w, ldw, w_expert, dst, M, K, experts, stream
    good = [A, 100, 1700, B, 17, 100, 3, None]
    bad = refuser(L.qg_pack_f8, good)
    if no_gpu():
        assert bad() in (EDEV, EUNSUP)
        assert bad((0, A + 1)) in (EDEV, EUNSUP)  # weights need no alignment
        assert bad((2, 0), (6, 1)) in (EDEV, EUNSUP)
    assert bad((0, None)) == ENULL and bad((3, None)) == ENULL
    assert bad((1, 99)) == ESHAPE and bad((1, 1 << 40)) == ESHAPE
    assert bad((2, 1699)) == ESHAPE and bad((2, 1 << 40)) == ESHAPE
    assert bad((4, 0)) == ESHAPE and bad((4, 4194304)) == ESHAPE and bad((5, 0)) == ESHAPE and bad((5, 131073)) == ESHAPE
    assert bad((6, 0)) == ESHAPE and bad((6, 1025)) == ESHAPE
    assert bad((3, B + 8)) == EALIGN
    assert bad((3, A + 2048)) == ESHAPE  # overlap


def test_quantize_validation(L):
    #       x, type, ldx, gated, count, N, K, q, ldq, scale, lds, stream
    good = [A, 0, 200, 1, None, 4, 100, B, 128, C, 4, None]
    bad = refuser(L.qg_quantize_f8_rows, good)
    if no_gpu():
        assert bad() in (EDEV, EUNSUP)
        assert bad((0, A + 2), (1, 1), (4, D)) in (EDEV, EUNSUP)
    assert [bad((i, None)) for i in (0, 7, 9)] == [ENULL] * 3
    assert bad((1, 3)) == ESHAPE and bad((1, -1)) == ESHAPE and bad((3, 2)) == ESHAPE
    assert bad((2, 199)) == ESHAPE and bad((2, 1 << 40)) == ESHAPE
    assert bad((5, 0)) == ESHAPE and bad((5, 4194304)) == ESHAPE
    assert bad((6, 0)) == ESHAPE and bad((6, 131073)) == ESHAPE
    assert bad((8, 112)) == ESHAPE and bad((8, 136)) == ESHAPE
    assert bad((10, 3)) == ESHAPE and bad((10, 6)) == ESHAPE and bad((6, 700), (2, 1400), (8, 768)) == ESHAPE
    assert bad((0, A + 2)) == EALIGN and bad((7, B + 8)) == EALIGN and bad((9, C + 4)) == EALIGN and bad((4, D + 2)) == EALIGN
    assert bad((7, A + 16)) == ESHAPE and bad((9, A + 16)) == ESHAPE and bad((9, B + 128)) == ESHAPE and bad((4, B + 4)) == ESHAPE


def test_product_validation(L):
    #       w, w_scale, xq, ldx, x_scale, ldxs, bias, Y, type, ldy, M, K, N, ws, ws_bytes, stream
    good = [A, B, C, 128, D, 4, None, E, 0, 20, 20, 100, 3, None, 0, None]
    bad = refuser(L.qgemm_f8, good)
    if no_gpu():
        assert bad() in (EDEV, EUNSUP)
    assert [bad((i, None)) for i in (0, 1, 2, 4, 7)] == [ENULL] * 5
    assert bad((3, 112)) == ESHAPE and bad((3, 136)) == ESHAPE and bad((3, 1 << 40)) == ESHAPE
    assert bad((5, 0)) == ESHAPE and bad((5, 2)) == ESHAPE and bad((5, 1 << 21)) == ESHAPE
    assert bad((8, 3)) == ESHAPE and bad((8, -1)) == ESHAPE
    assert bad((9, 16)) == ESHAPE and bad((9, 22)) == ESHAPE
    assert bad((10, 0)) == ESHAPE and bad((11, 0)) == ESHAPE and bad((12, 0)) == ESHAPE
    assert bad((10, 4194304)) == ESHAPE and bad((11, 131073)) == ESHAPE and bad((12, 4194304)) == ESHAPE
    assert bad((9, 65540), (10, 65537), (12, 65537)) == ESHAPE  # M N over 2^32
    for i in (0, 2, 4, 7):
        assert bad((i, good[i] + 8)) == EALIGN
    assert bad((1, B + 2)) == EALIGN and bad((6, F + 2)) == EALIGN
    for i in (0, 1, 2, 4):  # Y over an input
        assert bad((7, good[i])) == ESHAPE
    assert bad((6, E + 16)) == ESHAPE
    need = L.qgemm_f8_workspace_bytes(3584, 18944, 64, 2)
    if need:
        big = [(3, 18944), (5, 148), (8, 2), (9, 3584), (10, 3584), (11, 18944), (12, 64)]
        assert bad(*big) == EWS
        assert bad(*big, (13, F), (14, need - 1)) == EWS
        assert bad(*big, (13, F + 8), (14, need)) == EALIGN
        assert bad(*big, (13, E), (14, need)) == ESHAPE and bad(*big, (13, A), (14, need)) == ESHAPE


def grouped(**kw):
    d = dict(w_packed=A, w_scale=B, xq=C, ldx=128, x_scale=D, ldxs=4, x_rows=7, row=None, offsets=F, bias=None, Y=E, y_type=2,
             ldy=20, M=20, K=100, experts=3, rows=7)
    d.update(kw)
    p = qg._F8Grouped(*[d[n] for n, _ in qg._F8Grouped._fields_])
    return qg.lib().qgemm_f8_grouped(ctypes.byref(p), None)


def test_grouped_validation(L):
    if no_gpu():
        assert grouped() in (EDEV, EUNSUP)
        assert grouped(row=G, rows=50) in (EDEV, EUNSUP)
    assert L.qgemm_f8_grouped(None, None) == ENULL
    for n in ("w_packed", "w_scale", "xq", "x_scale", "offsets", "Y"):
        assert grouped(**{n: None}) == ENULL
    for kw in [dict(ldx=112), dict(ldx=136), dict(ldxs=2), dict(y_type=3), dict(ldy=16), dict(ldy=22), dict(M=0), dict(K=0),
               dict(experts=0), dict(experts=1025), dict(rows=0), dict(x_rows=0), dict(rows=4194304, x_rows=4194304),
               dict(x_rows=4194304), dict(x_rows=6), dict(M=65537, ldy=65540, rows=65537, x_rows=65537),
               dict(row=G, x_rows=4194303, ldx=1040), dict(row=G, x_rows=4194303, ldxs=260)]:
        assert grouped(**kw) == ESHAPE, kw
    for kw in [dict(w_packed=A + 8), dict(xq=C + 8), dict(x_scale=D + 4), dict(Y=E + 8), dict(w_scale=B + 2), dict(bias=G + 1),
               dict(offsets=F + 2), dict(row=G + 2)]:
        assert grouped(**kw) == EALIGN, kw
    for n in ("w_packed", "w_scale", "xq", "x_scale", "offsets"):
        assert grouped(**{n: E}) == ESHAPE
    assert grouped(row=E + 16) == ESHAPE and grouped(bias=E + 16) == ESHAPE


def experts_out(**kw):
    d = dict(expert=B, weight=C, position=D, row=E, offsets=F)
    d.update(kw)
    return qg._ExpertsOut(*[d[n] for n, _ in qg._ExpertsOut._fields_])


def test_select_validation(L):
    def f(logits=A, t=0, ld=60, N=10, E=60, k=4, normalize=0, scale=1.0, ws=None, wb=0, out=None, **kw):
        o = experts_out(**kw) if out is None else out
        return L.logits_expert_select(logits, t, ld, N, E, k, normalize, scale, ws, wb, ctypes.byref(o), None)

    if no_gpu():
        assert f() in (EDEV, EUNSUP)
        assert f(logits=A + 2, t=2, ld=61) in (EDEV, EUNSUP)
    assert f(logits=None) == ENULL and L.logits_expert_select(A, 0, 60, 10, 60, 4, 0, 1.0, None, 0, None, None) == ENULL
    for n in ("expert", "weight", "position", "row", "offsets"):
        assert f(**{n: None}) == ENULL
        assert f(**{n: B + 2}) == EALIGN
        assert f(**{n: A}) == ESHAPE
    for kw in [dict(t=3), dict(ld=59), dict(ld=1 << 38), dict(N=0), dict(E=0), dict(E=1025, ld=1025), dict(k=0), dict(k=61), dict(E=40, k=33),
               dict(N=4194303, k=4), dict(normalize=2), dict(scale=float("inf")), dict(scale=float("nan")), dict(expert=C)]:
        assert f(**kw) == ESHAPE, kw
    assert f(logits=A + 2) == EALIGN
    need = L.logits_expert_select_workspace_bytes(1000, 60, 4)
    assert need > 0 and f(N=1000) == EWS and f(N=1000, ws=G, wb=need - 1) == EWS
    assert f(N=1000, ws=G + 8, wb=need) == EALIGN and f(N=1000, ws=A, wb=need) == ESHAPE and f(N=1000, ws=E, wb=need) == ESHAPE


def test_combine_validation(L):
    #       Y, y_type, ldy, rows, position, weight, k, add, ldadd, out, out_type, ldo, N, M, stream
    good = [A, 2, 50, 30, B, C, 3, D, 50, E, 2, 50, 10, 50, None]
    bad = refuser(L.qg_expert_combine, good)
    if no_gpu():
        assert bad() in (EDEV, EUNSUP)
        assert bad((9, D)) in (EDEV, EUNSUP)  # onto add itself
        assert bad((0, A + 2), (9, E + 2)) in (EDEV, EUNSUP)
        assert bad((7, None), (8, 0)) in (EDEV, EUNSUP)
    assert [bad((i, None)) for i in (0, 4, 5, 9)] == [ENULL] * 4
    for pairs in [[(1, 3)], [(10, -1)], [(2, 49)], [(8, 49)], [(11, 49)], [(2, 1 << 40)], [(3, 0)], [(6, 0)], [(6, 33)], [(12, 0)],
                  [(13, 0)], [(12, 4194304)], [(3, 4194304)], [(12, 4194303), (13, 1 << 14), (2, 1 << 14), (8, 1 << 14), (11, 1 << 14)]]:
        assert bad(*pairs) == ESHAPE, pairs
    assert bad((0, A + 1)) == EALIGN and bad((7, D + 1)) == EALIGN and bad((9, E + 1)) == EALIGN
    assert bad((4, B + 2)) == EALIGN and bad((5, C + 2)) == EALIGN
    for i in (0, 4, 5):
        assert bad((9, good[i])) == ESHAPE
    assert bad((9, D + 2)) == ESHAPE and bad((9, D), (8, 60)) == ESHAPE


def test_binding_refuses_host_tensors_and_other_types():
    f8 = torch.float8_e4m3fn
    q, s = torch.zeros(4, 128).to(f8), torch.zeros(4, 4)
    for call in (lambda: qg.pack_f8(q), lambda: qg.quantize_f8_rows(torch.zeros(4, 128)), lambda: qg.expert_combine(s, s, s),
                 lambda: qg.qgemm_f8(torch.zeros(4096, dtype=torch.uint8), s, q, s, 16, 128),
                 lambda: qg.qgemm_f8_grouped(torch.zeros(4096, dtype=torch.uint8), s, q, s, 16, 128, torch.zeros(2, dtype=torch.int32)),
                 lambda: qg.logits_expert_select(s, 2)):
        with pytest.raises(ValueError, match="on the GPU"):
            call()
    with pytest.raises(ValueError, match="must be torch.float32 or torch.float16 or torch.bfloat16|on the GPU"):
        qg.quantize_f8_rows(torch.zeros(4, 128, dtype=torch.float64))

"""CPU-side checks of the int8 product's and the beam search's C entry points: sizes
and the refusals, none of which reaches a device."""
import ctypes

import pytest
import torch

import quantized_gemv_argmax_amd as qg

OK, ENULL, ESHAPE, EALIGN, EWS, EDEV, EUNSUP = range(7)
A, B, C, D, E, F = (0x10000000 * i for i in range(1, 7))  # device addresses that nothing dereferences


@pytest.fixture(scope="module")
def L():
    return qg.lib()


def no_gpu():
    return not torch.cuda.is_available()


def test_i8_sizes(L):
    assert L.qg_i8_bytes(16, 64) == 1024
    assert L.qg_i8_bytes(17, 65) == 2 * 2 * 1024
    assert L.qg_i8_bytes(152064, 3584) == 152064 * 3584
    for m, k in [(0, 64), (16, 0), (4194304, 64), (16, 131072)]:
        assert L.qg_i8_bytes(m, k) == 0
        assert L.qgemm_i8_workspace_bytes(m, k, 4) == 0
    assert L.qgemm_i8_workspace_bytes(16, 64, 0) == 0


def test_pack_validation(L):
    f = L.qg_pack_i8
    #  wq, ldw, dst, M, K, stream
    assert f(None, 64, B, 16, 64, None) == ENULL
    assert f(A, 64, None, 16, 64, None) == ENULL
    assert f(A, 63, B, 16, 64, None) == ESHAPE
    assert f(A, 64, B, 0, 64, None) == ESHAPE
    assert f(A, 131072, B, 16, 131072, None) == ESHAPE
    assert f(A, 64, B + 8, 16, 64, None) == EALIGN
    assert f(A, 64, A + 512, 16, 64, None) == ESHAPE  # overlap
    if no_gpu():
        assert f(A + 1, 65, B, 16, 64, None) in (EDEV, EUNSUP)  # weights need no alignment


def test_quantize_validation(L):
    f = L.qg_quantize_i8_rows
    #  x, type, ldx, N, K, q, ldq, scale, stream
    good = [A, 0, 100, 4, 100, B, 128, C, None]
    if no_gpu():
        assert f(*good) in (EDEV, EUNSUP)
        assert f(A + 2, 1, 101, 4, 100, B, 144, C, None) in (EDEV, EUNSUP)

    def bad(i, v):
        a = list(good)
        a[i] = v
        return f(*a)

    assert [bad(i, None) for i in (0, 5, 7)] == [ENULL] * 3
    assert bad(1, 3) == ESHAPE and bad(1, -1) == ESHAPE
    assert bad(2, 99) == ESHAPE and bad(2, 1 << 40) == ESHAPE
    assert bad(3, 0) == ESHAPE and bad(3, 4194304) == ESHAPE
    assert bad(4, 0) == ESHAPE and bad(4, 131072) == ESHAPE
    assert bad(6, 112) == ESHAPE and bad(6, 136) == ESHAPE
    assert bad(0, A + 2) == EALIGN and bad(5, B + 8) == EALIGN and bad(7, C + 2) == EALIGN
    assert bad(5, A + 16) == ESHAPE and bad(7, A + 8) == ESHAPE and bad(7, B + 128) == ESHAPE


def test_product_validation(L):
    f = L.qgemm_i8
    #  w, w_scale, xq, ldx, x_scale, bias, Y, type, ldy, M, K, N, ws, ws_bytes, stream
    good = [A, B, C, 128, D, None, E, 0, 20, 20, 100, 3, None, 0, None]
    if no_gpu():
        assert f(*good) in (EDEV, EUNSUP)

    def bad(*pairs):
        a = list(good)
        for i, v in pairs:
            a[i] = v
        return f(*a)

    assert [bad((i, None)) for i in (0, 1, 2, 4, 6)] == [ENULL] * 5
    assert bad((3, 112)) == ESHAPE and bad((3, 136)) == ESHAPE and bad((3, 1 << 40)) == ESHAPE
    assert bad((7, 3)) == ESHAPE and bad((7, -1)) == ESHAPE
    assert bad((8, 16)) == ESHAPE and bad((8, 22)) == ESHAPE
    assert bad((9, 0)) == ESHAPE and bad((10, 0)) == ESHAPE and bad((11, 0)) == ESHAPE
    assert bad((9, 4194304)) == ESHAPE and bad((10, 131072)) == ESHAPE and bad((11, 4194304)) == ESHAPE
    assert bad((8, 65540), (9, 65537), (11, 65537)) == ESHAPE  # M N over 2^32
    for i in (0, 2, 6):
        assert bad((i, good[i] + 8)) == EALIGN
    assert bad((1, B + 2)) == EALIGN and bad((4, D + 1)) == EALIGN and bad((5, F + 2)) == EALIGN
    for i in (0, 1, 2, 4):  # Y over an input
        assert bad((6, good[i])) == ESHAPE
    assert bad((5, E + 16)) == ESHAPE
    need = L.qgemm_i8_workspace_bytes(3584, 18944, 64)
    if need:
        big = [(3, 18944), (8, 3584), (9, 3584), (10, 18944), (11, 64), (6, 0x100000000)]
        assert bad(*big) == EWS
        assert bad(*big, (12, F), (13, need - 1)) == EWS
        assert bad(*big, (12, F + 8), (13, need)) == EALIGN


def beam_in(**kw):
    d = dict(logits=A, logits_type=0, ld=100, batch=2, beams=3, vocab=100, score=B, finished=None, length=None,
             length_penalty=0.0, eos=-1)
    d.update(kw)
    return qg._BeamIn(*[d[n] for n, _ in qg._BeamIn._fields_])


def beam_out(**kw):
    d = dict(token=C, parent=C + 4096, score=C + 8192, finished=None, length=None)
    d.update(kw)
    return qg._BeamOut(*[d[n] for n, _ in qg._BeamOut._fields_])


def test_select_sizes(L):
    f = L.logits_beam_select_workspace_bytes
    assert f(0, 2, 3, 100, 3) > 0
    for bad in [(3, 2, 3, 100, 3), (0, 0, 3, 100, 3), (0, 2, 0, 100, 3), (0, 2, 33, 100, 3), (0, 2, 3, 0, 3),
                (0, 2, 3, 262145, 3), (0, 2, 3, 100, 0), (0, 2, 3, 100, 65), (0, 1 << 20, 3, 100, 3)]:
        assert f(*bad) == 0, bad
    assert f(0, 16, 8, 152064, 8) < 8 << 20  # a small share of the logits


def test_select_validation(L):
    f = L.logits_beam_select
    need = L.logits_beam_select_workspace_bytes(0, 2, 3, 100, 3)

    def call(i=None, o=None, n=3, ws=D, wb=need):
        i, o = i or beam_in(), o or beam_out()
        return f(ctypes.byref(i), n, ws, wb, ctypes.byref(o), None)

    if no_gpu():
        assert call() in (EDEV, EUNSUP)
        # a step in place: the input arrays as outputs, n == beams
        i = beam_in(finished=E, length=F, eos=4, length_penalty=1.0)
        assert call(i, beam_out(score=B, finished=E, length=F)) in (EDEV, EUNSUP)
        assert call(beam_in(ld=101, logits_type=2)) in (EDEV, EUNSUP)
    assert f(None, 3, D, need, ctypes.byref(beam_out()), None) == ENULL
    assert f(ctypes.byref(beam_in()), 3, D, need, None, None) == ENULL
    for k in ("logits", "score"):
        assert call(beam_in(**{k: None})) == ENULL
    for k in ("token", "parent", "score"):
        assert call(o=beam_out(**{k: None})) == ENULL
    for kw in [dict(logits_type=3), dict(batch=0), dict(beams=0), dict(beams=33), dict(vocab=0), dict(vocab=262145, ld=262145),
               dict(ld=99), dict(ld=1 << 40), dict(eos=100), dict(eos=-2), dict(finished=E), dict(length_penalty=16.5, length=F),
               dict(length_penalty=float("nan"), length=F), dict(batch=1 << 20)]:
        assert call(beam_in(**kw), wb=1 << 40) == ESHAPE, kw
    assert call(n=0) == ESHAPE and call(n=65) == ESHAPE
    assert call(beam_in(length_penalty=1.0)) == ENULL
    assert call(o=beam_out(length=F)) == ENULL
    assert call(beam_in(logits=A + 4)) == EALIGN
    assert call(beam_in(score=B + 2)) == EALIGN
    assert call(o=beam_out(token=C + 1)) == EALIGN
    assert call(ws=None) == EWS and call(wb=need - 1) == EWS and call(ws=D + 8) == EALIGN
    # overlaps: outputs with each other, with an input shifted or of another length, the workspace
    assert call(o=beam_out(parent=C + 20)) == ESHAPE
    assert call(o=beam_out(score=B + 4)) == ESHAPE
    assert call(o=beam_out(score=B), n=4, wb=1 << 20) == ESHAPE
    assert call(o=beam_out(token=B)) == ESHAPE
    assert call(o=beam_out(token=A)) == ESHAPE
    assert call(ws=C - 256 & ~15) == ESHAPE


def state(**kw):
    d = dict(src=A, dst=B, src_row=1024, dst_row=1024, src_outer=0, dst_outer=0, outer=1, span=1024)
    d.update(kw)
    return qg._BeamState(*[d[n] for n, _ in qg._BeamState._fields_])


def test_reorder_validation(L):
    f = L.qg_beam_reorder

    def call(*states, parent=C, batch=2, bi=3, bo=3, count=None):
        arr = (qg._BeamState * max(1, len(states)))(*states)
        return f(ctypes.addressof(arr), len(states) if count is None else count, parent, batch, bi, bo, None)

    if no_gpu():
        for ok in [state(), state(dst=A), state(src_row=0), state(outer=4, span=64, src_outer=128, dst_outer=64, dst_row=256),
                   state(outer=4, span=64, src_outer=6144, dst_outer=384, src_row=64, dst_row=64), state(src=A + 1, span=7)]:
            assert call(ok) in (EDEV, EUNSUP)
        assert call(state(), bi=1, bo=5) in (EDEV, EUNSUP)
    assert f(None, 1, C, 2, 3, 3, None) == ENULL
    assert call(state(), parent=None) == ENULL
    assert call(state(src=None)) == ENULL and call(state(dst=None)) == ENULL
    assert call(state(), count=0) == ESHAPE
    assert call(*[state(dst=B + 0x100000 * i) for i in range(57)]) == ESHAPE
    for kw in [dict(bi=0), dict(bo=0), dict(bi=33), dict(bo=33), dict(batch=0), dict(batch=65536)]:
        assert call(state(), **kw) == ESHAPE, kw
    assert call(state(), parent=C + 2) == EALIGN
    for kw in [dict(span=0), dict(outer=0), dict(span=1 << 40), dict(src_row=-1), dict(dst_row=-16), dict(src_outer=1 << 41),
               dict(dst_row=1008), dict(outer=2, dst_outer=1008, dst_row=4096), dict(outer=2, dst_outer=1024, dst_row=1024),
               dict(outer=2, dst_outer=2048, dst_row=1024),  # pieces of one row over the next one
               dict(dst=A, dst_row=2048), dict(dst=A + 64), dict(dst=A - 64), dict(dst=C - 64)]:
        assert call(state(**kw)) == ESHAPE, kw
    assert call(state(dst=A), bi=3, bo=2) == ESHAPE
    assert call(state(outer=1 << 30, span=1, src_outer=1 << 40, dst_outer=1 << 40, src_row=1, dst_row=1)) == ESHAPE
    # one result twice, a result that another state reads
    assert call(state(), state(src=D)) == ESHAPE
    assert call(state(), state(src=B, dst=D)) == ESHAPE
    assert call(state(src=D, dst=E), state(dst=D)) == ESHAPE
    if no_gpu():
        assert call(state(), state(dst=D)) in (EDEV, EUNSUP)  # one source twice is fine
    assert call(state(span=1 << 36, src_row=1 << 36, dst_row=1 << 36, dst=1 << 45)) == ESHAPE  # 2^32 columns of 16 bytes


def test_reorder_check_refuses_alike_and_launches_nothing(L):
    def call(*states, bi=3, bo=3, parent=C):
        arr = (qg._BeamState * len(states))(*states)
        return L.qg_beam_reorder_check(ctypes.addressof(arr), len(states), parent, 2, bi, bo)

    assert call(state()) == OK and call(state(), state(dst=D)) == OK  # without a device, too
    assert call(state(), state(src=D)) == ESHAPE and call(state(dst=C - 64)) == ESHAPE
    assert call(state(dst=A), bo=2) == ESHAPE and call(state(span=0)) == ESHAPE
    assert call(state(src=None)) == ENULL and call(state(), parent=C + 2) == EALIGN
    assert call(*[state(dst=B + 0x100000 * i) for i in range(57)]) == ESHAPE
    assert b"57" in L.qg_last_error()

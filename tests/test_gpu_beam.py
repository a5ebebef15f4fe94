"""GPU parity of the beam selection and the state reordering (logits_beam_select,
beam_reorder) against 64-bit references: tokens, parents, flags, lengths and moved
rows exactly, scores to their one rounding to float32 (plus 1e-12 of the double
arithmetic on both sides: under 2^18 terms, each within 2^-52)."""
import numpy as np
import pytest
import torch

import quantized_gemv_argmax_amd as qg
from tests import beamref
from tests.gpu_helpers import DEV, case, to_dev

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def check_selection(out, ref, what, length=True):
    torch.cuda.synchronize()
    for f in ("token", "parent", "finished") + (("length",) if length else ()):
        got = getattr(out, f).cpu().numpy()
        assert np.array_equal(got.astype(np.int64), ref[f].astype(np.int64)), f"{what}: {f}\n{got}\n{ref[f]}"
    s, r = out.score.double().cpu().numpy(), ref["score"]
    fin = np.isfinite(r)
    assert np.array_equal(s[~fin], r[~fin]), what
    assert np.all(np.abs(s[fin] - r[fin]) <= (2.0 ** -24 + 1e-12) * np.abs(r[fin]) + 1e-12), what


def logits_case(rows, V, kind, rng, t):
    z = rng.standard_normal((rows, V)).astype(np.float32) * 2.5
    big = np.float32(np.finfo(np.float16).max if t == "f16" else np.finfo(np.float32).max)
    low = float(torch.finfo(TYPES[t]).min)
    if kind == "ties":
        z = rng.integers(-2, 3, (rows, V)).astype(np.float32)
    elif kind == "flat":
        z[:] = 0.25
    elif kind == "masked":
        z[rng.random((rows, V)) < 0.9] = -np.inf
        z[0] = -np.inf
        if rows > 1:
            z[1] = -np.inf
            z[1, V // 2] = 3.0
    elif kind == "special":
        z[rng.random((rows, V)) < 0.2] = -np.inf
        z[rng.random((rows, V)) < 0.2] = np.nan
        z[rng.random((rows, V)) < 0.1] = -0.0
        z[rng.random((rows, V)) < 0.1] = 0.0
        z[rng.random((rows, V)) < 0.1] = low
        z[-1] = low
        if rows > 2:
            z[rows // 2, : max(1, V // 3)] = np.inf
            z[0] = big
    elif kind == "sorted":
        z = np.sort(z, axis=1)
    elif kind == "reversed":
        z = -np.sort(-z, axis=1)
    return to_dev(z).to(TYPES[t])


def run_select(B, W, V, n, kind, t, seed, finished=False, alpha=0.0, ld=None, off=0):
    rng = np.random.default_rng(seed)
    zd = logits_case(B * W, V, kind, rng, t)
    if ld is not None:
        wide = torch.full((B * W, ld), 50.0, dtype=zd.dtype, device=DEV)  # what lies between rows would win
        wide[:, :V] = zd
        zd = wide[:, :V]
    score = (-rng.random((B, W)) * 20).astype(np.float32)
    fin = rng.random((B, W)) < 0.3 if finished else None
    ln = rng.integers(0, 90, (B, W)).astype(np.int32)
    eos = int(rng.integers(0, V))
    case(f"logits_beam_select B={B} W={W} V={V} n={n} {kind} {t} finished={finished} alpha={alpha} ld={ld} seed={seed}")
    out = qg.logits_beam_select(zd, to_dev(score), n, finished=None if fin is None else to_dev(fin), length=to_dev(ln),
                                eos=eos, length_penalty=alpha)
    z = zd.double().cpu().numpy().reshape(B, W, V)
    ref = beamref.beam_select(z, score, n, fin, ln, eos, alpha)
    check_selection(out, ref, f"{B}x{W}x{V} n={n} {kind} {t}")


@pytest.mark.parametrize("kind", ["normal", "ties", "flat", "masked", "special", "sorted", "reversed"])
@pytest.mark.parametrize("B,W,V,n", [(1, 1, 1, 1), (1, 1, 5, 8), (2, 3, 7, 6), (1, 4, 64, 8), (3, 2, 129, 64),
                                     (2, 5, 1000, 10), (1, 32, 777, 64), (4, 4, 5003, 4), (1, 2, 20000, 64)])
def test_select(B, W, V, n, kind):
    for i, t in enumerate(TYPES):
        run_select(B, W, V, n, kind, t, seed=B * 1000 + V + n + i, finished=i != 1, alpha=[0.0, 0.7, 1.5][i])


@pytest.mark.parametrize("t", list(TYPES))
def test_select_large_vocabulary(t):
    run_select(2, 4, 152064, 8, "normal", t, seed=5, finished=True, alpha=0.8)
    run_select(1, 3, 262144, 64, "special", t, seed=6)
    run_select(1, 3, 152064, 64, "flat", t, seed=7)


@pytest.mark.parametrize("t", list(TYPES))
def test_select_rows_at_any_alignment(t):
    for V, ld in [(1000, 1001), (333, 340), (5003, 5003), (17, 19), (4097, 4099), (1, 3)]:
        run_select(2, 4, V, 8, "normal", t, seed=V + ld, ld=ld)


def test_identical_beams_rank_the_lower_first():
    z = np.tile(np.random.default_rng(8).standard_normal(300).astype(np.float32), (6, 1))
    score = np.full((2, 3), -1.25, np.float32)
    case("logits_beam_select identical beams")
    out = qg.logits_beam_select(to_dev(z), to_dev(score), 9)
    ref = beamref.beam_select(z.astype(np.float64).reshape(2, 3, 300), score, 9)
    check_selection(out, ref, "identical", length=False)
    assert out.parent.cpu().tolist()[0] == [0, 1, 2] * 3 and out.length is None


def test_shifted_beams_tie_exactly():
    # a constant added to a row (a power of two grid) changes no probability: still ties
    base = (np.random.default_rng(9).integers(-64, 64, 500) / 16).astype(np.float32)
    z = np.stack([base, base + 32, base - 1024])
    case("logits_beam_select shifted beams")
    out = qg.logits_beam_select(to_dev(z), torch.zeros(1, 3, device=DEV), 9)
    p = out.parent.cpu().numpy()[0]
    ref = beamref.beam_select(z.astype(np.float64)[None], np.zeros((1, 3)), 9)
    check_selection(out, ref, "shifted", length=False)
    assert p.tolist() == ref["parent"][0].tolist()


def test_dead_and_finished_beams():
    rng = np.random.default_rng(10)
    z = rng.standard_normal((8, 50)).astype(np.float32)
    score = np.array([[0, -np.inf, -np.inf, -np.inf], [np.nan, -np.inf, -3, -np.inf]], np.float32)  # a first step
    case("logits_beam_select dead beams")
    out = qg.logits_beam_select(to_dev(z), to_dev(score), 60)
    ref = beamref.beam_select(z.astype(np.float64).reshape(2, 4, 50), score, 60)
    check_selection(out, ref, "dead", length=False)
    # every beam finished, one of them dead: fewer candidates than asked for
    fin = np.ones((2, 4), bool)
    ln = np.arange(8, dtype=np.int32).reshape(2, 4)
    out = qg.logits_beam_select(to_dev(z), to_dev(score), 4, finished=to_dev(fin), length=to_dev(ln), eos=7, length_penalty=1.0)
    ref = beamref.beam_select(z.astype(np.float64).reshape(2, 4, 50), score, 4, fin, ln, 7, 1.0)
    check_selection(out, ref, "all finished")


def test_select_in_place_graph_and_stream():
    B, W, V = 3, 4, 9001
    rng = np.random.default_rng(11)
    z = rng.standard_normal((B * W, V)).astype(np.float32) * 3
    score0 = (-rng.random((B, W)) * 5).astype(np.float32)
    fin0, ln0 = rng.random((B, W)) < 0.3, rng.integers(1, 9, (B, W)).astype(np.int32)
    zd = to_dev(z)
    out = qg.BeamSelection(B, W, DEV, True)
    out.score, out.finished, out.length = to_dev(score0), to_dev(fin0), to_dev(ln0)

    def step():
        qg.logits_beam_select(zd, out.score, W, finished=out.finished, length=out.length, eos=17, length_penalty=0.9, out=out)

    case("logits_beam_select in place, captured")
    step()  # (a call before the capture, then the state set back)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    s, f, ln = score0.astype(np.float64), fin0, ln0
    out.score.copy_(to_dev(score0)), out.finished.copy_(to_dev(fin0)), out.length.copy_(to_dev(ln0))
    for i in range(4):
        g.replay()
        torch.cuda.synchronize()
        ref = beamref.beam_select(z.astype(np.float64).reshape(B, W, V), s, W, f, ln, 17, 0.9)
        check_selection(out, ref, f"replay {i}")
        s, f, ln = out.score.cpu().numpy(), ref["finished"], ref["length"]
        other = torch.cuda.Stream()
        with torch.cuda.stream(other):  # a second call at once, with a workspace of its own
            again = qg.logits_beam_select(zd, to_dev(score0), 8)
        other.synchronize()
        check_selection(again, beamref.beam_select(z.astype(np.float64).reshape(B, W, V), score0, 8), "stream", length=False)


def test_select_refusals():
    z, s = torch.zeros(6, 100, device=DEV), torch.zeros(2, 3, device=DEV)
    f, ln = torch.zeros(2, 3, dtype=torch.bool, device=DEV), torch.ones(2, 3, dtype=torch.int32, device=DEV)
    qg.logits_beam_select(z, s, 6)
    for kw in [dict(n=0), dict(n=65), dict(n=3, eos=100), dict(n=3, eos=-2), dict(n=3, finished=f),
               dict(n=3, length_penalty=1.0), dict(n=3, length=ln, length_penalty=float("nan")),
               dict(n=3, length=ln, length_penalty=17.0)]:
        with pytest.raises(qg.QGError):
            qg.logits_beam_select(z, s, **kw)
    for a, b in [(z.double(), s), (z, s.double()), (z[:5], s), (z.cpu(), s), (z.t(), s), (z, s.t())]:
        with pytest.raises(ValueError):
            qg.logits_beam_select(a, b, 3)
    out = qg.BeamSelection(2, 3, DEV, False)
    out.token = out.parent
    with pytest.raises(qg.QGError):
        qg.logits_beam_select(z, s, 3, out=out)
    out = qg.BeamSelection(2, 2, DEV, False)
    out.score = s.view(-1)[:4].view(2, 2)  # in place needs n == beams
    with pytest.raises(qg.QGError):
        qg.logits_beam_select(z, s, 2, out=out)
    with pytest.raises(qg.QGError):
        qg.logits_beam_select(torch.zeros(6, 262145, device=DEV), s, 3)


# ------------------------------------------------------------------ reordering
def states_like(rng, rows, which):
    mk = lambda *shape: to_dev(rng.integers(-1000, 1000, shape).astype(np.int16))  # noqa: E731
    if which == "cache":       # (rows, heads, room, D), the filled part
        return [mk(rows, 4, 33, 64)[:, :, :21], mk(rows, 2, 20, 8)[:, :, :1]]
    if which == "rows":        # block tables, histories, odd sizes
        return [mk(rows, 7), mk(rows, 1), mk(rows, 3, 5), to_dev(rng.integers(0, 9, (rows, 5)).astype(np.int32)),
                to_dev(rng.integers(0, 2, (rows, 3)).astype(np.uint8)), to_dev(rng.integers(0, 9, rows).astype(np.int64))]
    if which == "sequence":    # positions first
        return [mk(50, rows, 4, 16)[:37].transpose(0, 1)]
    return [mk(rows, 1000) for _ in range(60)]


@pytest.mark.parametrize("which", ["cache", "rows", "sequence", "many"])
@pytest.mark.parametrize("B,W", [(1, 1), (1, 2), (3, 4), (2, 7), (5, 8), (2, 32), (1, 12)])
def test_reorder(B, W, which):
    rng = np.random.default_rng(B * 100 + W)
    states = states_like(rng, B * W, which)
    parent = rng.integers(0, W, (B, W)).astype(np.int32)
    parent[0, 0] = -1
    if W > 3:
        parent[-1, 2] = W
        parent[-1, 0], parent[-1, 1] = 1, 0  # a cycle
    before = [s.cpu().numpy() for s in states]
    case(f"beam_reorder B={B} W={W} {which}")
    outs = [torch.zeros_like(s) + 5 for s in states]
    zero = [o.cpu().numpy() for o in outs]
    got = qg.beam_reorder(states, to_dev(parent), out=outs)
    assert all(a is b for a, b in zip(got, outs))
    torch.cuda.synchronize()
    for s, o, b, z in zip(states, outs, before, zero):
        np.testing.assert_array_equal(o.cpu().numpy(), beamref.reorder(b, parent, W, z))
        np.testing.assert_array_equal(s.cpu().numpy(), b)
    qg.beam_reorder(states, to_dev(parent))
    torch.cuda.synchronize()
    for s, b in zip(states, before):
        np.testing.assert_array_equal(s.cpu().numpy(), beamref.reorder(b, parent, W, b))


def test_reorder_leaves_the_room_of_a_cache():
    full = torch.arange(6 * 3 * 10 * 4, dtype=torch.int32, device=DEV).view(6, 3, 10, 4)
    want = full.clone()
    parent = torch.tensor([[1, 1, 0], [2, 2, 2]], dtype=torch.int32, device=DEV)
    case("beam_reorder room of a cache")
    qg.beam_reorder([full[:, :, :7]], parent)
    rows = (torch.arange(2, device=DEV)[:, None] * 3 + parent).view(-1).long()
    want[:, :, :7] = want[:, :, :7][rows]
    assert torch.equal(full, want)
    qg.beam_reorder([full[:, :, :0]], parent)  # nothing cached yet
    assert torch.equal(full, want)


def test_reorder_expands_and_shrinks():
    rng = np.random.default_rng(12)
    one = to_dev(rng.standard_normal((2, 3, 9, 8)).astype(np.float32))   # one prompt an item
    parent = torch.zeros(2, 5, dtype=torch.int32, device=DEV)
    out = torch.zeros(10, 3, 12, 8, device=DEV)
    case("beam_reorder 1 -> 5 and 5 -> 2 beams")
    qg.beam_reorder([one], parent, out=[out[:, :, :9]])  # pieces of the result, whole rows of the state
    assert torch.equal(out[:, :, :9], one.repeat_interleave(5, 0)) and int(out[:, :, 9:].count_nonzero()) == 0
    p = torch.tensor([[4, 0], [3, 3]], dtype=torch.int32, device=DEV)
    less = torch.empty(4, 3, 9, 8, device=DEV)
    qg.beam_reorder([out[:, :, :9]], p, out=[less])
    assert torch.equal(less, out[:, :, :9][torch.tensor([4, 0, 8, 8], device=DEV)])


def test_reorder_graph_replays():
    rng = np.random.default_rng(13)
    s0 = rng.standard_normal((8, 2, 30, 16)).astype(np.float32)
    state, parent = to_dev(s0), torch.zeros(2, 4, dtype=torch.int32, device=DEV)
    g = torch.cuda.CUDAGraph()
    case("beam_reorder captured")
    with torch.cuda.graph(g):
        qg.beam_reorder([state[:, :, :20]], parent)
    want = s0.copy()
    for i in range(4):
        p = rng.integers(0, 4, (2, 4)).astype(np.int32)
        parent.copy_(to_dev(p))
        g.replay()
        torch.cuda.synchronize()
        want[:, :, :20] = beamref.reorder(want[:, :, :20], p, 4, want[:, :, :20])
        np.testing.assert_array_equal(state.cpu().numpy(), want)


def test_reorder_refusals():
    s, p = torch.zeros(6, 8, device=DEV), torch.zeros(2, 3, dtype=torch.int32, device=DEV)
    for bad in [([], p, None), ([s], p.long(), None), ([s[:5]], p, None), ([s], p[:, :2].contiguous(), None),
                ([s], p, []), ([s], p, [s.double()]), ([s], p, [s[:4]]), ([s.cpu()], p, None),
                ([torch.zeros(6, 4, 4, 4, device=DEV)[:, :3, :3, :3]], p, None), ([s], p[:, ::2], None)]:
        with pytest.raises(ValueError):
            qg.beam_reorder(bad[0], bad[1], out=bad[2])
    with pytest.raises(qg.QGError):  # rows of the result on top of each other
        qg.beam_reorder([s], p, out=[torch.zeros(1, 8, device=DEV).expand(6, 8)])
    with pytest.raises(qg.QGError):  # one state twice
        qg.beam_reorder([s, s], p)
    both = torch.zeros(9, 8, device=DEV)
    with pytest.raises(qg.QGError):
        qg.beam_reorder([both[:6]], p, out=[both[3:]])
    with pytest.raises(qg.QGError):
        qg.beam_reorder([p.view(6, 1)], p)


# ------------------------------------------------------------------ a run of all of them
def test_beam_search_run():
    """Six steps of beam search over a small int8 model (one projection and a head): rows
    quantized, products, selection in place and the states' reordering, each step
    against the 64-bit references on the step's own logits; the histories that the
    reordering keeps are those that following the parents gives."""
    B, W, D, V, steps, eos = 2, 4, 192, 1003, 6, 5
    rng = np.random.default_rng(14)
    emb = rng.standard_normal((V, D)).astype(np.float32)
    ed = to_dev(emb)
    w1, s1 = qg.quantize_i8_rows(to_dev((rng.standard_normal((D, D)) / 8).astype(np.float32)))
    w2, s2 = qg.quantize_i8_rows(to_dev((rng.standard_normal((V, D)) / 4).astype(np.float32)))
    p1, p2 = qg.pack_i8(w1[:, :D]), qg.pack_i8(w2[:, :D])
    hidden = to_dev(np.repeat(rng.standard_normal((B, D)).astype(np.float32), W, 0))
    out = qg.BeamSelection(B, W, DEV, True)
    first = np.full((B, W), -np.inf, np.float32)
    first[:, 0] = 0
    out.score, out.finished, out.length = to_dev(first), torch.zeros(B, W, dtype=torch.bool, device=DEV), \
        torch.zeros(B, W, dtype=torch.int32, device=DEV)
    history = torch.full((B * W, steps), -1, dtype=torch.int32, device=DEV)
    mirror = np.full((B * W, steps), -1, np.int32)
    s, f, ln = first, np.zeros((B, W), bool), np.zeros((B, W), np.int32)
    for t in range(steps):
        case(f"beam search step {t}")
        xq, xs = qg.quantize_i8_rows(hidden)
        h = torch.tanh(qg.qgemm_i8(p1, s1, xq, xs, D, D)[:, :D])
        hq, hs = qg.quantize_i8_rows(h)
        logits = qg.qgemm_i8(p2, s2, hq, hs, V, D)[:, :V]
        # the products, from the quants that were used
        yr, p = beamref.product(hq[:, :D].cpu().numpy(), hs.cpu().numpy(), w2[:, :D].cpu().numpy(), s2.cpu().numpy())
        assert np.all(np.abs(logits.double().cpu().numpy() - yr) <= beamref.product_tolerance(yr, p, 0.0, 2.0 ** -149))
        z = logits.double().cpu().numpy().reshape(B, W, V)
        qg.logits_beam_select(logits, out.score, W, finished=out.finished, length=out.length, eos=eos, length_penalty=0.6,
                              out=out)
        ref = beamref.beam_select(z, s, W, f, ln, eos, 0.6)
        check_selection(out, ref, f"step {t}")
        s, f, ln = out.score.cpu().numpy(), ref["finished"], ref["length"].astype(np.int32)
        par = ref["parent"].astype(np.int32)
        qg.beam_reorder([hidden, history], out.parent)
        mirror = beamref.reorder(mirror, par, W, mirror)
        mirror[:, t] = ref["token"].reshape(-1)
        history[:, t] = out.token.view(-1)
        torch.cuda.synchronize()
        np.testing.assert_array_equal(history.cpu().numpy(), mirror)
        hidden = torch.tanh(hidden + ed[out.token.view(-1).clamp(min=0).long()])


def test_signalling_nans_are_masked():
    z = np.random.default_rng(15).standard_normal((2, 5000)).astype(np.float32)
    bits = z.view(np.uint32)
    bits[0, [0, 7, 4999]] = 0x7F800001   # signalling NaNs of both signs
    bits[1, ::3] = 0xFFA00000
    case("logits_beam_select signalling NaNs")
    out = qg.logits_beam_select(to_dev(bits.view(np.int32)).view(torch.float32), torch.zeros(1, 2, device=DEV), 20)
    ref = beamref.beam_select(z.astype(np.float64)[None], np.zeros((1, 2)), 20)
    check_selection(out, ref, "sNaN", length=False)


@pytest.mark.parametrize("kind", ["normal", "flat", "special"])
@pytest.mark.parametrize("B,W,V,n", [(40, 8, 20000, 16), (70, 5, 9001, 10), (300, 1, 30000, 64), (16, 32, 33333, 32)])
def test_select_many_rows(B, W, V, n, kind):
    # enough rows for the longer segments
    for i, t in enumerate(TYPES):
        run_select(B, W, V, n, kind, t, seed=B + V + i, finished=i == 1, alpha=[0.0, 1.0, 0.0][i], ld=V + 3 * i)


@pytest.mark.parametrize("span", [1, 2, 3, 5, 8, 14, 15, 16, 17, 31, 33, 66, 271])
def test_reorder_any_span_and_alignment(span):
    # pieces of every length at odd addresses, in place: what surrounds them stays
    rng = np.random.default_rng(span)
    B, W, outer = 2, 6, 3
    base = to_dev(rng.integers(0, 256, (B * W, outer, span + 5)).astype(np.uint8))
    want = base.cpu().numpy().copy()
    parent = rng.integers(-1, W + 1, (B, W)).astype(np.int32)
    case(f"beam_reorder span={span}")
    qg.beam_reorder([base[:, :, 3:3 + span]], to_dev(parent))
    want[:, :, 3:3 + span] = beamref.reorder(want[:, :, 3:3 + span], parent, W, want[:, :, 3:3 + span])
    torch.cuda.synchronize()
    np.testing.assert_array_equal(base.cpu().numpy(), want)


def test_workspaces():
    # one workspace serves the selection and split products in turn, keeps what a captured
    # graph holds when it grows, and is refused by calls that need zeros (and theirs here)
    ws = qg.Workspace(DEV)
    z = to_dev(np.random.default_rng(16).standard_normal((8, 30000)).astype(np.float32))
    score = torch.zeros(2, 4, device=DEV)
    case("workspaces")
    sel = qg.logits_beam_select(z, score, 8)
    M, K, N = 256, 18944, 40
    w = torch.randint(-127, 128, (M, K), dtype=torch.int8, device=DEV)
    x = torch.randint(-127, 128, (N, K), dtype=torch.int8, device=DEV)
    wp, one_m, one_n = qg.pack_i8(w), torch.ones(M, device=DEV), torch.ones(N, device=DEV)
    assert qg.qgemm_i8_workspace_bytes(M, K, N) > 0
    y = qg.qgemm_i8(wp, one_m, x, one_n, M, K)
    out = qg.BeamSelection(2, 8, DEV, False)
    qg.logits_beam_select(z, score, 8, out=out, ws=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qg.logits_beam_select(z, score, 8, out=out, ws=ws)
    for _ in range(3):
        assert torch.equal(qg.qgemm_i8(wp, one_m, x, one_n, M, K, ws=ws), y)
        ws.ensure(2 * ws.nbytes())  # outgrown while a graph holds the old buffer
        out.token.fill_(-5)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.token, sel.token) and torch.equal(out.parent, sel.parent)
        assert torch.equal(out.score, sel.score)
    with pytest.raises(ValueError):
        qg.logits_topk(z[0].contiguous(), 20, ws=ws)
    zeros = qg.Workspace(DEV)
    qg.logits_topk(z[0].contiguous(), 20, ws=zeros)
    with pytest.raises(ValueError):
        qg.logits_beam_select(z, score, 8, ws=zeros)
    with pytest.raises(ValueError):
        qg.qgemm_i8(wp, one_m, x, one_n, M, K, ws=zeros)


def test_calls_from_several_threads():
    import threading
    z = to_dev(np.random.default_rng(17).standard_normal((4, 999)).astype(np.float32))
    want = qg.logits_beam_select(z, torch.zeros(1, 4, device=DEV), 4)
    got = []

    def work():
        got.append(qg.logits_beam_select(z, torch.zeros(1, 4, device=DEV), 4))
        torch.cuda.synchronize()

    case("logits_beam_select from two threads")
    ts = [threading.Thread(target=work) for _ in range(2)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert len(got) == 2 and all(torch.equal(r.token, want.token) for r in got)


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("V,n", [(97, 64), (255, 33), (1025, 64), (2244, 64), (4091, 17), (4096, 64), (4103, 64),
                                 (8185, 64), (8192, 3), (8201, 64)])
def test_select_short_rows(V, n, t):
    """Rows around the lengths at which the bound is taken differently, with and without
    room beside them."""
    for i, kind in enumerate(["normal", "ties", "masked", "special"]):
        run_select(2, 3, V, n, kind, t, seed=V + n + i, ld=V + 5 if i % 2 else None)


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("V,live,n", [(900, 5, 16), (5000, 0, 64), (20000, 40, 64), (152064, 100, 64), (152064, 3, 8)])
def test_select_masked_by_the_lowest_value(V, live, n, t):
    """Masked entries at the type's lowest finite value are values like others: they rank
    last, the lower token first."""
    rng = np.random.default_rng(V + live)
    z = torch.full((4, V), torch.finfo(TYPES[t]).min, dtype=TYPES[t])
    for row in z:
        at = torch.from_numpy(rng.choice(V, live, replace=False))
        row[at] = torch.from_numpy(rng.standard_normal(live) * 3).to(TYPES[t])
    score = (-rng.random((2, 2)) * 20).astype(np.float32)
    case(f"logits_beam_select lowest V={V} live={live} n={n} {t}")
    out = qg.logits_beam_select(z.to(DEV), to_dev(score), n)
    ref = beamref.beam_select(z.double().numpy().reshape(2, 2, V), score, n)
    check_selection(out, ref, f"lowest {V} {live} {n} {t}", length=False)


def test_workspace_of_another_device_and_wrapped_token():
    z, s = torch.zeros(6, 100, device=DEV), torch.zeros(2, 3, device=DEV)
    with pytest.raises(ValueError, match="workspace is on cpu"):
        qg.logits_beam_select(z, s, 3, ws=qg.Workspace("cpu"))
    M, K, N = 256, 8192, 64  # split along K
    assert qg.qgemm_i8_workspace_bytes(M, K, N) > 0
    w = qg.pack_i8(torch.zeros(M, K, dtype=torch.int8, device=DEV))
    xq, xs = torch.zeros(N, K, dtype=torch.int8, device=DEV), torch.ones(N, device=DEV)
    with pytest.raises(ValueError, match="workspace is on cpu"):
        qg.qgemm_i8(w, torch.ones(M, device=DEV), xq, xs, M, K, ws=qg.Workspace("cpu"))
    for eos in (2 ** 32 + 5, -(2 ** 32) - 1):  # not the token of its low 32 bits
        with pytest.raises(ValueError, match="eos"):
            qg.logits_beam_select(z, s, 3, eos=eos)


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("V,gap", [(5003, 0), (50257, 0), (333, 0), (1001, 2), (4096, 1), (9001, 3), (152063, 0)])
def test_equal_beams_tie_wherever_their_rows_start(V, gap, t):
    """Rows that are equal, or equal but for a constant, at every alignment that an odd
    vocabulary or stride gives them: with equal scores their candidates tie, and the
    lower beam's come first. Values are halves below 16 shifted to at most 108, exact in
    every type."""
    B, W, n = 2, 8, 16
    rng = np.random.default_rng(V + gap)
    for shifts in (np.zeros(W), np.array([0, 32, -100, 0, 64, 32, -32, 96])):
        base = rng.integers(-16, 16, (B, 1, V)) / 2
        z = torch.from_numpy((base + shifts[None, :, None]).reshape(B * W, V))
        wide = torch.full((B * W, V + gap), 50.0, dtype=TYPES[t], device=DEV)
        wide[:, :V] = z.to(TYPES[t]).to(DEV)
        zd = wide[:, :V]
        assert torch.equal(zd.double().cpu(), z)
        score = np.full((B, W), -1.25, np.float32)
        case(f"logits_beam_select ties V={V} gap={gap} {t} shifted={bool(shifts.any())}")
        out = qg.logits_beam_select(zd, to_dev(score), n)
        ref = beamref.beam_select(z.numpy().reshape(B, W, V), score, n)
        check_selection(out, ref, f"ties {V} {gap} {t}", length=False)
    z = rng.standard_normal((B, 1, V)).astype(np.float32) * 3  # values of full precision, beams alike
    z = torch.from_numpy(np.broadcast_to(z, (B, W, V)).reshape(B * W, V).copy()).to(TYPES[t])
    wide = torch.full((B * W, V + gap), 50.0, dtype=TYPES[t], device=DEV)
    wide[:, :V] = z.to(DEV)
    case(f"logits_beam_select ties V={V} gap={gap} {t} alike")
    out = qg.logits_beam_select(wide[:, :V], to_dev(score), n)
    ref = beamref.beam_select(z.double().numpy().reshape(B, W, V), score, n)
    check_selection(out, ref, f"alike {V} {gap} {t}", length=False)


@pytest.mark.parametrize("at,count", [(56, 57), (63, 64), (120, 130)])
def test_reorder_of_many_states_refuses_before_it_moves(at, count):
    """More states than one launch takes: a result given twice, one that another state
    reads, and one refused by itself, each beyond the first group. Nothing has moved."""
    rng = np.random.default_rng(at)
    all_ = to_dev(rng.integers(-99, 99, (count, 6, 8)).astype(np.int32))
    second = torch.full_like(all_, 7)
    parent = torch.tensor([[1, 2, 0], [2, 2, 1]], dtype=torch.int32, device=DEV)
    before = all_.clone()
    case(f"beam_reorder {count} states, refused at {at}")
    for first in (0, 3):
        states = list(all_.unbind())
        states[at] = states[first]
        with pytest.raises(ValueError, match="share a result"):
            qg.beam_reorder(states, parent)
        states, out = list(all_.unbind()), list(second.unbind())
        out[at] = out[first]
        with pytest.raises(ValueError, match="share a result"):
            qg.beam_reorder(states, parent, out=out)
        states[at], out = out[first], list(second.unbind())  # reads what the first group writes
        with pytest.raises(ValueError, match="share a result"):
            qg.beam_reorder(states, parent, out=out)
    states = list(all_.unbind())
    states[at] = parent.view(6, 1)  # a state over the parents
    with pytest.raises(qg.QGError):
        qg.beam_reorder(states, parent)
    states, out = list(all_.unbind()), list(second.unbind())
    both = torch.zeros(9, 8, dtype=torch.int32, device=DEV)
    states[at], out[at] = both[:6], both[3:]
    with pytest.raises(qg.QGError):
        qg.beam_reorder(states, parent, out=out)
    torch.cuda.synchronize()
    assert torch.equal(all_, before) and bool((second == 7).all())
    states = list(all_.unbind())
    states[at] = states[first]
    out = list(second.unbind())  # one source twice is fine
    qg.beam_reorder(states, parent, out=out)
    rows = torch.tensor([1, 2, 0, 5, 5, 4], device=DEV)
    assert all(torch.equal(o, s[rows]) for o, s in zip(out, states))
    qg.beam_reorder(list(all_.unbind()), parent)
    assert torch.equal(all_, before[:, rows])


def test_counts_beyond_32_bits_are_refused():
    # (of 2^32 + 3 the library would see 3)
    z, s = torch.zeros(6, 100, device=DEV), torch.zeros(2, 3, device=DEV)
    for n in (2 ** 32 + 3, 2 ** 31, -(2 ** 32) + 3):
        with pytest.raises(ValueError, match="does not fit 32 bits"):
            qg.logits_beam_select(z, s, n)
    many = torch.zeros(1, 1, dtype=torch.uint8, device=DEV).expand(2 ** 32 + 3, 1)
    with pytest.raises(ValueError, match="does not fit 32 bits"):
        qg.beam_reorder([many], torch.zeros(1, 3, dtype=torch.int32, device=DEV), out=[torch.zeros(3, 1, dtype=torch.uint8, device=DEV)])

"""GPU parity of the selection of experts and of their combination (logits_expert_select,
expert_combine) against 64-bit references, and a mixture-of-experts layer run with them."""
import numpy as np
import pytest
import torch

import quantized_gemv_argmax_amd as qg
from tests import f8ref
from tests.gpu_helpers import DEV, case, to_dev

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -133}


def check_select(z, k, normalize, scale, what):
    case(what)
    r = qg.logits_expert_select(z, k, normalize=normalize, scale=scale)
    torch.cuda.synchronize()
    e, w, p, row, o = f8ref.select(z.double().cpu().numpy(), k, normalize, scale)
    np.testing.assert_array_equal(r.offsets.cpu().numpy(), o, err_msg=what)
    np.testing.assert_array_equal(r.expert.cpu().numpy(), e, err_msg=what)
    np.testing.assert_array_equal(r.row.cpu().numpy(), row, err_msg=what)
    np.testing.assert_array_equal(r.position.cpu().numpy(), p, err_msg=what)
    # float32: two exponentials of differences (rounded: |d| 2^-24 relative, |d| up to 104 before it
    # underflows, and 2^-23 of their own), a sum of E terms in at most E / 64 + 6 additions, a quotient, a product
    E = z.shape[1]
    d = np.abs(np.log(np.maximum(w / np.maximum(w[:, :1], 1e-300), 1e-300)))
    tol = np.abs(w) * (2 * np.minimum(d, 104) + 8 + E / 64 + 6 + 4) * 2.0 ** -23 + 2.0 ** -126 * max(1.0, abs(scale))
    got = r.weight.double().cpu().numpy()
    assert (np.abs(got - w) <= tol).all(), (what, np.abs(got - w).max())


SELECTIONS = [(1, 1, 1), (1, 128, 8), (3, 7, 7), (45, 37, 3), (32, 64, 2), (33, 65, 4), (31, 129, 32), (64, 256, 8), (500, 8, 2),
              (257, 1024, 6), (4096, 128, 8), (2050, 60, 4), (9000, 16, 1), (20, 1000, 8), (300, 257, 1)]


@pytest.mark.parametrize("N,E,k", SELECTIONS)
def test_select(N, E, k):
    for i, t in enumerate(TYPES):
        g = torch.Generator(device=DEV).manual_seed(N * 7 + E + k + i)
        z = (torch.randn(N, E, generator=g, device=DEV) * 2).to(TYPES[t])
        check_select(z, k, i % 2 == 0, 1.0 if i < 2 else 2.5, f"logits_expert_select N={N} E={E} k={k} {t}")


@pytest.mark.parametrize("N", [20, 300])
def test_select_masks_and_ties(N):
    g = torch.Generator(device=DEV).manual_seed(N)
    inf = float("inf")
    for E, k in [(5, 5), (128, 8), (300, 6)]:
        z = torch.randint(-2, 3, (N, E), generator=g, device=DEV).float()  # ties everywhere
        z[:, E // 2] = -inf                      # an expert switched off
        z[3] = -inf                              # padding
        z[N - 1] = -inf
        z[4] = torch.finfo(torch.float32).min    # masked by the type's lowest value: all equal
        z[5, 1:] = -inf                          # one candidate
        z[6, 0], z[6, 1] = inf, inf              # count as the largest finite value, equal
        z[7] = float("nan")
        z[8, ::2] = float("nan")
        z[9] = 0.0
        z[9, ::2] = -0.0
        for normalize in (False, True):
            check_select(z, k, normalize, 1.0, f"logits_expert_select masked N={N} E={E} k={k} normalize={normalize}")
    check_select(torch.full((N, 9), -inf, device=DEV), 4, False, 1.0, f"logits_expert_select all masked N={N}")
    one = torch.full((N, 9), -inf, device=DEV)
    one[:, 4] = 1.0                              # everything to one expert
    check_select(one, 4, True, 1.0, f"logits_expert_select one expert N={N}")


@pytest.mark.parametrize("N,E,k", [(8193, 512, 3), (20011, 300, 4), (16385, 1024, 2), (70001, 37, 5)])
def test_select_long(N, E, k):
    """Rows whose expert's words are counted and ordered in parts, the last ones ragged, some rows masked."""
    g = torch.Generator(device=DEV).manual_seed(N)
    z = torch.randn(N, E, generator=g, device=DEV).half()
    z[:, 1] += 3                                 # one expert with most rows
    z[:, E - 1] = -float("inf")                  # and one with none
    z[N // 3: N // 2] = -float("inf")            # padding: the rows behind the last are told by -1
    check_select(z, k, N % 2 == 0, 1.0, f"logits_expert_select long N={N} E={E} k={k}")


def test_select_strided_rows_and_own_outputs():
    base = torch.randn(50, 203, device=DEV).bfloat16()
    check_select(base[:, 3:163], 6, True, 1.0, "logits_expert_select strided")
    z = base[:, 3:163].contiguous()
    out = qg.ExpertSelection(50, 160, 6, DEV)
    ws = qg.Workspace(DEV)
    assert qg.logits_expert_select(z, 6, normalize=True, out=out, ws=ws) is out
    again = qg.logits_expert_select(z, 6, normalize=True)
    for name in ("expert", "weight", "position", "row", "offsets"):
        assert torch.equal(getattr(out, name), getattr(again, name)), name


def check_combine(N, k, M, R, yt, ot, add, seed, inplace=False, off=0):
    case(f"expert_combine N={N} k={k} M={M} R={R} {yt} {ot} add={add}")
    g = torch.Generator(device=DEV).manual_seed(seed)
    y = torch.randn(R, M + off, generator=g, device=DEV).to(TYPES[yt])[:, off:]
    pos = torch.randint(-2, R + 2, (N, k), generator=g, device=DEV, dtype=torch.int32)
    w = torch.randn(N, k, generator=g, device=DEV)
    w[(pos < 0) | (pos >= R)] = float("nan")  # what is skipped may weigh anything
    a = torch.randn(N, M + off, generator=g, device=DEV).to(TYPES[ot])[:, off:] if add else None
    yn, an = y.double().cpu().numpy(), None if a is None else a.double().cpu().numpy()
    out = qg.expert_combine(y, pos, w, add=a, out=a if inplace else None, dtype=None if inplace or add else TYPES[ot])
    torch.cuda.synchronize()
    assert out.dtype == TYPES[ot] and out.shape == (N, M)
    ref, err = f8ref.combine(yn, pos.cpu().numpy(), w.cpu().numpy(), an)
    tol = err + (np.abs(ref) + err) * HALF[ot] + TINY[ot]
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()


COMBINATIONS = [(1, 1, 1, 1), (3, 2, 7, 5), (45, 3, 517, 135), (7, 8, 2048, 56), (1, 8, 4096, 8), (300, 6, 100, 1800), (5, 32, 33, 160),
                (2000, 9, 264, 999)]


@pytest.mark.parametrize("N,k,M,R", COMBINATIONS)
def test_combine(N, k, M, R):
    for i, yt in enumerate(TYPES):
        for j, ot in enumerate(TYPES):
            check_combine(N, k, M, R, yt, ot, (i + j) % 2 == 0, seed=N + M + i * 3 + j, inplace=i == j, off=(i + 2 * j) % 4)


def layer(x, logits, w1, s1, w2, s2, I, K, k, dtype, Ys=None):
    """A mixture-of-experts layer: down(silu(gate) * up) of each token's experts, weighted."""
    sel = qg.logits_expert_select(logits, k, normalize=True)
    xq, xs = qg.quantize_f8_rows(x)
    h = qg.qgemm_f8_grouped(w1, s1, xq, xs, 2 * I, K, sel.offsets, row=sel.row, dtype=dtype)
    hq, hs = qg.quantize_f8_rows(h[:, :2 * I], gated=True, count=sel.offsets[-1:])
    y = qg.qgemm_f8_grouped(w2, s2, hq, hs, K, I, sel.offsets, dtype=dtype)
    return qg.expert_combine(y, sel.position, sel.weight, add=x, M=K)


def layer_inputs(N, E, K, I, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(N, K, generator=g, device=DEV).bfloat16()
    z = torch.randn(N, E, generator=g, device=DEV)
    z[:, 1] = -float("inf")
    if N > 4:
        z[2] = -float("inf")  # a padded token
    w = {}
    for name, (m, kk) in (("1", (2 * I, K)), ("2", (K, I))):
        v = torch.randn(E, m, kk, generator=g, device=DEV) * kk ** -0.5
        s = torch.empty(E, -(-m // 128), -(-kk // 128), device=DEV)
        q = torch.empty_like(v)
        for i in range(s.shape[1]):
            for j in range(s.shape[2]):
                b = v[:, 128 * i:128 * i + 128, 128 * j:128 * j + 128]
                s[:, i, j] = b.abs().amax((1, 2)) / 448
                q[:, 128 * i:128 * i + 128, 128 * j:128 * j + 128] = b / s[:, i, j][:, None, None]
        w["q" + name], w["s" + name] = q.to(torch.float8_e4m3fn), s
    return x, z, w


def values(q, s):
    m, k = q.shape
    return q.double() * s.double().repeat_interleave(128, 0)[:m].repeat_interleave(128, 1)[:, :k]


@pytest.mark.parametrize("N,E,K,I,k", [(1, 8, 256, 128, 2), (7, 8, 200, 72, 3), (40, 16, 384, 256, 4), (600, 8, 256, 192, 2)])
def test_layer(N, E, K, I, k):
    """All five operators as they are used together, against the layer in float64 on the
    quantized weights: what differs is the activations' rounding to e4m3 (2^-4 of a value,
    twice) and bf16's, so the outputs' norms agree to a few hundredths."""
    x, z, w = layer_inputs(N, E, K, I, seed=N + K)
    p1, p2 = qg.pack_f8(w["q1"]), qg.pack_f8(w["q2"])
    case(f"layer N={N} E={E} K={K} I={I} k={k}")
    out = layer(x, z, p1, w["s1"], p2, w["s2"], I, K, k, torch.bfloat16)
    torch.cuda.synchronize()
    e, wt, _, _, _ = f8ref.select(z.double().cpu().numpy(), k, True)
    want = x.double().clone()
    for n in range(N):
        for j in range(k):
            if e[n, j] >= 0:
                h = values(w["q1"][int(e[n, j])], w["s1"][int(e[n, j])]) @ x[n].double()
                h = torch.nn.functional.silu(h[:I]) * h[I:]
                want[n] += float(wt[n, j]) * (values(w["q2"][int(e[n, j])], w["s2"][int(e[n, j])]) @ h)
    # relative to what the experts add: two roundings of at most 2^-4, 2^-4 / sqrt(3) in the mean
    added = (want - x.double()).norm()
    assert float((out.double() - want).norm()) <= 2 ** -4 * float(added) + 2 ** -8 * float(want.norm())
    if N > 4:
        assert torch.equal(out[2], x[2])  # no expert: the token itself


def test_layer_in_a_graph():
    """Captured once, replayed with other tokens, eager work between the replays; a small and
    a large batch, which take different forms."""
    for N in (5, 300):
        x, z, w = layer_inputs(N, 8, 256, 128, seed=N)
        p1, p2 = qg.pack_f8(w["q1"]), qg.pack_f8(w["q2"])
        args = (p1, w["s1"], p2, w["s2"], 128, 256, 2, torch.bfloat16)
        xs, zs = x.clone(), z.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            layer(xs, zs, *args)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        case(f"layer in a graph N={N}")
        with torch.cuda.graph(graph):
            out = layer(xs, zs, *args)
        for i in range(4):
            g = torch.Generator(device=DEV).manual_seed(100 + i)
            x2 = torch.randn(N, 256, generator=g, device=DEV).bfloat16()
            z2 = torch.randn(N, 8, generator=g, device=DEV)
            if i == 2:
                z2[:] = -float("inf")
                z2[:, 3] = 0.0  # all to one expert
            xs.copy_(x2)
            zs.copy_(z2)
            graph.replay()
            want = layer(x2, z2, *args)
            torch.cuda.synchronize()
            assert torch.equal(out, want), (N, i)


def test_layer_on_another_stream():
    x, z, w = layer_inputs(300, 8, 256, 128, seed=1)
    p1, p2 = qg.pack_f8(w["q1"]), qg.pack_f8(w["q2"])
    args = (p1, w["s1"], p2, w["s2"], 128, 256, 2, torch.bfloat16)
    want = layer(x, z, *args)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    case("layer on three streams at once")
    outs = []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(layer(x, z, *args))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_one_workspace_of_any_contents():
    """Selections that count, that do not and that need none, and products split along K, in turn on one workspace
    that holds garbage before every call."""
    ws = qg.Workspace(DEV, 1 << 24)
    g = torch.Generator(device=DEV).manual_seed(8)
    w = (torch.randn(300, 9000, generator=g, device=DEV) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    wp, wsc = qg.pack_f8(w), torch.rand(3, 71, generator=g, device=DEV) + 0.5
    case("one workspace of any contents")
    for N, E, k, cols in [(9000, 40, 3, 100), (300, 200, 8, 20), (40, 64, 2, 300), (20000, 16, 1, 70)]:
        z = torch.randn(N, E, generator=g, device=DEV)
        xq, xs = qg.quantize_f8_rows(torch.randn(cols, 9000, generator=g, device=DEV))
        want, y = qg.logits_expert_select(z, k), qg.qgemm_f8(wp, wsc, xq, xs, 300, 9000)[:, :300].clone()
        for fill in (0xff, 0x01, 0x80):
            ws.buf.fill_(fill)
            r = qg.logits_expert_select(z, k, ws=ws)
            for name in ("expert", "weight", "position", "row", "offsets"):
                assert torch.equal(getattr(r, name), getattr(want, name)), (N, E, k, name)
            ws.buf.fill_(fill)
            assert torch.equal(qg.qgemm_f8(wp, wsc, xq, xs, 300, 9000, ws=ws)[:, :300], y), cols
    assert not ws.outgrown

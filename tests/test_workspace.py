"""Workspaces of the binding: which calls may share one, and what they find in it."""
import numpy as np
import pytest
import torch

import quantized_gemv_argmax_amd as qg


def test_calls_that_need_zeros_find_them():
    # (buffers in host memory: only the rules are tested here)
    ws = qg.Workspace("cpu", 64)
    ws.serve(64, "counters")
    ws.buf.fill_(7)  # what the K-sliced products leave
    ws.served("counters")
    assert int(ws.serve(64, "zeros").buf.count_nonzero()) == 0
    ws.serve(64, "counters")
    ws.buf.fill_(7)
    ws.served("counters")  # a captured LM-head call finds zeros, too
    assert int(ws.buf.count_nonzero()) == 0
    ws.buf.fill_(7)  # a captured product, replayed
    assert int(ws.serve(64, "zeros").buf.count_nonzero()) == 0


def test_calls_of_one_kind_are_not_cleared():
    for kind in ("zeros", "counters", "scratch"):
        ws = qg.Workspace("cpu", 64)
        for _ in range(2):
            ws.serve(64, kind)
            ws.buf[5] = 1
            ws.served(kind)
        assert int(ws.serve(64, kind).buf[5]) == 1
        assert int(ws.clear().buf.count_nonzero()) == 0


@pytest.mark.parametrize("other", ["zeros", "counters"])
def test_undefined_contents_are_not_shared(other):
    for a, b in ((other, "scratch"), ("scratch", other)):
        ws = qg.Workspace("cpu")
        ws.serve(64, a)
        with pytest.raises(ValueError, match="give each kind its own"):
            ws.serve(64, b)
        ws.serve(64, a)  # goes on serving its own


def test_default_workspace_is_kept_for_calls_that_need_zeros(monkeypatch):
    monkeypatch.setattr(qg, "_default_ws", {})
    with pytest.raises(ValueError, match="give each kind its own"):
        qg.default_workspace("cpu:0").serve(64, "scratch")
    qg._ws(None, 64, "cpu:0")  # what the LM-head calls take


def test_outgrown_buffers_stay_smaller_than_the_current_one():
    ws = qg.Workspace("cpu")
    for need in range(1 << 20, 12 << 20, 1 << 18):  # shapes that grow step by step
        ws.serve(need, "zeros")
        assert ws.nbytes() >= need and int(ws.buf.count_nonzero()) == 0
        assert sum(b.numel() for b in ws.outgrown) < ws.nbytes()
    assert 0 < len(ws.outgrown) <= 4
    ws.buf[3] = 1
    assert not ws.release_outgrown().outgrown and int(ws.buf[3]) == 1


def test_a_buffer_made_in_inference_mode_can_be_cleared_outside():
    ws = qg.Workspace("cpu")
    with torch.inference_mode():
        ws.serve(64, "counters")
        ws.buf[0] = 1
    assert int(ws.serve(64, "zeros").buf[0]) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("first", ["product", "head", "topk"])
def test_products_and_heads_share_a_workspace(first):
    """K-sliced products, the LM head and the top-k on one workspace in every order, the
    products and the head captured as well: results are those of workspaces of their own."""
    import workloads
    from tests.gpu_helpers import DEV, case, packed_q4k, packed_q8_0, to_dev
    M, K, N = 3584, 18944, 32
    Y = torch.zeros((N, M), device=DEV)
    probs = [(packed_q4k(workloads.q4k_blocks(M, K, key=(95,)), M, K), to_dev(workloads.x_columns(K, N, key=(95,))), Y, M, K)]
    Mh, Kh = 20000, 1024
    wh = packed_q8_0(workloads.q8_0_blocks(Mh, Kh, key=(96,)), Mh, Kh)
    xh = to_dev((workloads.x_vector(Kh, key=(96,)) * 0.05).astype(np.float32))
    z = to_dev(np.random.default_rng(97).standard_normal(Mh).astype(np.float32))
    need = qg.qgemm_q4k_smalln_batch_workspace_bytes(probs)
    assert need > 0
    oi, ov = torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros(1, device=DEV)

    def product(ws):
        qg.qgemm_q4k_smalln_batch_ws(probs, ws)
        return [Y]

    def head(ws):
        qg.lmhead_argmax(wh, xh, Mh, Kh, out_index=oi, out_value=ov, ws=ws)
        return [oi, ov]

    def topk(ws):
        r = qg.logits_topk(z, 20, ws=ws)
        return [r.index, r.logit]

    def run(what, ws):
        for t in (Y, oi, ov):
            t.fill_(-3)
        out = [t.clone() for t in calls[what](ws)]
        torch.cuda.synchronize()
        return out

    calls = {"product": product, "head": head, "topk": topk}
    want = {}
    for what in calls:
        case(f"workspace of its own: {what}")
        want[what] = run(what, qg.Workspace(DEV, 8 << 20))
    ws = qg.Workspace(DEV, max(need, 8 << 20))

    def check(what, got):
        assert all(torch.equal(a, b) for a, b in zip(got, want[what])), what

    order = [first] + [w for w in calls if w != first]
    graphs = {}

    def capture(what):
        graphs[what] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[what]):
            calls[what](ws)

    case(f"shared workspace, {first} first")
    check(first, run(first, ws))
    if first != "topk":
        capture(first)  # before the workspace has served another kind
    for what in order + order[::-1] + order:
        case(f"shared workspace, {first} first: {what}")
        check(what, run(what, ws))
    for what in ("product", "head"):
        if what not in graphs:
            capture(what)
    for i in range(3):
        for what in ("product", "head", "head", "product"):
            case(f"shared workspace, {first} first: {what}, replay {i}")
            for t in (Y, oi, ov):
                t.fill_(-3)
            graphs[what].replay()
            torch.cuda.synchronize()
            check(what, [Y] if what == "product" else [oi, ov])
            check("topk", run("topk", ws))
            check(what, run(what, ws))

"""Calls of the norms around a block, the checkpoints and the gated feed-forward block that their
sizes, their company or their tensors make special: offsets past 32 bits, two threads at once, a
workspace of a larger batch, outputs in place, rows on any boundary, weights that train in bf16."""

import math
import threading

import pytest
import torch

import quantized_moe_grouped_route_gb300 as q
from quantized_moe_grouped_route_gb300 import qmoe
from tests.test_block_operators import (ROUND, TINY, U, _block_inputs, _case, _ffn_grads, _ffn_inputs,
                                        _forms, _gen, _near, _norm_call, _norm_grads, _norm_inputs,
                                        _rows, _train_block, _up)

pytestmark = pytest.mark.gpu


def _of_rows(c, s, rows):
    return dict(c, M=len(rows)), {k: t[rows] if t is not None and t.dim() == 2 and
                                  t.shape[0] == c["M"] else t for k, t in s.items()}


def test_norm_past_32_bits():
    """More than 2^31 elements: the last rows, each as it is alone (bounds of test_block_norm)."""
    H, dt = 4104, torch.bfloat16
    c = _case((1 << 31) // H + 20, H, gate="token")
    s = _norm_inputs(c, 1)
    out, normed, post, pre = _norm_call(c, s)
    rows = torch.tensor([0, c["M"] // 2, c["M"] - 2, c["M"] - 1], device="cuda")
    few, sf = _of_rows(c, s, rows)
    v, size, n64, post64, pre64 = _forms(few, sf)
    e = (0.5 * H + 16) * U
    ev = (e + 16 * U) * size
    _near(out[rows], v, ev + ROUND[dt] * (v.abs() + ev), "out")
    far = ev.norm(dim=1, keepdim=True) / v.norm(dim=1, keepdim=True) + e
    w = sf["pre"].double().abs()
    bound = w * pre64 * (ev + (1.01 * far + 16 * U) * v.abs())
    _near(normed[rows], n64, bound + ROUND[dt] * (n64.abs() + bound), "normed")
    # (of the sums over all tokens only that they are finite: they are tested where they are small)
    dy, dres, dgate, dpost, dpre = q.qmoe_block_norm_backward(
        normed, out, s["y"], out=out, gate=s["gate"], post_weight=s["post"], pre_weight=s["pre"],
        post_rstd=post, pre_rstd=pre)
    assert torch.isfinite(dpost).all() and torch.isfinite(dpre).all()
    want = _norm_grads(few, sf, out[rows], normed[rows], out[rows], post[rows], pre[rows])
    for name, t in (("dy", dy), ("dresidual", dres), ("dgate", dgate)):
        ref, bound = want[name]
        _near(t[rows], ref, bound + ROUND[t.dtype] * (ref.abs() + bound), name)


def test_checkpoint_past_32_bits():
    C = 4100
    M = (1 << 31) // C + 50
    x = torch.randn(M, C, device="cuda", dtype=torch.bfloat16)
    codes, scales = q.qmoe_checkpoint8(x)
    back = q.qmoe_checkpoint8_restore(codes, scales)
    rows = torch.tensor([0, M // 2, M - 1], device="cuda")
    one = q.qmoe_checkpoint8(x[rows])
    assert torch.equal(codes[rows], one[0]) and torch.equal(scales[rows], one[1])
    assert torch.equal(back[rows], q.qmoe_checkpoint8_restore(*one))


@pytest.mark.parametrize("bits", [16, 8])
def test_gated_ffn_past_32_bits(bits):
    """u beside g has more than 2^31 elements (bounds of the tests of small batches)."""
    H, I, dt = 72, 4096, torch.bfloat16
    M = (1 << 31) // (2 * I) + 300
    x, w13, w2 = _ffn_inputs(M, H, I, dt)
    out, saved = q.qmoe_gated_ffn_saved(x, w13, w2, checkpoint=bits)
    rows = torch.tensor([0, M // 2, M - 300, M - 1], device="cuda")
    ug, eug, h, eh = _up("silu", math.inf, x[rows], w13)
    r, w = ROUND[dt], w2.double()
    eh = eh + r * (h.abs() + eh)
    ref = h @ w.t()
    bound = eh @ w.abs().t() + (I + 4) * 2 * U * ((h.abs() + eh) @ w.abs().t())
    _near(out[rows], ref, bound + r * (ref.abs() + bound), "out")
    if bits == 16:
        _near(saved[0][rows], ug, eug + r * (ug.abs() + eug), "kept")
        kept = saved[0][rows].double()
    else:
        step = torch.exp2(saved[1][rows].double() - 127).repeat_interleave(32, 1)
        kept = saved[0][rows].double() * step
        _near(kept, ug, step / 2 + eug, "kept")
    dx, dw13, dw2 = q.qmoe_gated_ffn_backward(out, x, w13, w2, saved)
    assert torch.isfinite(dw13).all() and torch.isfinite(dw2).all()
    want = _ffn_grads("silu", math.inf, out[rows], x[rows], w13, w2, kept[:, :I], kept[:, I:], dt)
    _near(dx[rows], *want["dx"], "dx")


@pytest.mark.parametrize("sizes", [((1, 1024, 512), (2, 2048, 256)), ((40, 1024, 512), (100, 512, 776)),
                                   ((300, 512, 512), (513, 264, 1032))])
def test_two_threads(sizes):
    """Each with a stream, a workspace and a problem of its own: the results it has alone.  (A thread's
    first call may be of any operator.)"""
    sides = []
    for M, H, I in sizes:
        x, w13, w2 = _ffn_inputs(M, H, I, torch.bfloat16)
        dout = _rows(_gen(M), M, H, torch.bfloat16)
        ws = torch.empty(q.qmoe_gated_ffn_workspace_size(M, H, I), dtype=torch.uint8, device="cuda")
        wb = torch.empty(q.qmoe_gated_ffn_backward_workspace_size(M, H, I), dtype=torch.uint8,
                         device="cuda")
        _, saved = q.qmoe_gated_ffn_saved(x, w13, w2)
        weight = torch.ones(H, device="cuda")

        def call(stream, x=x, w13=w13, w2=w2, dout=dout, ws=ws, wb=wb, saved=saved, weight=weight):
            y = q.qmoe_gated_ffn(x, w13, w2, workspace=ws, stream=stream)
            out, n, p, r = q.qmoe_block_norm(y, residual=x, post_weight=weight, pre_weight=weight,
                                             stream=stream)
            grads = q.qmoe_gated_ffn_backward(dout, x, w13, w2, saved, workspace=wb, stream=stream)
            return [y, out, n, p, r, *grads]
        sides.append((call, torch.cuda.Stream()))
    torch.cuda.synchronize()
    want = []
    for call, stream in sides:
        want.append(call(stream))
        stream.synchronize()
    start, wrong = threading.Barrier(2), [0, 0]

    def work(i):
        call, stream = sides[i]
        start.wait()
        try:
            for _ in range(40):
                got = call(stream)
                with torch.cuda.stream(stream):
                    wrong[i] += sum(not torch.equal(a, b) for a, b in zip(got, want[i]))
        except Exception as e:
            wrong[i] = e
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert wrong == [0, 0]


@pytest.mark.parametrize("H,I", [(512, 264), (1160, 1032)])
def test_a_workspace_serves_smaller_batches(H, I):
    most = 700
    n = q.qmoe_gated_ffn_workspace_size(most, H, I)
    sizes = [q.qmoe_gated_ffn_workspace_size(M, H, I) for M in range(0, most + 1)]
    assert sizes == sorted(sizes)
    for bits in (8, 16):
        sizes = [q.qmoe_gated_ffn_backward_workspace_size(M, H, I, bits) for M in range(0, most + 1)]
        assert sizes == sorted(sizes)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)
    for M in (700, 3, 90, 200, 1, 513):
        x, w13, w2 = _ffn_inputs(M, H, I, torch.bfloat16)
        got = q.qmoe_gated_ffn(x, w13, w2, workspace=ws)
        assert qmoe.qmoe_read_error(ws) == (qmoe.QMOE_OK, 0)
        assert torch.equal(got, q.qmoe_gated_ffn(x, w13, w2))


@pytest.mark.parametrize("H", [1001, 1000, 520, 7168])
@pytest.mark.parametrize("M", [5, 400])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_in_place(M, H, dtype):
    c = _case(M, H, dtype, gate="channel")
    s = _norm_inputs(c, 2)
    want = _norm_call(c, s)
    for k in ("y", "residual"):
        into = s[k].clone()
        got = _norm_call(c, dict(s, **{k: into}), out=into)
        assert got[0] is into
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("offset", [1, 2, 4])
@pytest.mark.parametrize("M,H", [(6, 512), (400, 512), (400, 104)])
def test_rows_on_any_boundary(M, H, offset):
    """The same rows at other addresses give the same results but for the order of their sums, and
    nothing around the outputs is written."""
    dt = torch.bfloat16
    c = _case(M, H, gate="full")
    s = _norm_inputs(c, 4)
    g = _gen(3)
    dout, dn = _rows(g, M, H, dt), _rows(g, M, H, dt)
    moved = {}
    for k, t in s.items():
        if t.dim() == 2:
            big = torch.full((M, H + 2 * offset), math.nan, dtype=dt, device="cuda")
            big[:, offset:offset + H] = t
            moved[k] = big[:, offset:offset + H]
        else:
            big = torch.full((H + 2 * offset,), math.nan, dtype=dt, device="cuda")
            big[offset:offset + H] = t
            moved[k] = big[offset:offset + H]
    guard = torch.full((M * H + 64,), 3.0, dtype=dt, device="cuda")
    into = guard[offset:offset + M * H].view(M, H)
    out, normed, post, pre = _norm_call(c, moved, out=into)
    assert (guard[:offset] == 3.0).all() and (guard[offset + M * H:] == 3.0).all()
    v, size, n64, post64, pre64 = _forms(c, s)
    e = (0.5 * H + 16) * U
    ev = (e + 16 * U) * size
    _near(out, v, ev + ROUND[dt] * (v.abs() + ev), "out")
    got = q.qmoe_block_norm_backward(dout, dn, moved["y"], out=out, gate=moved["gate"],
                                     post_weight=moved["post"], pre_weight=moved["pre"],
                                     post_rstd=post, pre_rstd=pre)
    want = _norm_grads(c, s, out, dout, dn, post, pre)
    for name, t in zip(("dy", "dresidual", "dgate", "dpost", "dpre"), got):
        ref, bound = want[name]
        _near(t, ref, bound + ROUND[t.dtype] * (ref.abs() + bound), name)
    big = torch.full((M, H + 2 * offset), math.inf, dtype=dt, device="cuda")
    big[:, offset:offset + H] = s["y"]
    for a, b in zip(q.qmoe_checkpoint8(big[:, offset:offset + H]), q.qmoe_checkpoint8(s["y"])):
        assert torch.equal(a, b)


def test_weights_that_train_in_bf16():
    """Gradients come in the leaves' own types, as casts of the explicit call's."""
    c = _case(33, 264, gate="token", sigmoid=True)
    s = _norm_inputs(c, 6)
    leaves = {k: t.clone().requires_grad_(True) for k, t in s.items()}
    out, n, post, pre = _norm_call(c, leaves)
    g = _gen(2)
    dout, dn = _rows(g, 33, 264, torch.bfloat16), _rows(g, 33, 264, torch.bfloat16)
    torch.autograd.backward([out, n], [dout, dn])
    want = q.qmoe_block_norm_backward(dout, dn, s["y"], out=out.detach(), gate=s["gate"],
                                      gating=q.QMOE_GATING_SIGMOID, post_weight=s["post"],
                                      pre_weight=s["pre"], post_rstd=post, pre_rstd=pre)
    for k, t in zip(("y", "residual", "gate", "post", "pre"), want):
        assert leaves[k].grad.dtype == torch.bfloat16
        assert torch.equal(leaves[k].grad, t.to(torch.bfloat16))


def test_a_gate_of_all_tokens():
    """One gate for all tokens (a stride of 0), whose gradient is the tokens' sum."""
    c = _case(50, 128, torch.float32, gate="token")
    s = _norm_inputs(c, 7)
    one = torch.tensor([[0.75]], device="cuda", requires_grad=True)
    out, *_ = _norm_call(c, dict(s, gate=one.expand(50, 1)))
    assert torch.equal(out, _norm_call(c, dict(s, gate=torch.full((50, 1), 0.75, device="cuda")))[0])
    out.sum().backward()
    v, *_ = _forms(dict(c, pre=False), dict(s, gate=torch.ones(50, 1, device="cuda"), residual=None))
    # a sum of 50 x 128 terms
    assert abs(float(one.grad) - float(v.sum())) <= 6400 * U * float(v.abs().sum())


def test_an_eager_step_after_a_captured_one():
    x, w = _block_inputs(20, 256, 392)
    leaves = {k: t.clone().requires_grad_(True) for k, t in dict(w, x=x).items()}

    def step():
        out, n = _train_block(leaves["x"], leaves, 16)
        return torch.autograd.grad(out.float().sum() + n.float().sum(), list(leaves.values()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    got = []
    for graph in graphs:
        with torch.cuda.graph(graph):
            got.append(step())
    for graph in graphs + graphs:
        graph.replay()
    for a, b, c, d in zip(want, *got, step()):
        assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(a, d)
    assert q.qmoe_default_read_error() == (qmoe.QMOE_OK, 0)

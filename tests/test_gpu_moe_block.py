"""The operators beside the layer run together: an MoE block (norm, layer, norm,
gate and residual) trained for a step, with 16-bit per-expert maps on the
layer's own groups, and all gradients clipped by their global norm."""
import math

import pytest
import torch

from mixture_experts_layer_40_b200 import inputs as I
from tests import helpers as H

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    from __graft_entry__ import build
    build()
    assert torch.cuda.is_available()


def a_layer(T=64, Hs=256, N=16, K=4, inter=256):
    from mixture_experts_layer_40_b200.layer import MoELayer, device_weights
    w = I.Workload("block", T=T, H=Hs, N=N, K=K, I=inter, bias_range=0.1)
    case = H.make_case(w)
    layer = MoELayer(T, Hs, N, K, inter, device_weights(w, case.pool, case.gate_w, "cuda"))
    return case, layer, torch.from_numpy(case.bias).cuda()


@pytest.mark.parametrize("res", [BF16, torch.float32])
def test_block_step(res):
    """Forward and backward of the block equal its parts called one by one; the
    residual path and the norms are held against float64 around the layer."""
    from mixture_experts_layer_40_b200.block import GradClip, MoEBlock
    case, layer, bias = a_layer()
    T, Hs = layer.T, layer.H
    gen = torch.Generator(device="cuda").manual_seed(0)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    pre, post, scale = 1 + 0.2 * rn(Hs), 1 + 0.2 * rn(Hs), 0.5 + 0.1 * rn(Hs)
    x, gate = H.x_to_device(case.x_bits).to(res), rn(T).sigmoid()
    block = MoEBlock(layer, pre, post, scale, alpha=0.5)
    r, u_next = block.forward(x, bias, gate, next_weight=post)
    assert layer.status() == 0
    norm = lambda v, w: v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6) * w  # noqa: E731
    # a bf16 rounding is half a step of 2^-7: eps / 2 = 2^-8 relative
    step = 2.0 ** -8
    u = norm(x.double(), pre.double())
    assert ((block.u.double() - u).abs() <= step * 1.01 * u.abs()).all()
    ref = x.double() + 0.5 * scale.double() * gate.double()[:, None] * norm(block.z.double(), post.double())
    slack = (step if res == BF16 else 0) * ref.abs() + 2.0 ** -17 * (ref.abs() + 4)
    assert ((r.double() - ref).abs() <= slack).all()
    un = norm(ref, post.double())
    assert ((u_next.double() - un).abs() <= step * un.abs() + 2.0 ** -15).all()

    dr = (rn(T, Hs) * 0.1).to(res)
    g = block.backward(dr)
    assert layer.status() == 0
    # dx - dr is what the layer's gradient gives through the first norm: against
    # the formula with the layer's own backward of the same dz
    xd = x.double().requires_grad_()
    z = block.z.double().requires_grad_()
    (0.5 * scale.double() * gate.double()[:, None] * norm(z, post.double()) * dr.double()).sum().backward()
    dz = z.grad
    du, dgates, dw13, dw2 = layer.backward(dz.to(BF16), block.u)
    (norm(xd, pre.double()) * du.double()).sum().backward()
    want = dr.double() + xd.grad
    # dz may round the other way in few places, which moves the FP8 layer's
    # gradients by single code steps: 2^-4 of their part
    assert ((g["dx"].double() - want).norm() / xd.grad.norm()) < 2.0 ** -4
    assert (g["w2"] - dw2).norm() <= 2.0 ** -4 * dw2.norm()
    assert (g["gates"] - dgates).norm() <= 2.0 ** -6 * dgates.norm()
    assert set(g) == {"dx", "gates", "gate", "pre_weight", "post_weight", "scale", "w13", "w2"}

    names = ["pre_weight", "post_weight", "scale", "w13", "w2"]
    before = {k: g[k].clone() for k in names}
    total = math.sqrt(sum(float((before[k].double() ** 2).sum()) for k in names))
    clip = GradClip([g[k] for k in names])
    assert abs(float(clip(total / 3)) - total) <= 1e-6 * total
    for k in names:
        assert torch.allclose(g[k], before[k] / 3, rtol=1e-5, atol=1e-12)


def test_sixteen_bit_experts_on_the_layers_groups():
    """An expert FFN in bf16 on the forward's permuted rows: the two grouped maps
    and all their gradients over the workspace's groups, whose padding rows hold
    anything."""
    from mixture_experts_layer_40_b200.block import GroupedLinear
    case, layer, bias = a_layer()
    x = H.x_to_device(case.x_bits)
    layer.forward(x, bias)
    G, L = layer.N + 1, layer.layout
    rows = layer.view("group_rows", torch.int32, (G,))
    start = layer.view("row_start", torch.int32, (G,))
    total = L.rows_total
    gen = torch.Generator(device="cuda").manual_seed(1)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(BF16)  # noqa: E731
    xr = torch.full((total, layer.H), float("nan"), dtype=BF16, device="cuda")
    token = layer.view("row_token", torch.int32, (L.routed_cap,)).long()
    spans = list(zip(start.tolist(), rows.tolist()))
    for s, c in spans[:-1]:
        xr[s:s + c] = x[token[s:s + c]]
    xr[L.routed_cap:L.routed_cap + layer.T] = x
    up = GroupedLinear(rn(G, 512, layer.H) / 16)
    down = GroupedLinear(rn(G, layer.H, 256) / 16)
    gu = up.forward(xr, rows, start)
    h = (torch.nn.functional.silu(gu[:, :256].float()) * gu[:, 256:].float()).to(BF16)
    y = down.forward(h, rows, start)
    dy = rn(total, layer.H)
    dh, dw2 = down.backward(dy, h, rows, start)
    dw2_twice = dw2.clone()
    down.backward(dy, h, rows, start, dw=dw2_twice, accumulate=True)
    dgu = rn(total, 512)
    dx, dw13 = up.backward(dgu, xr, rows, start)
    assert layer.status() == 0
    used = torch.zeros(total, dtype=torch.bool, device="cuda")
    for g, (s, c) in enumerate(spans):
        used[s:s + c] = True
        a, b = xr[s:s + c].double(), h[s:s + c].double()
        for got, want in [(gu[s:s + c], a @ up.weight[g].double().T),
                          (y[s:s + c], b @ down.weight[g].double().T),
                          (dh[s:s + c], dy[s:s + c].double() @ down.weight[g].double()),
                          (dx[s:s + c], dgu[s:s + c].double() @ up.weight[g].double())]:
            # half a bf16 step of each element, and the sums' error, which for
            # K <= 512 is under 2^-15 of |row| |column|
            tol = 2.0 ** -8 * want.abs() + 2.0 ** -15 * (layer.H + 256)
            assert ((got.double() - want).abs() <= tol).all(), g
        p = dy[s:s + c].double().T @ b
        assert ((dw2[g].double() - p).abs() <= 2.0 ** -15 * (c + 1)).all()
        assert ((dw2_twice[g].double() - 2 * p).abs() <= 2.0 ** -14 * (c + 1)).all()
        assert ((dw13[g].double() - dgu[s:s + c].double().T @ a).abs() <= 2.0 ** -14 * (c + 1)).all()
    for t in (gu, y, dh, dx):
        assert not t[~used].any()


def test_step_in_a_graph():
    """The block's forward and backward captured once and replayed on new input,
    beside eager calls, bit for bit."""
    from mixture_experts_layer_40_b200.block import MoEBlock
    case, layer, bias = a_layer()
    x = H.x_to_device(case.x_bits)
    w = torch.ones(layer.H, device="cuda")
    block = MoEBlock(layer, w, w)
    dr = torch.randn_like(x)
    r = torch.empty_like(x)
    block.forward(x, bias, r=r)
    block.backward(dr)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.forward(x, bias, r=r)
        g = block.backward(dr)
    x.mul_(-0.5)
    graph.replay()
    torch.cuda.synchronize()
    got = {k: v.clone() for k, v in g.items()}
    got_r = r.clone()
    eager_r = block.forward(x, bias)
    eager = block.backward(dr)
    torch.cuda.synchronize()
    assert torch.equal(got_r, eager_r)
    for k in eager:
        assert torch.equal(got[k], eager[k]), k

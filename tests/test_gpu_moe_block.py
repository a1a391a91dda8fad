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


def norm64(v, w):
    return v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6) * w


@pytest.mark.parametrize("res", [BF16, torch.float32])
@pytest.mark.parametrize("gate_kind", ["row", "full", "none"])
@pytest.mark.parametrize("with_du", [False, True])
def test_every_gradient_of_the_block(res, gate_kind, with_du):
    """All of the backward's gradients: bit for bit what the norms' two backwards
    and the layer's give one by one, and against float64 around the layer, with
    and without a gradient of the second output u = N(r; next_weight).

    The norms' sums are off by at most 2^-15 of their terms' magnitudes (512 units
    of 2^-24), which for sums of 64 random terms are about 8 times the result:
    2^-12 in the norm. dx in bf16 is rounded once, with du also half-way: 2^-7."""
    from mixture_experts_layer_40_b200 import capi
    from mixture_experts_layer_40_b200.block import MoEBlock
    case, layer, bias = a_layer()
    T, Hs = layer.T, layer.H
    gen = torch.Generator(device="cuda").manual_seed(2)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    pre, post, scale = 1 + 0.2 * rn(Hs), 1 + 0.2 * rn(Hs), 0.5 + 0.1 * rn(Hs)
    nxt = 1 + 0.2 * rn(Hs)
    x = H.x_to_device(case.x_bits).to(res)
    gate = {"row": rn(T).sigmoid(), "full": rn(T, Hs).sigmoid().to(BF16), "none": None}[gate_kind]
    block = MoEBlock(layer, pre, post, scale, alpha=0.5)
    r, u = block.forward(x, bias, gate, next_weight=nxt)
    dr, du = rn(T, Hs).to(res), rn(T, Hs).to(BF16) if with_du else None
    got = block.backward(dr, du=du)
    assert layer.status() == 0
    names = {"dx", "gates", "pre_weight", "post_weight", "scale", "w13", "w2"}
    names |= {"gate"} if gate is not None else set()
    assert set(got) == names | ({"next_weight"} if with_du else set())

    # the parts one by one
    ws = torch.empty(capi.moe_block_norm_backward_workspace_size(Hs), dtype=torch.uint8, device="cuda")
    col = lambda: torch.empty(Hs, device="cuda")  # noqa: E731
    e, dz, dpost, dscale = torch.empty_like(dr), torch.empty_like(block.z), col(), col()
    dgate = None if gate is None else torch.empty_like(gate)
    more = {"du": du, "pre_weight": nxt, "dx": e, "dpre": col()} if with_du else {}
    capi.moe_block_norm_backward(r, 1e-6, ws, dr=dr, z=block.z, post_weight=post, gate=gate,
                                 scale=scale, alpha=0.5, dz=dz, dgate=dgate, dscale=dscale,
                                 dpost=dpost, **more)
    d_in, dgates, dw13, dw2 = layer.backward(dz, block.u)
    dx, dpre = torch.empty_like(x), col()
    capi.moe_block_norm_backward(x, 1e-6, ws, dr=e if with_du else dr, du=d_in, pre_weight=pre,
                                 dx=dx, dpre=dpre)
    want = {"dx": dx, "gates": dgates, "pre_weight": dpre, "post_weight": dpost, "scale": dscale,
            "gate": dgate, "w13": dw13, "w2": dw2, "next_weight": more.get("dpre")}
    for k in got:
        assert torch.equal(got[k], want[k]), k

    # around the layer in float64
    leaf = lambda t: None if t is None else t.double().requires_grad_()  # noqa: E731
    near = lambda a, b, t: (a.double() - b).norm() <= t * b.norm()  # noqa: E731
    rl, nl, zl, pl, sl, gl, xl, wl = map(leaf, (r, nxt, block.z, post, scale, gate, x, pre))
    up = dr.double()
    if with_du:
        (norm64(rl, nl) * du.double()).sum().backward()
        up = up + rl.grad
        assert near(got["next_weight"], nl.grad, 2.0 ** -12)
    branch = 0.5 * sl * norm64(zl, pl)
    if gate is not None:
        branch = branch * (gl[:, None] if gate_kind == "row" else gl)
    (branch * up).sum().backward()
    assert near(got["post_weight"], pl.grad, 2.0 ** -12) and near(got["scale"], sl.grad, 2.0 ** -12)
    assert near(dz, zl.grad, 2.0 ** -8)
    if gate is not None:
        assert near(got["gate"], gl.grad, 2.0 ** -12 if gate_kind == "row" else 2.0 ** -8)
    (norm64(xl, wl) * d_in.double()).sum().backward()
    assert near(got["pre_weight"], wl.grad, 2.0 ** -12)
    assert near(got["dx"], up + xl.grad, 2.0 ** -12 if res != BF16 else 2.0 ** -7)


def test_gradient_of_u_needs_its_weight():
    from mixture_experts_layer_40_b200.block import MoEBlock
    case, layer, bias = a_layer()
    x = H.x_to_device(case.x_bits)
    block = MoEBlock(layer, torch.ones(layer.H, device="cuda"))
    block.forward(x, bias)
    with pytest.raises(ValueError, match="next_weight"):
        block.backward(x, du=x)


def test_grouped_linear_reports_bad_groups():
    """Without a status word of the caller's, the holder's own tells of group
    tables that fail the checks, in the forward and in the backward."""
    from mixture_experts_layer_40_b200.block import GroupedLinear
    gen = torch.Generator(device="cuda").manual_seed(3)
    lin = GroupedLinear(torch.randn(2, 32, 64, generator=gen, device="cuda").to(BF16))
    x = torch.randn(20, 64, generator=gen, device="cuda").to(BF16)
    dy = torch.randn(20, 32, generator=gen, device="cuda").to(BF16)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    good, bad = (ints(10, 10), ints(0, 10)), (ints(10, 11), ints(0, 10))
    lin.forward(x, *good)
    lin.backward(dy, x, *good)
    assert lin.status() == 0
    lin.forward(x, *bad)
    assert lin.status() == -5 and lin.status() == 0  # MOE_ERR_BOUNDS, told once
    lin.backward(dy, x, *bad)
    assert lin.status() == -5
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    lin.forward(x, *bad, status=word)
    assert lin.status() == 0 and int(word) != 0


def test_dropped_holders_keep_their_memory_until_done():
    """A block and a grouped map used on another stream than the one they were
    made on and dropped at once: the memory they made goes to nobody else while
    that stream still has their work before it."""
    from mixture_experts_layer_40_b200.block import GroupedLinear, MoEBlock
    case, layer, bias = a_layer()
    x = H.x_to_device(case.x_bits)
    w = torch.ones(layer.H, device="cuda")
    rows = torch.tensor([layer.T], dtype=torch.int32, device="cuda")
    start = torch.zeros_like(rows)
    maps = torch.randn(1, 64, layer.H, device="cuda").to(BF16)
    # every kernel once: loading one waits for the GPU
    MoEBlock(layer, w).forward(x, bias)
    GroupedLinear(maps).forward(x, rows, start)
    torch.cuda._sleep(1)
    torch.full((8,), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    block, lin = MoEBlock(layer, w), GroupedLinear(maps)
    places = [(t.data_ptr(), t.numel() * t.element_size()) for t in (block.u, block.z, lin._status)]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(1_000_000_000)  # half a second
    r = block.forward(x, bias, stream=side)
    y = lin.forward(x, rows, start, stream=side)
    del block, lin
    held = [torch.full((size,), 255, dtype=torch.uint8, device="cuda")
            for _ in range(300) for _, size in places]
    taken = {t.data_ptr() for t in held}
    assert not side.query()
    assert not any(at in taken for at, _ in places)
    torch.cuda.synchronize()
    assert torch.equal(r, MoEBlock(layer, w).forward(x, bias))
    assert torch.equal(y, GroupedLinear(maps).forward(x, rows, start))


def test_backward_after_another_pass_of_the_layer_is_refused():
    """Two blocks around one layer, or a call of the layer itself between a block's
    forward and its backward: the layer's routing and rows are another pass's."""
    from mixture_experts_layer_40_b200.block import MoEBlock
    case, layer, bias = a_layer()
    x = H.x_to_device(case.x_bits)
    w = torch.ones(layer.H, device="cuda")
    first, second = MoEBlock(layer, w), MoEBlock(layer, w)
    step = layer.graphed_step(x, bias)
    first.forward(x, bias)
    want = first.backward(x)
    for between in (lambda: second.forward(x, bias), lambda: layer.forward(x, bias),
                    lambda: layer.route(x, bias), step.replay):
        first.forward(x, bias)
        between()
        with pytest.raises(ValueError, match="another"):
            first.backward(x)
    second.forward(x, bias)
    got = second.backward(x)
    assert all(torch.equal(got[k], want[k]) for k in want)
    second.backward(x)  # twice after one forward


def test_block_of_no_rows():
    """An empty batch: empty outputs, and zero weight gradients to the last one."""
    from mixture_experts_layer_40_b200.block import MoEBlock
    from mixture_experts_layer_40_b200.layer import MoELayer
    case, layer, bias = a_layer()
    empty = MoELayer(0, layer.H, layer.N, layer.K, layer.I, layer.weights)
    w = torch.ones(layer.H, device="cuda")
    block = MoEBlock(empty, w, w, w)
    x = torch.empty(0, layer.H, dtype=BF16, device="cuda")
    filler = [torch.full((17, 512, 256), 7.0, device="cuda") for _ in range(4)]
    del filler  # memory that is not zero for the gradients
    r, u = block.forward(x, bias, torch.empty(0, device="cuda"), next_weight=w)
    g = block.backward(r, du=u)
    assert r.shape == u.shape == g["dx"].shape == (0, layer.H) and empty.status() == 0
    for k in ("pre_weight", "post_weight", "scale", "next_weight", "w13", "w2"):
        assert not g[k].any(), k

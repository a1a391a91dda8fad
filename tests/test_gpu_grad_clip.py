"""Global gradient norm and clipping against float64.

Tolerances, before any run, with u = 2^-24: 4 or 8 squares are added in fp32
(8 u of their sum), the rest in fp64, and the root halves that, so with its
own rounding the norm is off by at most 6 u of it; the factor's rounding and
the product's add 2 u, a 16-bit output half a step (finfo.eps / 2, or half the
smallest subnormal)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def capi():
    from __graft_entry__ import build
    build()
    assert torch.cuda.is_available()
    from mixture_experts_layer_40_b200 import capi as c
    return c


def grads_of(sizes, types, seed=0, std=1.0, shift=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        t = torch.randn(n + shift, generator=gen, device="cuda") * std
        out.append(t.to(types[i % len(types)])[shift:])
    return out


def clip(capi, grads, max_norm, out=None):
    gl = capi.make_grad_list(grads, out)
    partials = torch.full((capi.GRAD_PARTIALS,), 5.0, dtype=torch.float64, device="cuda")
    norm = torch.empty(1, device="cuda")
    capi.moe_grad_sumsq(gl, partials)
    capi.moe_grad_clip(gl, partials, max_norm, norm)
    return norm


def check(capi, grads, max_norm, out_of_place):
    ref = [g.double() for g in grads]
    total = math.sqrt(sum(float((g * g).sum()) for g in ref))
    c = min(1.0, max_norm / (total + 1e-6))
    out = [torch.full_like(g, 3.0) for g in grads] if out_of_place else None
    before = [g.clone() for g in grads]
    norm = clip(capi, grads, max_norm, out)
    assert abs(float(norm) - total) <= 6 * U * total
    for i, (got, r) in enumerate(zip(out or grads, ref)):
        want = r * c
        if c == 1.0:
            assert torch.equal(got, before[i]), i
            continue
        info = torch.finfo(got.dtype)
        tol = 9 * U * want.abs() + (0 if got.dtype == FP32 else info.eps / 2) * want.abs() * 1.001
        tol = tol + info.smallest_normal * info.eps
        assert ((got.double() - want).abs() <= tol).all(), i
    if out_of_place:
        assert all(torch.equal(g, b) for g, b in zip(grads, before))
    return norm


SIZES = [[1], [7], [0, 5, 0], [8192], [8193, 1, 8191], [100000, 3, 0, 70001, 16, 8], [1 << 22, 9]]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("types", [[FP32], [BF16], [FP16], [FP32, BF16, FP16]])
@pytest.mark.parametrize("out_of_place", [False, True])
def test_clip(capi, sizes, types, out_of_place):
    for max_norm in (0.5, 1e9):
        check(capi, grads_of(sizes, types), max_norm, out_of_place)


@pytest.mark.parametrize("n", [31, 32, 33, 256, 257, 700, 5000])
def test_many_tensors(capi, n):
    sizes = [(i * 37) % 1000 for i in range(n)]
    check(capi, grads_of(sizes, [FP32, BF16]), 1.0, False)
    check(capi, grads_of(sizes, [BF16, FP16]), 1.0, True)


@pytest.mark.parametrize("shift", [1, 2, 3, 5])
def test_misaligned(capi, shift):
    sizes = [20000, 1, 3, 9000]
    check(capi, grads_of(sizes, [FP32, BF16], shift=shift), 1.0, False)
    g = grads_of(sizes, [FP32, BF16], shift=shift)
    o = [torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")[1:] for x in g]
    total = math.sqrt(sum(float((x.double() ** 2).sum()) for x in g))
    norm = clip(capi, g, 1.0, o)
    assert abs(float(norm) - total) <= 6 * U * total
    for x, y in zip(g, o):
        want = x.double() / (total + 1e-6)
        tol = (9 * U + (0 if x.dtype == FP32 else torch.finfo(x.dtype).eps / 2 * 1.001)) * want.abs()
        assert ((y.double() - want).abs() <= tol + 1e-40).all()


def test_flat_buffer_of_views(capi):
    flat = torch.randn(1_000_003, device="cuda")
    ref = flat.double()
    views = list(flat.split([1, 2, 3, 100_000, 77, 899_920]))
    norm = clip(capi, views, 2.0)
    total = float(ref.norm())
    assert abs(float(norm) - total) <= 6 * U * total
    want = ref * (2.0 / (total + 1e-6))
    assert ((flat.double() - want).abs() <= 9 * U * want.abs()).all()


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e18, 1e30])
def test_squares_outside_fp32(capi, scale):
    g = grads_of([5000, 77, 3], [FP32, BF16], std=scale)
    total = math.sqrt(sum(float((x.double() ** 2).sum()) for x in g))
    norm = clip(capi, g, math.inf)
    assert abs(float(norm) - total) <= 6 * U * total


def test_zero_and_empty(capi):
    g = [torch.zeros(9000, device="cuda"), torch.zeros(3, dtype=BF16, device="cuda")]
    assert float(clip(capi, g, 1.0)) == 0.0
    assert not any(x.any() for x in g)
    assert float(clip(capi, [torch.empty(0, device="cuda")], 1.0)) == 0.0
    # max_norm 0 clears finite gradients
    g = grads_of([100], [FP32])
    clip(capi, g, 0.0)
    assert not g[0].any()


def test_no_tensors(capi):
    gl = capi.make_grad_list([])
    partials = torch.full((capi.GRAD_PARTIALS,), 5.0, dtype=torch.float64, device="cuda")
    norm = torch.full((1,), 5.0, device="cuda")
    capi.moe_grad_sumsq(gl, partials)
    capi.moe_grad_clip(gl, partials, 1.0, norm)
    assert float(norm) == 0.0 and not partials.any()


def test_non_finite(capi):
    g = grads_of([9000, 50], [FP32, BF16])
    g[0][4321] = float("inf")
    norm = clip(capi, g, 1.0)
    assert float(norm) == math.inf
    assert torch.isnan(g[0][4321]) and not g[1].any()
    assert int(torch.isnan(g[0]).sum()) == 1 and int((g[0] != 0).sum()) == 1
    for at in (0, 8999):
        g = grads_of([9000, 50], [FP32, BF16])
        g[0][at] = float("nan")
        norm = clip(capi, g, 1.0)
        assert math.isnan(float(norm)) and torch.isnan(g[0]).all() and torch.isnan(g[1]).all()


def test_infinite_limit(capi):
    """c = inf / (norm + 1e-6): 1 for a finite norm, NaN for an infinite one."""
    g = grads_of([9000, 50], [FP32, BF16])
    before = [t.clone() for t in g]
    clip(capi, g, math.inf)
    assert all(torch.equal(a, b) for a, b in zip(g, before))
    g[0][0] = math.inf
    assert float(clip(capi, g, math.inf)) == math.inf
    assert all(bool(torch.isnan(t).all()) for t in g)


def test_partials_add_over_shards(capi):
    """Two ranks' partials, added, clip both by the norm of all gradients."""
    a, b = grads_of([5000, 3], [FP32], 1), grads_of([70000], [FP32], 2)
    total = math.sqrt(sum(float((x.double() ** 2).sum()) for x in a + b))
    la, lb = capi.make_grad_list(a), capi.make_grad_list(b)
    p, q = torch.empty(2, capi.GRAD_PARTIALS, dtype=torch.float64, device="cuda")
    capi.moe_grad_sumsq(la, p)
    capi.moe_grad_sumsq(lb, q)
    p += q
    norm = torch.empty(1, device="cuda")
    for gl in (la, lb):
        capi.moe_grad_clip(gl, p, 1.0, norm)
        assert abs(float(norm) - total) <= 6 * U * total
    after = math.sqrt(sum(float((x.double() ** 2).sum()) for x in a + b))
    assert abs(after - 1.0) <= 1e-5


def test_past_32_bits(capi):
    n = (1 << 31) + 12345
    g = torch.zeros(n, dtype=BF16, device="cuda")
    g[-1], g[0] = 3.0, 4.0
    norm = clip(capi, [g], 2.5)
    assert float(norm) == 5.0
    assert float(g[-1]) == 1.5 and float(g[0]) == 2.0 and int((g != 0).sum()) == 2


def test_reproducible_streams_and_graphs(capi):
    g = grads_of([300000, 77, 12345], [FP32, BF16])
    out = [torch.empty_like(x) for x in g]
    norm = clip(capi, g, 1.0, out)
    gl = capi.make_grad_list(g, [torch.empty_like(x) for x in g])
    partials = torch.empty(capi.GRAD_PARTIALS, dtype=torch.float64, device="cuda")
    n2 = torch.empty(1, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    capi.moe_grad_sumsq(gl, partials, stream=side)
    capi.moe_grad_clip(gl, partials, 1.0, n2, stream=side)
    side.synchronize()
    assert torch.equal(norm, n2) and all(torch.equal(a, b) for a, b in zip(out, gl.out))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        capi.moe_grad_sumsq(gl, partials)
        capi.moe_grad_clip(gl, partials, 1.0, n2)
    g[0].mul_(0.5)
    graph.replay()
    norm = clip(capi, g, 1.0, out)
    torch.cuda.synchronize()
    assert torch.equal(norm, n2) and all(torch.equal(a, b) for a, b in zip(out, gl.out))


def test_binding_refuses(capi):
    a = torch.zeros(64, device="cuda")
    with pytest.raises(ValueError, match="overlap"):
        capi.make_grad_list([a, a])
    with pytest.raises(ValueError, match="overlap"):
        capi.make_grad_list([a[:40], a[30:]])
    with pytest.raises(ValueError):
        capi.make_grad_list([a], [torch.zeros(63, device="cuda")])
    with pytest.raises(ValueError):
        capi.make_grad_list([a], [a.half()])
    with pytest.raises(ValueError):
        capi.make_grad_list([a.double()])
    with pytest.raises(ValueError):
        capi.make_grad_list([a.view(8, 8).T])
    with pytest.raises(ValueError):
        capi.moe_grad_sumsq(capi.make_grad_list([a]), a)


@pytest.mark.parametrize("n", [3, 40])
def test_dropped_holders_keep_their_memory_until_done(capi, n):
    """A GradClip, and a list with its table, used on another stream than the one
    they were made on and dropped at once: their memory goes to nobody else while
    that stream still has their work before it."""
    from mixture_experts_layer_40_b200.block import GradClip
    g = grads_of([500] * n, [FP32, BF16])
    total = math.sqrt(sum(float((x.double() ** 2).sum()) for x in g))
    side = torch.cuda.Stream()
    # every kernel once: loading one waits for the GPU
    GradClip(g)(math.inf)
    torch.cuda._sleep(1)
    torch.full((8,), 255, dtype=torch.uint8, device="cuda")
    for explicit in (True, False):
        clip = GradClip(g)
        table = clip.list._table
        places = [(clip.partials.data_ptr(), 8192)]
        places += [(table.data_ptr(), table.numel())] if table is not None else []
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(1_000_000_000)  # half a second
        if explicit:
            norm = clip(math.inf, stream=side)
        else:
            with torch.cuda.stream(side):
                norm = clip(math.inf)
        del clip, table
        held = [torch.full((size,), 255, dtype=torch.uint8, device="cuda")
                for _ in range(300) for _, size in places]
        taken = {t.data_ptr() for t in held}
        assert not side.query()
        assert not any(at in taken for at, _ in places)
        torch.cuda.synchronize()
        assert abs(float(norm) - total) <= 6 * U * total
        del held


def test_long_list_in_a_graph(capi):
    """A list with a table, made before a capture: the graph clips what its
    gradients hold at each replay."""
    from mixture_experts_layer_40_b200.block import GradClip
    g = grads_of([(i * 91) % 3000 + 1 for i in range(50)], [FP32, BF16])
    clip = GradClip(g)
    clip(math.inf)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = clip(1.0)
    for scale in (3.0, 0.25):
        fresh = grads_of([t.numel() for t in g], [FP32, BF16], seed=9, std=scale)
        for a, b in zip(g, fresh):
            a.copy_(b)
        graph.replay()
        total = math.sqrt(sum(float((x.double() ** 2).sum()) for x in fresh))
        assert abs(float(norm) - total) <= 6 * U * total
        for a, b in zip(g, fresh):
            want = b.double() / (total + 1e-6)
            tol = (9 * U + (0 if a.dtype == FP32 else torch.finfo(a.dtype).eps / 2 * 1.001)) * want.abs()
            assert ((a.double() - want).abs() <= tol + 1e-40).all()

"""Products grouped by expert in 16 bits, and their gradients, against float64.

Tolerance of one output element, before any run: the 16-bit products are exact
in fp32; each tensor-core step adds 16 of them to the fp32 total and is off by
at most 2^-22 of the largest partial sum, which S = sum |a||b| bounds, so K/16
steps are off by (K/16 + 2) 2^-22 S; the rounding to the output's type adds
half a step, finfo.eps / 2 of the value (or half the smallest subnormal)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def capi():
    from __graft_entry__ import build
    build()
    assert torch.cuda.is_available()
    from mixture_experts_layer_40_b200 import capi as c
    return c


def layout(counts, align=1, lead=0, tail=0):
    """Device group arrays for these counts, starts rounded up to `align`."""
    starts, at = [], lead
    for c in counts:
        at = -(-at // align) * align
        starts.append(at)
        at += c
    dev = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in (counts, starts)]
    return dev[0], dev[1], starts, at + tail


def close(got, ref, mag, terms, what):
    """Every element within the tolerance of the module's docstring."""
    info = torch.finfo(got.dtype)
    acc = (terms / 16 + 2) * 2.0 ** -22 * mag
    tol = acc + (info.eps / 2) * (ref.abs() + acc) + info.smallest_normal * info.eps / 2
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((err / tol).max()))


def randn(gen, *shape, dtype=BF16, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


def check_matmul(capi, counts, K, N, dtype=BF16, out_dtype=None, trans=True, align=1, lead=0,
                 tail=0, seed=0, poison=True):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    gr, gs, starts, rows = layout(counts, align, lead, tail)
    G = len(counts)
    a = randn(gen, max(rows, 1), K, dtype=dtype)[:rows]
    b = randn(gen, G, N, K, dtype=dtype, std=K ** -0.5)
    b_arg = b if trans else b.transpose(1, 2).contiguous()
    inside = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for s, c in zip(starts, counts):
        inside[s:s + c] = True
    if poison:  # rows of no group hold anything at all
        a[~inside] = float("nan")
    out = torch.full((rows, N), 7.0, dtype=out_dtype or dtype, device="cuda")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    capi.moe_grouped_matmul(a, b_arg, gr, gs, out, trans_b=trans, status=status)
    assert capi.moe_get_status(status) == 0
    assert (out[~inside] == 7.0).all()
    for g, (s, c) in enumerate(zip(starts, counts)):
        if c:
            x, w = a[s:s + c].double(), b[g].double()
            close(out[s:s + c], x @ w.T, x.abs() @ w.abs().T, K, (g, counts))
    return a, b_arg, gr, gs, out


def check_wgrad(capi, counts, N, K, dtype=BF16, out_dtype=FP32, align=1, lead=0, tail=0, seed=0,
                accumulate=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    gr, gs, starts, rows = layout(counts, align, lead, tail)
    dy = randn(gen, max(rows, 1), N, dtype=dtype)[:rows]
    x = randn(gen, max(rows, 1), K, dtype=dtype)[:rows]
    inside = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for s, c in zip(starts, counts):
        inside[s:s + c] = True
    dy[~inside] = float("nan")
    x[~inside] = float("inf")
    base = randn(gen, len(counts), N, K, dtype=out_dtype)
    dw = base.clone() if accumulate else torch.full_like(base, 7.0)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    capi.moe_grouped_wgrad(dy, x, gr, gs, dw, accumulate=accumulate, status=status)
    assert capi.moe_get_status(status) == 0
    for g, (s, c) in enumerate(zip(starts, counts)):
        p, q = dy[s:s + c].double(), x[s:s + c].double()
        ref, mag = p.T @ q, p.abs().T @ q.abs()
        if accumulate:
            ref = ref + base[g].double()
            mag = mag + base[g].double().abs()
        if c == 0:
            assert torch.equal(dw[g], base[g] if accumulate else torch.zeros_like(base[g]))
        else:
            close(dw[g], ref, mag, c, (g, counts))
    return dy, x, gr, gs, dw


COUNTS = [[1], [0, 3, 0], [128, 128], [127, 129, 1, 0, 64], [33, 0, 0, 300, 5, 96, 97], [0, 0]]


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("trans", [True, False])
@pytest.mark.parametrize("dtype,out", [(BF16, None), (FP16, None), (BF16, FP32), (FP16, FP32)])
def test_matmul_ragged(capi, counts, trans, dtype, out):
    check_matmul(capi, counts, 200, 136, dtype, out, trans)


@pytest.mark.parametrize("K,N", [(8, 8), (64, 64), (72, 264), (128, 256), (1000, 40), (16, 520)])
@pytest.mark.parametrize("trans", [True, False])
def test_matmul_sizes(capi, K, N, trans):
    check_matmul(capi, [5, 0, 140, 31], K, N, trans=trans, seed=K + N)


@pytest.mark.parametrize("trans", [True, False])
def test_matmul_gaps_and_ends(capi, trans):
    check_matmul(capi, [100, 0, 7, 260], 136, 72, trans=trans, align=128, tail=60)
    check_matmul(capi, [100, 1, 7, 26], 136, 72, trans=trans, align=5, lead=3, tail=1)


@pytest.mark.parametrize("trans", [True, False])
def test_matmul_wide_tiles(capi, trans):
    # enough tiles for the 128- and the 256-wide variants
    check_matmul(capi, [300] * 40, 264, 1304, trans=trans)
    check_matmul(capi, [1] * 130, 136, 648, trans=trans)
    check_matmul(capi, [257, 1000, 3, 4000, 129, 640] * 3, 456, 1800, trans=trans)


def test_matmul_many_groups(capi):
    counts = [(g * 7) % 5 for g in range(1025)]
    check_matmul(capi, counts, 64, 24)


@pytest.mark.parametrize("counts", COUNTS + [[16], [17, 15, 47, 49], [63, 65, 191]])
@pytest.mark.parametrize("dtype,out", [(BF16, FP32), (FP16, FP32), (BF16, BF16), (FP16, FP16)])
def test_wgrad_ragged(capi, counts, dtype, out):
    check_wgrad(capi, counts, 136, 200, dtype, out)


@pytest.mark.parametrize("N,K", [(8, 8), (64, 64), (264, 72), (128, 256), (40, 1000), (520, 16)])
def test_wgrad_sizes(capi, N, K):
    check_wgrad(capi, [5, 0, 140, 31], N, K, seed=K + N)


@pytest.mark.parametrize("out", [FP32, BF16])
def test_wgrad_accumulates(capi, out):
    check_wgrad(capi, [5, 0, 140, 31], 136, 264, out_dtype=out, accumulate=True)


def test_wgrad_gaps_and_wide_tiles(capi):
    check_wgrad(capi, [100, 0, 7, 260], 136, 72, align=128, tail=60)
    check_wgrad(capi, [100, 1, 7, 26], 136, 72, align=5, lead=3, tail=1)
    check_wgrad(capi, [300, 0, 257, 1, 64] * 4, 520, 1304)


def test_no_rows(capi):
    gr, gs = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    w = torch.ones(3, 16, 24, dtype=BF16, device="cuda")
    out = torch.empty(0, 16, dtype=BF16, device="cuda")
    capi.moe_grouped_matmul(torch.empty(0, 24, dtype=BF16, device="cuda"), w, gr, gs, out)
    dw = torch.ones(3, 16, 24, device="cuda")
    e = torch.empty(0, 16, dtype=BF16, device="cuda"), torch.empty(0, 24, dtype=BF16, device="cuda")
    capi.moe_grouped_wgrad(*e, gr, gs, dw, accumulate=True)
    assert (dw == 1).all()
    capi.moe_grouped_wgrad(*e, gr, gs, dw)
    assert (dw == 0).all()


def test_special_values_stay_in_their_rows(capi):
    gen = torch.Generator(device="cuda").manual_seed(1)
    a, b = randn(gen, 70, 64), randn(gen, 2, 48, 64)
    gr, gs, starts, _ = layout([40, 30])
    a[3, 5], a[45, 7] = float("inf"), float("nan")
    out = torch.zeros(70, 48, dtype=BF16, device="cuda")
    capi.moe_grouped_matmul(a, b, gr, gs, out)
    fine = torch.isfinite(out).all(1)
    assert not fine[3] and not fine[45] and int(fine.sum()) == 68
    dw = torch.zeros(2, 48, 64, device="cuda")
    dy = randn(gen, 70, 48)
    capi.moe_grouped_wgrad(dy, a, gr, gs, dw)
    cols = torch.isfinite(dw).all(1)  # [G, K]
    assert not cols[0, 5] and not cols[1, 7] and int(cols.sum()) == 126


def test_bad_groups_are_flagged_and_skipped(capi):
    """Group tables that fail the kernel's checks set the bounds status, and
    only the groups that pass are computed."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    a, b = randn(gen, 50, 64), randn(gen, 4, 32, 64)
    for rows, start, good in [([10, -1, 10, 10], [0, 10, 20, 30], [0, 2, 3]),
                              ([10, 10, 10, 10], [0, 5, 20, 30], [0, 2, 3]),
                              ([10, 10, 10, 21], [0, 10, 20, 30], [0, 1, 2]),
                              ([10, 10, 10, 10], [-3, 10, 20, 30], [1, 2, 3]),
                              ([10, 10, 2 ** 31 - 1, 10], [0, 10, 2 ** 31 - 1, 30], [0, 1, 3]),
                              ([10, 10, 10, 10], [30, 20, 10, 0], [0])]:
        gr = torch.tensor(rows, dtype=torch.int32, device="cuda")
        gs = torch.tensor(start, dtype=torch.int32, device="cuda")
        out = torch.full((50, 32), 7.0, dtype=FP32, device="cuda")
        status = torch.zeros(4, dtype=torch.int32, device="cuda")
        capi.moe_grouped_matmul(a, b, gr, gs, out, status=status)
        assert capi.moe_get_status(status) == -5  # MOE_ERR_BOUNDS
        done = torch.zeros(50, dtype=torch.bool, device="cuda")
        for g in good:
            s, c = start[g], rows[g]
            done[s:s + c] = True
            x, w = a[s:s + c].double(), b[g].double()
            close(out[s:s + c], x @ w.T, x.abs() @ w.abs().T, 64, (g, rows))
        assert (out[~done] == 7.0).all()
        dw = torch.full((4, 32, 64), 7.0, device="cuda")
        dy = randn(gen, 50, 32)
        capi.moe_grouped_wgrad(dy, a, gr, gs, dw, status=status)
        assert capi.moe_get_status(status) == -5
        for g in range(4):
            assert good.count(g) or (dw[g] == 0).all()


def test_gradients_against_differences(capi):
    """L = sum dout * out is linear in a and in b: central differences of L, in
    float64 over fp32 outputs, give the gradients up to the outputs' error."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    counts, K, N = [9, 0, 70, 130], 72, 104
    gr, gs, _, rows = layout(counts)
    a, b, dout = randn(gen, rows, K), randn(gen, 4, N, K), randn(gen, rows, N)

    def forward(a, b):
        out = torch.zeros(rows, N, device="cuda")
        capi.moe_grouped_matmul(a, b, gr, gs, out)
        return out.double()

    da, dw = torch.zeros(rows, K, device="cuda"), torch.zeros(4, N, K, device="cuda")
    capi.moe_grouped_matmul(dout, b, gr, gs, da, trans_b=False)
    capi.moe_grouped_wgrad(dout, a, gr, gs, dw)
    for t, grad in ((a, da), (b, dw)):
        step = torch.sign(randn(gen, *t.shape))
        # t +- step must be exact in bf16: round the base to multiples of 1/8
        base = (t.float().clamp(-3, 3) * 8).round() / 8
        plus, minus = (base + step.float()).to(BF16), (base - step.float()).to(BF16)
        args = lambda v: (v, b) if t is a else (a, v)  # noqa: E731
        diff = ((forward(*args(plus)) - forward(*args(minus))) * dout.double()).sum() / 2
        want = (grad.double() * step.double()).sum()
        # both sides are sums of rows * N (grad: rows * K) fp32 values, each off
        # by at most (K/16 + 10) 2^-22 of its sum of magnitudes (under 8 * K)
        slack = (K / 16 + 10) * 2.0 ** -22 * 8 * K * float(dout.abs().double().sum()) * 2
        assert abs(float(diff - want)) <= slack, (float(diff), float(want), slack)


def test_reproducible_streams_and_graphs(capi):
    a, b, gr, gs, out = check_matmul(capi, [100, 0, 37, 260], 264, 520)
    again = torch.full_like(out, 7.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    capi.moe_grouped_matmul(a, b, gr, gs, again, stream=side)
    side.synchronize()
    assert torch.equal(out, again)
    dy, x, gr, gs, dw = check_wgrad(capi, [100, 0, 37, 260], 136, 264)
    captured, dw2 = torch.full_like(out, 7.0), torch.empty_like(dw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        capi.moe_grouped_matmul(a, b, gr, gs, captured)
        capi.moe_grouped_wgrad(dy, x, gr, gs, dw2)
    for counts in ([100, 0, 37, 260], [50, 40, 7, 13]):
        gr.copy_(torch.tensor(counts, dtype=torch.int32))
        captured.fill_(7.0)
        graph.replay()
        capi.moe_grouped_matmul(a, b, gr, gs, again.fill_(7.0))
        capi.moe_grouped_wgrad(dy, x, gr, gs, dw)
        torch.cuda.synchronize()
        assert torch.equal(captured, again) and torch.equal(dw, dw2)


def test_row_offsets_past_32_bits(capi):
    """Output and row offsets beyond 2^31 elements and 2^32 bytes."""
    K, N, rows = 8, 2056, 1_100_000
    gen = torch.Generator(device="cuda").manual_seed(5)
    counts = [40, 0, 33]
    gr = torch.tensor(counts, dtype=torch.int32, device="cuda")
    gs = torch.tensor([5, 7, rows - 33], dtype=torch.int32, device="cuda")
    a, b = torch.zeros(rows, K, dtype=BF16, device="cuda"), randn(gen, 3, N, K)
    out = torch.zeros(rows, N, dtype=BF16, device="cuda")
    for s, c in ((5, 40), (rows - 33, 33)):
        a[s:s + c] = randn(gen, c, K)
    capi.moe_grouped_matmul(a, b, gr, gs, out)
    for g, (s, c) in ((0, (5, 40)), (2, (rows - 33, 33))):
        x, w = a[s:s + c].double(), b[g].double()
        close(out[s:s + c], x @ w.T, x.abs() @ w.abs().T, K, g)
    assert not out[45:rows - 33].any()
    del a
    x = torch.zeros(rows, N, dtype=BF16, device="cuda")
    dy = torch.zeros(rows, K, dtype=BF16, device="cuda")
    for s, c in ((5, 40), (rows - 33, 33)):
        x[s:s + c], dy[s:s + c] = randn(gen, c, N), randn(gen, c, K)
    dw = torch.empty(3, K, N, device="cuda")
    capi.moe_grouped_wgrad(dy, x, gr, gs, dw)
    for g, (s, c) in ((0, (5, 40)), (2, (rows - 33, 33))):
        p, q = dy[s:s + c].double(), x[s:s + c].double()
        close(dw[g], p.T @ q, p.abs().T @ q.abs(), c, g)


def test_binding_refuses(capi):
    z = lambda *s, t=BF16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    i = z(2, t=torch.int32)
    a, b, out = z(10, 64), z(2, 32, 64), z(10, 32)
    for args in [(a, b.half(), i, i, out), (a, b, i, i, out.half()), (a, b, i, i, z(10, 64)),
                 (a, b, i, i, z(9, 32)), (a, z(2, 32, 72), i, i, out), (a, b, z(3, t=torch.int32), i, out),
                 (a, b, i.long(), i, out), (a.T, b, i, i, out), (a, b, i, i.cpu(), out),
                 (a, b.transpose(1, 2), i, i, out)]:
        with pytest.raises(ValueError):
            capi.moe_grouped_matmul(*args)
    with pytest.raises(ValueError):
        capi.moe_grouped_matmul(a, b, i, i, out, status=torch.zeros(0, device="cuda"))
    with pytest.raises(capi.MoeError):
        capi.moe_grouped_matmul(z(10, 60), z(2, 32, 60), i, i, out)
    with pytest.raises(capi.MoeError):  # rows that start off a 16-byte boundary
        capi.moe_grouped_matmul(z(641)[1:].view(10, 64), b, i, i, out)


@pytest.mark.parametrize("trans", [True, False])
@pytest.mark.parametrize("N", [72, 136, 256, 264, 520, 776])
@pytest.mark.parametrize("out", [None, FP32])
def test_matmul_long_groups(capi, trans, N, out):
    # pairs of CTAs, with one and with two accumulators, and tiles of every size
    check_matmul(capi, [256, 257, 0, 511, 1, 770, 16, 300], 200, N, out_dtype=out, trans=trans,
                 lead=2, tail=3)


@pytest.mark.parametrize("trans", [True, False])
@pytest.mark.parametrize("counts", [[1], [16], [17], [31, 0, 2], [40, 1, 1, 1], [0, 200] + [0] * 30,
                                    [3] * 20])
@pytest.mark.parametrize("K,N", [(520, 8), (1032, 264), (4104, 136), (6320, 144), (2056, 3080),
                                 (8200, 1032)])
def test_matmul_few_tiles_over_a_long_axis(capi, trans, counts, K, N):
    """Sums over K split over clusters of 2, 4 and 8 CTAs; few tiles, and with
    the wider N more than run at a time."""
    out = FP32 if K == 4104 else None
    dtype = FP16 if N == 264 else BF16
    a, b, gr, gs, first = check_matmul(capi, counts, K, N, dtype, out, trans, lead=2, tail=3)
    again = torch.full_like(first, 7.0)
    capi.moe_grouped_matmul(a, b, gr, gs, again, trans_b=trans)
    assert torch.equal(first, again)


@pytest.mark.parametrize("trans", [True, False])
@pytest.mark.parametrize("counts,N", [([33, 1], 896), ([33, 1], 2048), ([1, 0, 65, 0], 896)])
def test_matmul_split_sums_in_rounds(capi, trans, counts, N):
    # more row tiles than equal groups would have: clusters take several in turn
    check_matmul(capi, counts, 8200, N, trans=trans)


def test_matmul_each_row_count(capi):
    # every number of rows of a group from 0 to 140, all in one call and alone
    check_matmul(capi, list(range(141)), 72, 136)
    for rows in (15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 256, 257):
        check_matmul(capi, [rows], 72, 264)


def test_wgrad_long_groups_keep_fp32(capi):
    """Sums over many rows: segments of 512 rows added in fp32. A segment is off
    by at most its 32 steps' 2^-22 of its sum of magnitudes in the worst case and
    far less in the norm; over the whole gradient 2^-20 of its norm is allowed
    (the plain fp32 product has about 2^-22), however many rows there are."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    for counts in ([20000], [513, 3000, 512, 9001]):
        gr, gs, starts, rows = layout(counts)
        dy, x = randn(gen, rows, 264), randn(gen, rows, 520)
        dw = torch.empty(len(counts), 264, 520, device="cuda")
        capi.moe_grouped_wgrad(dy, x, gr, gs, dw)
        for g, (s, c) in enumerate(zip(starts, counts)):
            ref = dy[s:s + c].double().T @ x[s:s + c].double()
            assert float((dw[g] - ref).norm() / ref.norm()) < 2.0 ** -20


@pytest.mark.parametrize("counts", [[300], [520, 1, 0, 33], [4000], [4013, 2, 0], [0, 3500, 70],
                                    [64 * 70]])
@pytest.mark.parametrize("N,K", [(8, 8), (136, 264), (512, 512), (72, 1032), (1360, 112)])
@pytest.mark.parametrize("out,accumulate", [(FP32, False), (FP32, True), (BF16, False), (BF16, True)])
def test_wgrad_few_tiles_over_long_groups(capi, counts, N, K, out, accumulate):
    """Rows split over clusters of 2, 4 and 8 CTAs, some of which have no
    share of a short group."""
    dy, x, gr, gs, dw = check_wgrad(capi, counts, N, K, out_dtype=out, lead=2, tail=3,
                                    accumulate=accumulate)
    if not accumulate:
        again = torch.full_like(dw, 7.0)
        capi.moe_grouped_wgrad(dy, x, gr, gs, again)
        assert torch.equal(dw, again)


def test_wgrad_split_tiles_in_fp16(capi):
    check_wgrad(capi, [2500, 7], 264, 136, FP16, FP16, accumulate=True)
    check_wgrad(capi, [2500, 7], 264, 136, FP16, FP16)


def test_calls_on_several_streams_at_once(capi):
    """Each of the kernels beside itself and the others, on streams of their
    own: the same bits as one call after another."""
    gen = torch.Generator(device="cuda").manual_seed(8)
    calls = []
    for counts, K, N in (([1, 0, 3], 264, 520), ([300, 77, 450], 1032, 776), ([700, 900], 520, 1544),
                         ([4000], 264, 264)):
        gr = torch.tensor(counts, dtype=torch.int32, device="cuda")
        gs = torch.cumsum(gr, 0, dtype=torch.int32) - gr
        x, dy = randn(gen, sum(counts), K), randn(gen, sum(counts), N)
        w = randn(gen, len(counts), N, K)
        calls.append((x, dy, w, gr, gs))

    def outputs():
        return [(torch.zeros(x.shape[0], w.shape[1], dtype=BF16, device="cuda"),
                 torch.zeros_like(x), torch.zeros(w.shape, device="cuda"))
                for x, _, w, _, _ in calls]

    def run(call, out, stream):
        x, dy, w, gr, gs = call
        capi.moe_grouped_matmul(x, w, gr, gs, out[0], True, stream=stream)
        capi.moe_grouped_matmul(dy, w, gr, gs, out[1], False, stream=stream)
        capi.moe_grouped_wgrad(dy, x, gr, gs, out[2], stream=stream)

    alone, beside = outputs(), outputs()
    for call, out in zip(calls, alone):
        run(call, out, None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(10):
        for call, out, stream in zip(calls, beside, streams):
            run(call, out, stream)
    torch.cuda.synchronize()
    for a, b in zip(alone, beside):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def offset_and_error(capi, counts, K, N, dtype, out_dtype, trans, positive):
    """(mean relative offset, error in the norm) of the product against float64."""
    gen = torch.Generator(device="cuda").manual_seed(K + N)
    gr, gs, starts, rows = layout(counts)
    a, b = randn(gen, rows, K, dtype=dtype), randn(gen, len(counts), N, K, dtype=dtype)
    if positive:
        a, b = a.abs_(), b.abs_()
    b.mul_(K ** -0.5)
    out = torch.zeros(rows, N, dtype=out_dtype, device="cuda")
    capi.moe_grouped_matmul(a, b if trans else b.transpose(1, 2).contiguous(), gr, gs, out, trans)
    err = size = offset = 0.0
    for g, (s, c) in enumerate(zip(starts, counts)):
        ref = a[s:s + c].double() @ b[g].double().T
        d = out[s:s + c].double() - ref
        err, size = err + float(d.square().sum()), size + float(ref.square().sum())
        offset += float((d / ref).sum())
    return offset / out.numel(), (err / size) ** 0.5


@pytest.mark.parametrize("trans", [True, False])
@pytest.mark.parametrize("positive", [False, True])
@pytest.mark.parametrize("counts,K,N", [([1], 8192, 264), ([1, 3], 65608, 136), ([40, 17], 8200, 1032),
                                        ([300], 7168, 520), ([1000, 700], 8192, 1032),
                                        ([257, 0, 130], 65600, 264)])
def test_matmul_long_sums_keep_fp32(capi, counts, K, N, positive, trans):
    """Sums over a long K with an fp32 output. A TMEM sum takes 512 products in
    32 steps, each of which truncates by under 2^-23 of the running sum, half of
    that on the average, and the running sum is half of the whole on the average:
    32 x 2^-25 = 2^-20 of the segment; the segments' K / 512 <= 129 additions,
    rounded to nearest, add at most 2^-20 where they go like a random walk.
    2^-19 of the result's norm is allowed, however long K is."""
    assert offset_and_error(capi, counts, K, N, BF16, FP32, trans, positive)[1] < 2.0 ** -19


@pytest.mark.parametrize("counts,N", [([1], 136), ([40], 264), ([200, 130], 520)])
@pytest.mark.parametrize("dtype,K", [(FP16, 65544), (BF16, 262144)])
def test_matmul_long_sums_have_no_offset(capi, counts, N, dtype, K):
    """All products positive, 16-bit outputs: truncated sums are too small by a
    share that grows with their steps. A segment has 512 steps for fp16 and 4096
    for bf16, each off by at most 2^-22 of the running sum, which is half of the
    whole on the average: 2^-14 and 2^-11, an eighth of half a step of the type.
    The roundings of the outputs have no offset."""
    offset, err = offset_and_error(capi, counts, K, N, dtype, dtype, True, True)
    half = torch.finfo(dtype).eps / 2
    assert abs(offset) < half / 8 and err < half, (offset, err)


def test_wgrad_short_group_behind_seconds_of_others(capi):
    """A CTA works for longer than the kernel's wait limit (2 s) on a group whose
    rows need no clearing before it comes to one whose rows do. 149 groups of one
    tile are spread over 148 CTAs, so the first and the last share one; the first has a
    billion rows, at a quarter of a microsecond for 64. Sums of ones are exact."""
    from mixture_experts_layer_40_b200 import capi as c
    sms = c.LIB.moe_device_sm_count()
    long = 1_000_000_000 // 64 * 64
    x = torch.zeros(long + 5, 8, dtype=BF16, device="cuda")
    x[::1 << 20] = 1.0
    x[long:] = 2.0
    counts = torch.zeros(sms + 1, dtype=torch.int32)
    counts[0], counts[sms] = long, 5
    starts = torch.cumsum(counts, 0, dtype=torch.int32) - counts
    dw = torch.full((sms + 1, 8, 8), 7.0, device="cuda")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    capi.moe_grouped_wgrad(x, x, counts.cuda(), starts.cuda(), dw, status=status)
    assert capi.moe_get_status(status) == 0
    assert (dw[0] == -(-long // (1 << 20))).all()
    assert (dw[sms] == 20.0).all() and not dw[1:sms].any()

"""Block norms and their gradients against float64.

Tolerances, before any run. With u = 2^-24: a row sum of positive terms is made
of at most 32 terms per thread, 5 shuffle and 16 warp additions, so a norm's
factor is off by under 40 u, and a value built from it with the few products
around it by under 64 u of its terms' magnitudes; values that go through both
norms, or through the second row sum of the backward, by under 256 u. Sums over
the rows take at most T / CTAs + 8 + CTAs / 8 + 8 additions, under 256 here, on
top: 512 u of the terms' magnitudes. A result's own rounding adds half a step,
finfo.eps / 2 of it (or half the smallest subnormal)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def capi():
    from __graft_entry__ import build
    build()
    assert torch.cuda.is_available()
    from mixture_experts_layer_40_b200 import capi as c
    return c


def close(got, ref, mag, units, what):
    info = torch.finfo(got.dtype)
    acc = units * U * mag
    half = 0.0 if got.dtype == FP32 else info.eps / 2
    tol = acc + half * (ref.abs() + acc) + info.smallest_normal * info.eps
    err = (got.double() - ref).abs()
    assert (err <= tol).all(), (what, int((~(err <= tol)).sum()), float((err / tol).max()))


def make(T, H, act, res, wt, gate, scale, z, post, pre, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    d = {"x": (rn(T, H) * 2).to(res), "z": rn(T, H).to(act) if z else None,
         "pre": (1 + 0.3 * rn(H)).to(wt) if pre else None,
         "post": (0.5 + 0.3 * rn(H)).to(wt) if post else None,
         "scale": (0.4 + 0.2 * rn(H)).to(wt) if scale else None, "gate": None, "alpha": 0.75,
         "dr": rn(T, H).to(res), "du": rn(T, H).to(act) if pre else None}
    if gate == "row":
        d["gate"] = rn(T).sigmoid()
    elif gate == "full":
        d["gate"] = rn(T, H).sigmoid().to(act)
    return d


def forward(capi, d, in_place=False):
    act = (d["z"] if d["z"] is not None else d["du"]).dtype
    x = d["x"].clone()
    z = None if d["z"] is None else d["z"].clone()
    r = None if z is None else (x if in_place else torch.empty_like(x))
    u = None
    if d["pre"] is not None:
        u = z if in_place and z is not None else torch.empty(x.shape, dtype=act, device="cuda")
    capi.moe_block_norm(x, EPS, pre_weight=d["pre"], u=u, z=z, post_weight=d["post"],
                        gate=d["gate"], scale=d["scale"], alpha=d["alpha"], r=r)
    return r, u


def backward(capi, d, r, stream=None, ws=None):
    H = r.shape[1]
    if ws is None:
        ws = torch.empty(capi.moe_block_norm_backward_workspace_size(H), dtype=torch.uint8,
                         device="cuda")
    like = lambda t: None if t is None else torch.full_like(t, 9.0)  # noqa: E731
    col = lambda t: None if t is None else torch.full((H,), 9.0, device="cuda")  # noqa: E731
    o = {"dx": like(r) if d["pre"] is not None else None, "dz": like(d["z"]),
         "dgate": like(d["gate"]), "dscale": col(d["scale"]), "dpost": col(d["post"]),
         "dpre": col(d["pre"])}
    capi.moe_block_norm_backward(r, EPS, ws, dr=d["dr"], du=d["du"], pre_weight=d["pre"],
                                 z=d["z"], post_weight=d["post"], gate=d["gate"],
                                 scale=d["scale"], alpha=d["alpha"], stream=stream, **o)
    return o


def dbl(d):
    e = {k: (v.double() if isinstance(v, torch.Tensor) else v) for k, v in d.items()}
    one = torch.ones((), dtype=torch.float64, device="cuda")
    e["g"] = one if e["gate"] is None else e["gate"][:, None] if e["gate"].dim() == 1 else e["gate"]
    e["s"] = one if e["scale"] is None else e["scale"]
    e["p"] = one if e["post"] is None else e["post"]
    return e


def check(capi, T, H, act=BF16, res=BF16, wt=BF16, gate="none", scale=False, z=True, post=True,
          pre=True, seed=0, in_place=False):
    d = make(T, H, act, res, wt, gate, scale, z, post, pre, seed)
    e = dbl(d)
    inv = lambda v: torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)  # noqa: E731
    r, u = forward(capi, d, in_place)
    # forward
    ref_r, mag_r = e["x"], e["x"].abs()
    if z:
        y = e["z"] * inv(e["z"]) if post else e["z"]
        branch = e["alpha"] * e["s"] * e["g"] * e["p"] * y
        ref_r, mag_r = e["x"] + branch, e["x"].abs() + branch.abs()
        close(r, ref_r, mag_r, 64, "r")
    if pre:
        R = inv(ref_r)
        close(u, ref_r * R * e["pre"], (mag_r * R * e["pre"]).abs(), 256, "u")
    # backward, from an r of its own (rounded to its type)
    rr = d["x"] if r is None or in_place else r
    o = backward(capi, d, rr)
    v = rr.double()
    up, mag = e["dr"], e["dr"].abs()
    if pre:
        R = inv(v)
        h, w = v * R, e["du"] * e["pre"]
        up = up + R * (w - h * (w * h).mean(1, keepdim=True))
        mag = mag + R * (w.abs() + h.abs() * (w * h).abs().mean(1, keepdim=True))
        close(o["dx"], up, mag, 256, "dx")
        close(o["dpre"], (e["du"] * h).sum(0), (e["du"] * h).abs().sum(0), 512, "dpre")
    if z:
        Z = inv(e["z"]) if post else torch.ones_like(e["z"][:, :1])
        y = e["z"] * Z
        k = e["alpha"] * e["s"] * e["p"]
        q, mq = k * e["g"] * up, (k * e["g"]).abs() * mag
        dz, mz = q, mq
        if post:
            dz = Z * (q - y * (q * y).mean(1, keepdim=True))
            mz = Z * (mq + y.abs() * (mq * y.abs()).mean(1, keepdim=True))
        close(o["dz"], dz, mz, 256, "dz")
        t, mt = e["alpha"] * up * y, e["alpha"] * mag * y.abs()
        if post:
            close(o["dpost"], (t * e["g"] * e["s"]).sum(0), (mt * (e["g"] * e["s"]).abs()).sum(0),
                  512, "dpost")
        if scale:
            close(o["dscale"], (t * e["g"] * e["p"]).sum(0), (mt * (e["g"] * e["p"]).abs()).sum(0),
                  512, "dscale")
        dg, mg = t * e["s"] * e["p"], mt * (e["s"] * e["p"]).abs()
        if gate == "row":
            close(o["dgate"], dg.sum(1), mg.sum(1), 256, "dgate")
        elif gate == "full":
            close(o["dgate"], dg, mg, 256, "dgate")


TYPES = [(BF16, BF16, BF16), (FP16, FP16, FP32), (FP32, FP32, FP32), (BF16, FP32, FP32),
         (FP16, FP32, FP16), (BF16, FP32, BF16)]


@pytest.mark.parametrize("T,H", [(1, 7168), (3, 8), (64, 256), (130, 1000), (17, 4104), (5, 16384),
                                 (7, 8192), (900, 64), (40, 512)])
@pytest.mark.parametrize("act,res,wt", TYPES)
def test_norms(capi, T, H, act, res, wt):
    check(capi, T, H, act, res, wt, gate="row", scale=True, seed=H)


@pytest.mark.parametrize("T,H", [(3, 1), (5, 7), (70, 257), (9, 1409), (4, 5001), (3, 16383)])
@pytest.mark.parametrize("act,res,wt", TYPES)
def test_odd_widths(capi, T, H, act, res, wt):
    check(capi, T, H, act, res, wt, gate="full", scale=True, seed=H)


@pytest.mark.parametrize("gate", ["none", "row", "full"])
@pytest.mark.parametrize("scale", [False, True])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("T,H", [(33, 328), (6, 331)])
def test_forms(capi, gate, scale, post, pre, T, H):
    check(capi, T, H, gate=gate, scale=scale, post=post, pre=pre)
    check(capi, T, H, BF16, FP32, FP32, gate, scale, True, post, pre)


@pytest.mark.parametrize("T,H", [(33, 328), (6, 331), (1, 7168)])
def test_norm_before_the_block_alone(capi, T, H):
    check(capi, T, H, z=False, post=False)
    check(capi, T, H, BF16, FP32, FP32, z=False, post=False)


def test_in_place(capi):
    check(capi, 50, 1024, in_place=True)
    check(capi, 50, 77, in_place=True)


def test_rows_past_32_bits(capi):
    """Rows whose element offsets pass 2^31."""
    T, H = 300_000, 7200
    x = torch.zeros(T, H, dtype=BF16, device="cuda")
    x[-1] = torch.randn(H, device="cuda").to(BF16)
    w = torch.ones(H, dtype=BF16, device="cuda")
    u = torch.empty_like(x)
    capi.moe_block_norm(x, EPS, pre_weight=w, u=u)
    v = x[-1:].double()
    ref = v * torch.rsqrt((v * v).mean() + EPS)
    close(u[-1:], ref, ref.abs(), 64, "u")
    assert not u[:-1].any()


def test_misaligned_rows(capi):
    """Views that start off a 16-byte boundary take the element-wise path, with
    the same results up to the order of a row's sum."""
    T, H = 20, 512
    d = make(T, H, BF16, BF16, BF16, "none", False, True, True, True)
    r, u = forward(capi, d)
    shift = lambda t: torch.cat([t.new_zeros(1), t.flatten()])[1:].view(t.shape)  # noqa: E731
    m = {k: shift(v) if isinstance(v, torch.Tensor) else v for k, v in d.items()}
    assert m["x"].data_ptr() % 16 == 2
    r2, u2 = forward(capi, m)
    assert torch.equal(r, r2) and torch.equal(u, u2)


def test_special_rows(capi):
    """A zero row has the factor 1/sqrt(eps); an infinity or NaN stays in its row."""
    d = make(6, 264, BF16, FP32, FP32, "row", False, True, True, True)
    d["x"][0], d["z"][0] = 0.0, 0.0
    d["x"][2, 5], d["z"][3, 9] = float("inf"), float("nan")
    r, u = forward(capi, d)
    assert (r[0] == 0).all() and (u[0] == 0).all()
    rows = torch.isfinite(u.float()).all(1)
    assert rows.tolist() == [True, True, False, False, True, True]
    assert torch.isfinite(r).all(1).tolist() == [True, True, False, False, True, True]
    o = backward(capi, d, r)
    assert torch.isfinite(o["dz"].float()).all(1).tolist() == [True, True, False, False, True, True]


def test_gradients_against_differences(capi):
    """Directional derivatives of L = sum(dr r) + sum(du u) by central differences
    in fp32: the step h = 2^-8 leaves a truncation of order h^2 (2e-5 of third
    derivatives of order one) and a rounding noise of order u / h, both under
    1e-3 of the gradient's size along a random direction."""
    T, H = 40, 320
    d = make(T, H, FP32, FP32, FP32, "full", True, True, True, True)
    r, _ = forward(capi, d)
    o = backward(capi, d, r)
    gen = torch.Generator(device="cuda").manual_seed(8)

    def loss(e):
        r, u = forward(capi, e)
        return (d["dr"].double() * r.double()).sum() + (d["du"].double() * u.double()).sum()

    h = 2.0 ** -8
    for name, grad in (("x", "dx"), ("z", "dz"), ("gate", "dgate"), ("scale", "dscale"),
                       ("post", "dpost"), ("pre", "dpre")):
        step = torch.randn(d[name].shape, generator=gen, device="cuda")
        diff = (loss({**d, name: d[name] + h * step}) - loss({**d, name: d[name] - h * step})) / (2 * h)
        want = (o[grad].double() * step.double()).sum()
        size = float(o[grad].double().norm())
        assert abs(float(diff - want)) <= 1e-3 * size + 1e-3, (name, float(diff), float(want))


def test_no_rows(capi):
    d = make(0, 64, BF16, BF16, BF16, "row", True, True, True, True)
    forward(capi, d)
    o = backward(capi, d, d["x"])
    for k in ("dpre", "dpost", "dscale"):
        assert (o[k] == 0).all(), k


def test_reproducible_streams_and_graphs(capi):
    d = make(500, 1024, BF16, FP32, FP32, "row", True, True, True, True)
    r, u = forward(capi, d)
    o = backward(capi, d, r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2 = backward(capi, d, r, stream=side)
    side.synchronize()
    ws = torch.empty(capi.moe_block_norm_backward_workspace_size(1024), dtype=torch.uint8,
                     device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r3, u3 = forward(capi, d)
        o3 = backward(capi, d, r3, ws=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(r, r3) and torch.equal(u, u3)
    for k in o:
        assert torch.equal(o[k], o2[k]) and torch.equal(o[k], o3[k]), k


def test_binding_refuses(capi):
    d = make(4, 64, BF16, BF16, BF16, "row", False, True, True, True)
    x, z, w = d["x"], d["z"], d["pre"]
    r, u = torch.empty_like(x), torch.empty_like(z)
    ok = dict(pre_weight=w, u=u, z=z, r=r)
    for bad in [dict(ok, z=z.half()), dict(ok, u=u.float()), dict(ok, r=r.float()),
                dict(ok, pre_weight=w[:63]), dict(ok, post_weight=w.float()),
                dict(ok, gate=d["gate"].to(BF16)), dict(ok, gate=d["gate"][:3].contiguous()),
                dict(ok, z=z.T), dict(ok, scale=w.cpu())]:
        with pytest.raises(ValueError):
            capi.moe_block_norm(x, EPS, **bad)
    with pytest.raises(capi.MoeError):  # a bf16 residual stream around an fp32 block
        capi.moe_block_norm(x, EPS, pre_weight=w.float(), u=u.float())
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(capi.MoeError):
        capi.moe_block_norm_backward(x, EPS, small, du=z, pre_weight=w, dx=r,
                                     dpre=torch.empty(64, device="cuda"))


@pytest.mark.parametrize("size,eps", [(1e13, EPS), (1e15, EPS), (1e17, EPS), (1e-8, EPS), (1e-8, 0.0),
                                      (1e-14, 0.0), (1e-17, 0.0)])
@pytest.mark.parametrize("dtype", [FP32, BF16])
def test_gradients_of_large_and_small_rows(capi, size, eps, dtype):
    """Rows far from one in size, whose squares fp32 still holds: both norms'
    gradients by the formula, within the module's tolerances (the products of the
    factors stay in range: at 1e17 the smallest is 1e-34 of order-one terms)."""
    T, H = 9, 264
    gen = torch.Generator(device="cuda").manual_seed(3)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    v, up, w = (rn(T, H) * size).to(dtype), rn(T, H).to(dtype), (1 + 0.2 * rn(H)).to(dtype)
    gate = rn(T).sigmoid()
    ws = torch.empty(capi.moe_block_norm_backward_workspace_size(H), dtype=torch.uint8, device="cuda")
    dx, dz = torch.empty_like(v), torch.empty_like(v)
    dpre, dpost, dgate = torch.empty(H, device="cuda"), torch.empty(H, device="cuda"), torch.empty_like(gate)
    capi.moe_block_norm_backward(v, eps, ws, du=up, pre_weight=w, dx=dx, dpre=dpre)
    capi.moe_block_norm_backward(up, eps, ws, dr=up, z=v, post_weight=w, gate=gate, dz=dz,
                                 dgate=dgate, dpost=dpost)
    a, q = v.double(), up.double() * w.double()
    R = torch.rsqrt((a * a).mean(1, keepdim=True) + eps)
    h = a * R
    want = R * (q - h * (q * h).mean(1, keepdim=True))
    mag = R * (q.abs() + h.abs() * (q * h).abs().mean(1, keepdim=True))
    g = gate.double()[:, None]
    close(dx, want, mag, 256, "dx")
    close(dz, g * want, g * mag, 256, "dz")
    close(dgate, (q * h).sum(1), (q * h).abs().sum(1), 256, "dgate")
    t = up.double() * h
    close(dpre, t.sum(0), t.abs().sum(0), 512, "dpre")
    close(dpost, (g * t).sum(0), (g * t).abs().sum(0), 512, "dpost")


@pytest.mark.parametrize("T,H", [(300_000, 1024), (2_000_000, 64)])
@pytest.mark.parametrize("positive", [False, True])
def test_column_sums_over_many_rows(capi, T, H, positive):
    """A thread's running sum takes T / CTAs / teams rows, rounded to nearest: in
    the worst case half of 2^-23 of it a row, as a random walk the root of that:
    under 2^-19 of the terms' magnitudes for thousands of rows."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(T, H, generator=gen, device="cuda").to(BF16)
    du = torch.randn(T, H, generator=gen, device="cuda").to(BF16)
    if positive:
        du = du.abs() * x.sign()
    w = torch.ones(H, dtype=BF16, device="cuda")
    ws = torch.empty(capi.moe_block_norm_backward_workspace_size(H), dtype=torch.uint8, device="cuda")
    dx, dpre = torch.empty_like(x), torch.empty(H, device="cuda")
    capi.moe_block_norm_backward(x, EPS, ws, du=du, pre_weight=w, dx=dx, dpre=dpre)
    ref = torch.zeros(2, H, dtype=torch.float64, device="cuda")
    for a, b in zip(x.split(50_000), du.split(50_000)):
        t = b.double() * a.double() * torch.rsqrt((a.double() ** 2).mean(1, keepdim=True) + EPS)
        ref += torch.stack([t.sum(0), t.abs().sum(0)])
    assert ((dpre.double() - ref[0]).abs() <= 2.0 ** -19 * ref[1]).all()


@pytest.mark.parametrize("T,H", [(2000, 512), (700, 1409), (1500, 7168), (40, 16384), (33, 331), (5, 8)])
@pytest.mark.parametrize("act,res", [(BF16, FP32), (BF16, BF16), (FP32, FP32)])
@pytest.mark.parametrize("gate", ["row", "full"])
def test_backward_in_place(capi, T, H, act, res, gate):
    """dx may be dr, and dz may be z or du: bit for bit the results of outputs of
    their own, in the vector and the element-wise form, several rows a team."""
    d = make(T, H, act, res, act, gate, True, True, True, True, seed=T)
    want = backward(capi, d, d["x"])
    ws = torch.empty(capi.moe_block_norm_backward_workspace_size(H), dtype=torch.uint8, device="cuda")
    for on in ("z", "du"):
        e = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in d.items()}
        col = lambda: torch.empty(H, device="cuda")  # noqa: E731
        got = {"dx": e["dr"], "dz": e[on], "dgate": torch.empty_like(e["gate"]), "dscale": col(),
               "dpost": col(), "dpre": col()}
        capi.moe_block_norm_backward(e["x"], EPS, ws, dr=e["dr"], du=e["du"], pre_weight=e["pre"],
                                     z=e["z"], post_weight=e["post"], gate=e["gate"],
                                     scale=e["scale"], alpha=e["alpha"], **got)
        for k in want:
            assert torch.equal(got[k], want[k]), (on, k)


@pytest.mark.parametrize("gate", ["none", "row", "full"])
def test_misaligned_rows_backward(capi, gate):
    """Views that start off a 16-byte boundary take the element-wise path, whose
    gradients are within the tolerances of the formula as well."""
    T, H = 300, 512
    d = make(T, H, BF16, FP32, BF16, gate, True, True, True, True)
    shift = lambda t: torch.cat([t.new_zeros(1), t.flatten()])[1:].view(t.shape)  # noqa: E731
    m = {k: shift(v) if isinstance(v, torch.Tensor) else v for k, v in d.items()}
    assert m["z"].data_ptr() % 16 == 2 and m["x"].data_ptr() % 16 == 4
    o, e = backward(capi, m, m["x"]), dbl(d)
    inv = lambda v: torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)  # noqa: E731
    R, Z = inv(e["x"]), inv(e["z"])
    h, y, w = e["x"] * R, e["z"] * Z, e["du"] * e["pre"]
    up = e["dr"] + R * (w - h * (w * h).mean(1, keepdim=True))
    mag = e["dr"].abs() + R * (w.abs() + h.abs() * (w * h).abs().mean(1, keepdim=True))
    k = e["alpha"] * e["s"] * e["p"] * e["g"]
    q, mq = k * up, k.abs() * mag
    close(o["dx"], up, mag, 256, "dx")
    close(o["dz"], Z * (q - y * (q * y).mean(1, keepdim=True)),
          Z * (mq + y.abs() * (mq * y.abs()).mean(1, keepdim=True)), 256, "dz")
    close(o["dpre"], (e["du"] * h).sum(0), (e["du"] * h).abs().sum(0), 512, "dpre")
    t, mt = e["alpha"] * e["g"] * up * y, e["alpha"] * e["g"] * mag * y.abs()
    close(o["dpost"], (t * e["s"]).sum(0), (mt * e["s"].abs()).sum(0), 512, "dpost")
    close(o["dscale"], (t * e["p"]).sum(0), (mt * e["p"].abs()).sum(0), 512, "dscale")

"""Refusals of the operators beside the layer (16-bit grouped products, block
norms, gradient clipping), on the host: the C entry points return the
documented codes before any device work, and the binding raises on tensors
that do not fit. No GPU is used: the pointers are never followed."""
import ctypes
import random

import pytest
import torch

from __graft_entry__ import build

SHAPE, NULL, WORKSPACE, ALIGN = -1, -2, -6, -7
P = 1 << 20  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def capi():
    build()
    from mixture_experts_layer_40_b200 import capi as c
    return c


def matmul(c, type=0, out_type=0, groups=4, gr=P, gs=P, rows=64, K=64, N=64, a=P, b=P, out=P):
    return c.LIB.moe_grouped_matmul(type, out_type, groups, gr, gs, rows, K, N, a, b, 1, out, None,
                                    None)


def wgrad(c, type=0, out_type=2, groups=4, gr=P, gs=P, rows=64, N=64, K=64, dy=P, x=P, dw=P):
    return c.LIB.moe_grouped_wgrad(type, out_type, groups, gr, gs, rows, N, K, dy, x, dw, 0, None,
                                   None)


@pytest.mark.parametrize("call", [matmul, wgrad])
@pytest.mark.parametrize("kw,code", [
    ({"type": 2}, SHAPE), ({"type": 3}, SHAPE), ({"type": 0, "out_type": 1}, SHAPE),
    ({"out_type": 3}, SHAPE), ({"out_type": -1}, SHAPE), ({"groups": 0}, SHAPE),
    ({"groups": 1026}, SHAPE), ({"rows": -1}, SHAPE), ({"rows": (1 << 31) - 256}, SHAPE),
    ({"K": 0}, SHAPE), ({"K": 12}, SHAPE), ({"N": 0}, SHAPE), ({"N": 20}, SHAPE),
    ({"N": (1 << 20) + 8}, SHAPE), ({"K": (1 << 20) + 8}, SHAPE),
    ({"gr": None}, NULL), ({"gs": None}, NULL)])
def test_grouped_arguments_refused(capi, call, kw, code):
    assert call(capi, **kw) == code


def test_grouped_pointers_refused(capi):
    for name in ("a", "b", "out"):
        assert matmul(capi, **{name: None}) == NULL
        assert matmul(capi, **{name: P + 8}) == ALIGN
    for name in ("dy", "x", "dw"):
        assert wgrad(capi, **{name: None}) == NULL
        assert wgrad(capi, **{name: P + 8}) == ALIGN
    # no rows: nothing to multiply, and the row buffers may be NULL
    assert matmul(capi, rows=0, a=None, out=None) == 0
    assert wgrad(capi, rows=0, dw=None) == NULL


def norm(c, T=4, H=64, res=0, act=0, w=0, kind=0, alpha=1.0, eps=1e-6, x=P, z=P, gate=None, pre=P,
         post=P, scale=None, r=P, u=P):
    return c.LIB.moe_block_norm(T, H, res, act, w, kind, alpha, eps, x, z, gate, pre, post, scale,
                                r, u, None)


def norm_backward(c, T=4, H=64, res=0, act=0, w=0, kind=0, alpha=1.0, eps=1e-6, r=P, z=P, gate=None,
                  pre=P, post=P, scale=None, dr=P, du=P, dx=P, dz=P, dgate=None, dpre=P, dpost=P,
                  dscale=None, ws=P, nbytes=1 << 40):
    return c.LIB.moe_block_norm_backward(T, H, res, act, w, kind, alpha, eps, r, z, gate, pre, post,
                                         scale, dr, du, dx, dz, dgate, dpre, dpost, dscale, ws,
                                         nbytes, None)


@pytest.mark.parametrize("call", [norm, norm_backward])
@pytest.mark.parametrize("kw,code", [
    ({"T": -1}, SHAPE), ({"H": 0}, SHAPE), ({"H": 16385}, SHAPE), ({"T": 1 << 40}, SHAPE),
    ({"act": 3}, SHAPE), ({"act": -1}, SHAPE), ({"res": 1}, SHAPE), ({"act": 2, "res": 0}, SHAPE),
    ({"w": 1}, SHAPE), ({"kind": 3}, SHAPE), ({"kind": -1}, SHAPE), ({"eps": -1.0}, SHAPE),
    ({"eps": float("nan")}, SHAPE),
    ({"z": None, "r": None, "dz": None, "dpost": None, "kind": 1, "gate": P, "post": None}, SHAPE),
    ({"z": None}, SHAPE), ({"z": None, "post": None, "pre": None}, SHAPE),
    ({"kind": 1}, NULL), ({"kind": 2}, NULL), ({"pre": P + 1}, ALIGN), ({"z": P + 1}, ALIGN),
    ({"kind": 1, "gate": P + 2, "dgate": P}, ALIGN), ({"w": 2, "post": P + 2}, ALIGN)])
def test_norm_arguments_refused(capi, call, kw, code):
    import inspect
    known = inspect.signature(call).parameters
    assert call(capi, **{k: v for k, v in kw.items() if k in known}) == code


def test_norm_pointers_refused(capi):
    for name in ("x", "r", "u"):
        assert norm(capi, **{name: None}) == NULL
        assert norm(capi, **{name: P + 1}) == ALIGN
    for name in ("r", "du", "dx", "dz", "dpre", "dpost", "ws"):
        assert norm_backward(capi, **{name: None}) == NULL
        assert norm_backward(capi, **{name: P + 1}) == ALIGN
    assert norm_backward(capi, scale=P) == NULL            # dscale missing
    assert norm_backward(capi, kind=1, gate=P) == NULL     # dgate missing
    assert norm_backward(capi, pre=None, dr=None) == NULL  # no upstream gradient at all
    need = capi.moe_block_norm_backward_workspace_size(64)
    assert need > 0 and norm_backward(capi, nbytes=need - 1) == WORKSPACE
    assert norm_backward(capi, ws=P + 128) == ALIGN
    assert capi.moe_block_norm_backward_workspace_size(0) == 0
    assert capi.moe_block_norm_backward_workspace_size(16385) == 0
    assert norm(capi, T=0, x=None, r=None, u=None, z=P) == 0


def grad_struct(c, ptrs, sizes, types, out=None):
    n = len(sizes)
    arr = (ctypes.c_void_p * n)(*ptrs)
    oarr = None if out is None else (ctypes.c_void_p * n)(*out)
    s, t = (ctypes.c_int64 * n)(*sizes), (ctypes.c_int32 * n)(*types)
    cast, pp = ctypes.cast, ctypes.POINTER(ctypes.c_void_p)
    st = c.moe_grad_list(n, cast(arr, pp), None if oarr is None else cast(oarr, pp),
                         cast(s, ctypes.POINTER(ctypes.c_int64)),
                         cast(t, ctypes.POINTER(ctypes.c_int32)), None)
    st.keep = (arr, oarr, s, t)
    return st


@pytest.mark.parametrize("ptrs,sizes,types,out,code", [
    ([P], [-1], [0], None, SHAPE), ([P], [1 << 43], [0], None, SHAPE), ([P], [4], [3], None, SHAPE),
    ([P], [4], [-1], None, SHAPE), ([None], [4], [0], None, NULL), ([P], [4], [0], [None], NULL),
    ([P + 1], [4], [0], None, ALIGN), ([P + 2], [4], [2], None, ALIGN),
    ([P], [4], [2], [P + 2], ALIGN), ([P] * 4, [1 << 42] * 4, [2] * 4, None, SHAPE)])
def test_gradient_lists_refused(capi, ptrs, sizes, types, out, code):
    st = grad_struct(capi, ptrs, sizes, types, out)
    assert capi.LIB.moe_grad_sumsq(ctypes.byref(st), P, None) == code
    assert capi.LIB.moe_grad_clip(ctypes.byref(st), P, 1.0, P, None) == code


def test_clip_arguments_refused(capi):
    st = grad_struct(capi, [P], [4], [2])
    lib, ref = capi.LIB, ctypes.byref(st)
    assert lib.moe_grad_sumsq(None, P, None) == NULL
    assert lib.moe_grad_sumsq(ref, None, None) == NULL
    assert lib.moe_grad_sumsq(ref, P + 4, None) == ALIGN
    assert lib.moe_grad_clip(ref, P, -1.0, P, None) == SHAPE
    assert lib.moe_grad_clip(ref, P, float("nan"), P, None) == SHAPE
    assert lib.moe_grad_clip(ref, P, 1.0, None, None) == NULL
    assert lib.moe_grad_clip(ref, P, 1.0, P + 2, None) == ALIGN
    bad = capi.moe_grad_list(-1)
    assert lib.moe_grad_sumsq(ctypes.byref(bad), P, None) == SHAPE
    assert lib.moe_grad_sumsq(ctypes.byref(capi.moe_grad_list(1)), P, None) == NULL


def test_gradient_tables(capi):
    """The table of a longer list: entries of 32 bytes (address, output, size,
    first chunk, type) of the tensors with elements, chunks in order."""
    import struct
    lib = capi.LIB
    n = 40
    sizes = [0 if i % 7 == 3 else 100000 * i + 5 for i in range(n)]
    ptrs = [P + (i << 24) + 4 * (i % 3) for i in range(n)]
    types = [2 if i % 2 else 0 for i in range(n)]
    st = grad_struct(capi, ptrs, sizes, types)
    nbytes = lib.moe_grad_table_size(ctypes.byref(st))
    assert nbytes == 32 * n
    buf = ctypes.create_string_buffer(nbytes)
    assert lib.moe_grad_table(ctypes.byref(st), buf) == 0
    assert lib.moe_grad_table(ctypes.byref(st), None) == NULL
    kept = [i for i in range(n) if sizes[i]]
    at = 0
    for k, i in enumerate(kept):
        g, out, size, chunk0, kind = struct.unpack_from("<QQqii", buf, 32 * k)
        assert (g, out, size, kind) == (ptrs[i], ptrs[i], sizes[i], types[i])
        assert chunk0 == at
        es = 4 if types[i] == 2 else 2
        total = sum(s * (4 if t == 2 else 2) for s, t in zip(sizes, types))
        length = max(1, min(8, total // (1024 * 256 * 16))) * 256 * 16 // es
        head = -g % 128 // es
        at += max(1, -(-(size - head) // length))
    # without its table a longer list is refused; a short one needs none
    assert lib.moe_grad_sumsq(ctypes.byref(st), P, None) == NULL
    assert lib.moe_grad_clip(ctypes.byref(st), P, 1.0, P, None) == NULL
    st.table = P + 8
    assert lib.moe_grad_sumsq(ctypes.byref(st), P, None) == ALIGN
    short = grad_struct(capi, ptrs[:32], sizes[:32], types[:32])
    assert lib.moe_grad_table_size(ctypes.byref(short)) == 0
    assert lib.moe_grad_table(ctypes.byref(short), None) == 0


def test_gradient_overlaps(capi):
    refuse = capi.GradList._refuse_overlap
    refuse([0, 16, 100], None, [16, 16, 4])             # touching tensors are apart
    refuse([0, 64], [0, 64], [32, 32])                  # in place, said as an output list
    refuse([0, 16], [64, 80], [16, 16])
    refuse([0, 0], [64, 80], [16, 16])                  # the same gradient read twice
    refuse([0, 0], None, [16, 0])                       # an empty tensor lies on nothing
    for grads, out, sizes in [([0, 0], None, [16, 16]), ([0, 8], None, [16, 16]),
                              ([0, 32], [64, 64], [16, 16]), ([0, 32], [64, 72], [16, 16]),
                              ([0, 32], [32, 0], [16, 16]), ([0, 32], [8, 64], [16, 16]),
                              ([0, 100], [24, 64], [16, 1000]), ([0, 0], [0, 64], [16, 16])]:
        with pytest.raises(ValueError, match="overlap"):
            refuse(grads, out, sizes)


def test_gradient_overlaps_by_brute_force(capi):
    rng = random.Random(3)
    seen = set()
    for _ in range(3000):
        n = rng.randint(1, 4)
        sizes = [rng.choice([0, 1, 2, 5]) for _ in range(n)]
        grads = [rng.randint(0, 14) for _ in range(n)]
        out = None if rng.random() < 0.3 else [g if rng.random() < 0.4 else rng.randint(0, 40)
                                               for g in grads]
        w = grads if out is None else out
        cells = [set(range(p, p + s)) for p, s in zip(w, sizes)]
        bad = any(cells[i] & cells[j] for i in range(n) for j in range(i))
        if out is not None:
            bad |= any(cells[i] & set(range(grads[j], grads[j] + sizes[j]))
                       and (i != j or grads[j] != out[i]) for i in range(n) for j in range(n))
        try:
            capi.GradList._refuse_overlap(grads, out, sizes)
            ok = True
        except ValueError:
            ok = False
        assert ok == (not bad), (grads, out, sizes)
        seen.add(ok)
    assert seen == {True, False}


def test_binding_refuses_host_tensors(capi):
    a, b = torch.zeros(8, 64, dtype=torch.bfloat16), torch.zeros(2, 64, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        capi.moe_grouped_matmul(a, b, i, i, a)
    with pytest.raises(ValueError, match="CUDA"):
        capi.moe_grouped_wgrad(a, a, i, i, b)
    with pytest.raises(ValueError, match="three-dimensional"):
        capi.moe_grouped_matmul(a, a, i, i, a)
    with pytest.raises(ValueError, match="bfloat16"):
        capi.moe_grouped_matmul(a.double(), b, i, i, a)
    w = torch.ones(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        capi.moe_block_norm(a, 1e-6, pre_weight=w, u=a)
    with pytest.raises(ValueError, match="goes with"):
        capi.moe_block_norm(a, 1e-6, pre_weight=w)
    with pytest.raises(ValueError, match="nothing"):
        capi.moe_block_norm(a, 1e-6)
    with pytest.raises(ValueError, match="dgate"):
        capi.moe_block_norm_backward(a, 1e-6, a, dr=a, z=a, dz=a, gate=w)
    with pytest.raises(ValueError, match="CUDA"):
        capi.make_grad_list([a])
    with pytest.raises(ValueError, match="outputs"):
        capi.make_grad_list([a], [])


class FakeLayer:
    T, H, device = 4, 64, "cpu"

    def __init__(self):
        self.fail = False

    def forward(self, u, bias, z, stream):
        if self.fail:
            raise RuntimeError("layer")

    def backward(self, dz, u, stream):
        return torch.zeros(4, 64), torch.zeros(4, 2)


def test_block_backward_needs_the_forwards_x(capi, monkeypatch):
    """The backward reads the forward's x: after a forward in place, or one
    that failed, there is none, and it says so."""
    from mixture_experts_layer_40_b200.block import MoEBlock

    monkeypatch.setattr(capi, "moe_block_norm", lambda *a, **k: None)
    monkeypatch.setattr(capi, "moe_block_norm_backward", lambda *a, **k: None)
    monkeypatch.setattr(capi, "moe_block_norm_backward_workspace_size", lambda H: 16)
    layer = FakeLayer()
    block = MoEBlock(layer, torch.ones(64))
    both = torch.zeros(2, 4, 64)
    x, r = both[0], both[1]

    with pytest.raises(ValueError, match="forward"):
        block.backward(r, weights=False)
    block.forward(x, None, r=r)
    assert "dx" in block.backward(r, weights=False)
    assert block.forward(x, None, r=x) is x  # in place
    with pytest.raises(ValueError, match="in place"):
        block.backward(r, weights=False)
    block.forward(x, None)
    block.backward(r, weights=False)
    layer.fail = True
    with pytest.raises(RuntimeError):
        block.forward(r, None)
    with pytest.raises(ValueError, match="forward"):
        block.backward(r, weights=False)


@pytest.mark.parametrize("off", [1, 2, 3])
def test_words_off_their_boundary_refused(capi, off):
    """The group arrays and the status word are read and written as 4-byte words."""
    lib = capi.LIB
    for gr, gs, status in [(P + off, P, None), (P, P + off, None), (P, P, P + off)]:
        for rows in (64, 0):
            assert lib.moe_grouped_matmul(0, 0, 4, gr, gs, rows, 64, 64, P, P, 1, P, status, None) == ALIGN
            assert lib.moe_grouped_wgrad(0, 2, 4, gr, gs, rows, 64, 64, P, P, P, 0, status, None) == ALIGN


def test_block_makes_its_device_the_current_one(capi, monkeypatch):
    """The layer launches on the current device, the norms on their tensors': a
    block on another device than the current one makes it current for both."""
    from mixture_experts_layer_40_b200.block import MoEBlock

    now = [0]

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            now.append(self.index)

        def __exit__(self, *exc):
            now.pop()

    class Layer(FakeLayer):
        seen = []

        def forward(self, u, bias, z, stream):
            self.seen.append(now[-1])

        def backward(self, dz, u, stream):
            self.seen.append(now[-1])
            return super().backward(dz, u, stream)

    monkeypatch.setattr(torch.cuda, "device", Device)
    for name in ("moe_block_norm", "moe_block_norm_backward", "keep_until_done"):
        monkeypatch.setattr(capi, name, lambda *a, **k: None)
    monkeypatch.setattr(capi, "moe_block_norm_backward_workspace_size", lambda H: 16)
    block = MoEBlock(Layer(), torch.ones(64))
    assert block._index == -1  # host memory: no device
    block._index = 1
    x = torch.zeros(4, 64)
    block.forward(x, None)
    block.backward(x, weights=False)
    assert Layer.seen == [1, 1] and now == [0]


def test_block_of_no_rows_has_a_backward(capi, monkeypatch):
    """Empty tensors all have the address 0: no forward in place."""
    from mixture_experts_layer_40_b200.block import MoEBlock

    for name in ("moe_block_norm", "moe_block_norm_backward"):
        monkeypatch.setattr(capi, name, lambda *a, **k: None)
    monkeypatch.setattr(capi, "moe_block_norm_backward_workspace_size", lambda H: 16)

    class Layer(FakeLayer):
        T = 0

    block = MoEBlock(Layer(), torch.ones(64))
    x = torch.zeros(0, 64)
    assert "dx" in (block.forward(x, None), block.backward(x, weights=False))[1]

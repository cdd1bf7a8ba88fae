"""Refusals of routing by scores, layer norm, dropout and embedding, without a GPU: the C entry points return before any
CUDA call, the Python functions before the library."""
import ctypes
import os

import pytest
import torch

P = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 1)
TWO = ctypes.c_void_p((1 << 20) + 2)
FOUR = ctypes.c_void_p((1 << 20) + 4)
NAN, INF = float("nan"), float("inf")
BIG = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_grouped_fp32_gb300 import build, moe
    if not os.path.exists(moe.LIB_PATH):
        build.build()
    return moe.load()


def _err(lib):
    return lib.moe_last_error_string().decode()


def refused(lib, call, cases, code=-1):
    for kw, fragment in cases:
        assert call(**kw) == code, kw
        assert fragment in _err(lib), (kw, _err(lib))


def test_route_scores(lib):
    def call(l=P, bf16=0, bias=None, T=4, E=16, k=2, how=0, groups=1, kept=1, renorm=1, scale=1.0, idx=P, w=P, s=None):
        return lib.moe_route_scores(l, bf16, bias, T, E, k, how, groups, kept, renorm, scale, idx, w, s, None)
    refused(lib, call, [
        (dict(T=-1), "T = -1"), (dict(T=BIG), "T = "), (dict(E=0), "E = 0"), (dict(E=257), "E = 257"), (dict(k=0), "top_k = 0"),
        (dict(k=9), "top_k = 9"), (dict(E=4, k=5), "top_k = 5"), (dict(how=2), "scoring = 2"), (dict(groups=0), "n_group = 0"),
        (dict(groups=3), "n_group = 3"), (dict(E=64, groups=64), "n_group = 64"), (dict(kept=0), "topk_group = 0"),
        (dict(groups=4, kept=5), "topk_group = 5"), (dict(groups=8, kept=1, k=3), "exceeds the 2 experts"),
        (dict(scale=NAN), "scale"), (dict(scale=INF), "scale"), (dict(l=None), "null"), (dict(idx=None), "null"),
        (dict(w=None), "null"), (dict(l=TWO), "aligned"), (dict(l=ODD, bf16=1), "aligned"), (dict(bias=TWO), "aligned"),
        (dict(idx=TWO), "aligned"), (dict(s=TWO), "aligned")])
    assert call(T=0, l=None, idx=None, w=None) == 0

    def back(l=P, bf16=0, idx=P, dw=P, ds=None, T=4, E=16, k=2, how=0, scale=1.0, out=P):
        return lib.moe_route_scores_backward(l, bf16, idx, dw, ds, 0, T, E, k, how, 1, scale, out, None)
    refused(lib, back, [
        (dict(T=-1), "T = -1"), (dict(E=300), "E = 300"), (dict(k=9), "top_k = 9"), (dict(how=-1), "scoring = -1"),
        (dict(scale=-INF), "scale"), (dict(l=None), "null"), (dict(out=None), "null"), (dict(idx=None), "null"),
        (dict(out=TWO), "aligned"), (dict(dw=TWO), "aligned"), (dict(ds=TWO), "aligned"), (dict(idx=TWO), "aligned")])
    assert back(T=0, l=None, idx=None, dw=None, out=None) == 0


def test_layer_norm(lib):
    def call(x=P, f32=1, h=None, w=None, b=None, T=4, d=16, eps=1e-5, p=0.0, at=None, y=P, n=P, st=P):
        return lib.moe_layer_norm(x, f32, h, w, b, T, d, eps, p, 1, 2, at, y, n, st, None)
    refused(lib, call, [
        (dict(T=-1), "T = -1"), (dict(T=BIG), "T = "), (dict(d=0), "d = 0"), (dict(d=65537), "d = 65537"), (dict(d=65521), "multiple of 8"),
        (dict(eps=-1.0), "eps"), (dict(eps=NAN), "eps"), (dict(eps=INF), "eps"), (dict(h=P, p=1.0), "p = 1"),
        (dict(h=P, p=0.999999), "p = 0.999999"), (dict(h=P, p=-0.1), "p = -0.1"), (dict(h=P, p=NAN), "p = "), (dict(p=0.5), "belongs to h"),
        (dict(x=None), "null"), (dict(n=None), "null"), (dict(st=None), "null"), (dict(h=P, y=None), "null"),
        (dict(x=TWO), "aligned"), (dict(x=ODD, f32=0), "aligned"), (dict(st=FOUR), "aligned"), (dict(w=TWO), "aligned"),
        (dict(b=TWO), "aligned"), (dict(n=ODD), "aligned"), (dict(h=ODD), "aligned"), (dict(at=FOUR), "aligned")])
    assert call(T=0, x=None, n=None, st=None) == 0
    need = lib.moe_layer_norm_backward_workspace_size(4, 16)
    assert need > 0 and lib.moe_layer_norm_backward_workspace_size(4, 0) == 0 and lib.moe_layer_norm_backward_workspace_size(-1, 8) == 0

    def back(x=P, st=P, dn=P, dy=None, w=None, T=4, d=16, p=0.0, at=None, dx=P, dh=None, dw=None, db=None, ws=P, n=need):
        return lib.moe_layer_norm_backward(x, 1, st, dn, dy, w, T, d, p, 1, 2, at, dx, dh, dw, db, ws, n, None)
    refused(lib, back, [
        (dict(T=-1), "T = -1"), (dict(d=70000), "d = 70000"), (dict(d=65535), "multiple of 8"), (dict(p=1.5), "p = 1.5"), (dict(x=None), "null"), (dict(st=None), "null"),
        (dict(dn=None), "null"), (dict(dx=None), "null"), (dict(dy=TWO), "aligned"), (dict(dw=TWO), "aligned"),
        (dict(db=TWO), "aligned"), (dict(dh=ODD), "aligned"), (dict(st=FOUR), "aligned"), (dict(ws=FOUR), "aligned"), (dict(at=FOUR), "aligned")])
    refused(lib, back, [(dict(ws=None), "workspace"), (dict(n=need - 1), "workspace")], code=-3)
    assert back(T=0, x=None, st=None, dn=None, dx=None, ws=None) == 0


def test_dropout(lib):
    def call(x=P, f32=1, r=None, r32=1, n=100, p=0.5, at=None, out=P):
        return lib.moe_dropout(x, f32, r, r32, n, p, 1, 2, at, out, None)
    refused(lib, call, [
        (dict(n=-1), "n = -1"), (dict(n=2 ** 41), "n = "), (dict(p=1.0), "p = 1"), (dict(p=NAN), "p = "), (dict(p=-0.5), "p = -0.5"),
        (dict(x=None), "null"), (dict(out=None), "null"), (dict(x=TWO), "aligned"), (dict(out=TWO), "aligned"),
        (dict(x=ODD, f32=0), "aligned"), (dict(r=TWO), "aligned"), (dict(r=ODD, r32=0), "aligned"), (dict(at=FOUR), "aligned")])
    assert call(n=0, x=None, out=None) == 0


def test_embed(lib):
    def call(ids=P, i64=0, t=P, f32=1, T=4, V=10, d=16, scale=1.0, out=P, st=None):
        return lib.moe_embed(ids, i64, t, f32, T, V, d, scale, out, 1, st, None)
    refused(lib, call, [
        (dict(T=-1), "T = -1"), (dict(T=BIG), "T = "), (dict(V=0), "V = 0"), (dict(V=BIG), "V = "), (dict(d=0), "d = 0"),
        (dict(d=65537), "d = 65537"), (dict(scale=NAN), "scale"), (dict(ids=None), "null"), (dict(t=None), "null"), (dict(out=None), "null"),
        (dict(ids=FOUR, i64=1), "aligned"), (dict(ids=TWO), "aligned"), (dict(t=TWO), "aligned"), (dict(t=ODD, f32=0), "aligned"),
        (dict(out=TWO), "aligned"), (dict(st=TWO), "aligned")])
    assert call(T=0, ids=None, t=None, out=None) == 0
    need = lib.moe_embed_backward_workspace_size(4, 10, 16)
    assert need > 0
    for bad in ((-1, 10, 16), (4, 0, 16), (4, 10, 0)):
        assert lib.moe_embed_backward_workspace_size(*bad) == 0

    def back(ids=P, i64=0, dy=P, f32=1, T=4, V=10, d=16, scale=1.0, out=P, o32=1, acc=0, ws=P, n=need, st=None):
        return lib.moe_embed_backward(ids, i64, dy, f32, T, V, d, scale, out, o32, acc, ws, n, st, None)
    refused(lib, back, [
        (dict(T=-1), "T = -1"), (dict(V=0), "V = 0"), (dict(d=0), "d = 0"), (dict(scale=INF), "scale"), (dict(o32=0, acc=1), "accumulate"),
        (dict(ids=None), "null"), (dict(dy=None), "null"), (dict(out=None), "null"), (dict(T=0, out=None), "null"),
        (dict(ids=FOUR, i64=1), "aligned"), (dict(dy=TWO), "aligned"), (dict(out=TWO), "aligned"), (dict(ws=FOUR), "aligned"), (dict(st=TWO), "aligned")])
    refused(lib, back, [(dict(ws=None), "workspace"), (dict(n=need - 1), "workspace")], code=-3)
    assert back(T=0, acc=1, ids=None, dy=None, out=None, ws=None) == 0


class Fake:
    """A contiguous CUDA tensor as the binding sees it."""
    device = torch.device("cuda", 0)

    def __init__(self, *shape, dtype=torch.float32, on=0, cuda=True, contiguous=True):
        self.shape, self.dtype, self.on, self.is_cuda, self._c = torch.Size(shape), dtype, on, cuda, contiguous
        self.nbytes = self.numel() * dtype.itemsize

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return self._c

    def get_device(self):
        return self.on if self.is_cuda else -1

    def data_ptr(self):
        return 1 << 20


@pytest.fixture
def moe(monkeypatch):
    """The binding without launches: the library's calls are noted."""
    from mixture_experts_grouped_fp32_gb300 import moe as m
    made = []
    monkeypatch.setattr(m, "_fast", None)
    monkeypatch.setattr(m, "_call", lambda name, *a: made.append(name))
    monkeypatch.setattr(m, "_stream", lambda s: None)
    monkeypatch.setattr(m, "_wrote", lambda *ts: None)
    monkeypatch.setattr(m, "_several", True)
    monkeypatch.setattr(m, "_empty", lambda shape, dtype, device, stream: Fake(*shape, dtype=dtype))
    monkeypatch.setattr(m, "_layer_norm_workspace", lambda *a: 64)
    monkeypatch.setattr(m, "embed_backward_workspace_size", lambda *a: 64)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    m.made = made
    yield m
    del m.made


B16, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


def f(*shape, **kw):
    return Fake(*shape, **kw)


def good(m):
    """A call of each kind that passes, by name, with the operands that it takes."""
    return {
        "route_scores": (m.route_scores, dict(logits=f(4, 16), top_k=2, bias=f(16), idx=f(4, 2, dtype=I32), w=f(4, 2), scores=f(4, 16))),
        "route_scores_backward": (m.route_scores_backward, dict(logits=f(4, 16), idx=f(4, 2, dtype=I32), dw=f(4, 2), dscores=f(16), dlogits=f(4, 16))),
        "layer_norm": (m.layer_norm, dict(x=f(4, 16), weight=f(16), bias=f(16), h=f(4, 16, dtype=B16), offset_tensor=f(1, dtype=I64), y=f(4, 16), n=f(4, 16, dtype=B16), stats=f(4, 2))),
        "layer_norm_backward": (m.layer_norm_backward, dict(x=f(4, 16), stats=f(4, 2), dn=f(4, 16, dtype=B16), dy=f(4, 16), weight=f(16), bias=f(16), workspace=f(64))),
        "dropout": (m.dropout, dict(x=f(4, 16, dtype=B16), p=0.1, seed=1, residual=f(4, 16), out=f(4, 16), offset_tensor=f(1, dtype=I64))),
        "embed": (m.embed, dict(ids=f(2, 3, dtype=I64), table=f(10, 16), out=f(2, 3, 16), status=f(1, dtype=I32))),
        "embed_backward": (m.embed_backward, dict(ids=f(2, 3, dtype=I32), dy=f(2, 3, 16, dtype=B16), V=10, out=f(10, 16), workspace=f(64), status=f(1, dtype=I32))),
    }


NAMES = ["route_scores", "route_scores_backward", "layer_norm", "layer_norm_backward", "dropout", "embed", "embed_backward"]


@pytest.mark.parametrize("name", NAMES)
def test_operands_are_checked_one_by_one(moe, name):
    call, kw = good(moe)[name]
    call(**kw)
    assert moe.made == ["moe_" + name]
    moe.made.clear()
    for key, t in kw.items():
        if not isinstance(t, Fake):
            continue
        bad = [f(*t.shape, dtype=t.dtype, on=1), f(*t.shape, dtype=t.dtype, cuda=False)]
        if key not in ("status", "workspace"):
            bad += [f(*t.shape, dtype=t.dtype, contiguous=False), f(*t.shape, dtype=torch.float16)]
            if key not in ("x", "ids", "table", "logits", "dy"):
                bad += [f(*t.shape[:-1], t.shape[-1] + 1, dtype=t.dtype)]
        for b in bad:
            with pytest.raises(ValueError):
                call(**{**kw, key: b})
    assert not moe.made


@pytest.mark.parametrize("name,change,match", [
    ("route_scores", dict(scoring="tanh"), "scoring must be"), ("route_scores", dict(logits=f(16)), r"\[T, E\]"),
    ("route_scores", dict(top_k=2 ** 31), "not below 2"), ("route_scores", dict(top_k=0), "at least 1"),
    ("route_scores_backward", dict(idx=None), "needs the idx"), ("route_scores_backward", dict(scoring=0), "scoring must be"),
    ("route_scores_backward", dict(dscores=f(4, 15)), "dscores must have shape"),
    ("layer_norm", dict(x=f(16)), r"\[T, d\]"), ("layer_norm", dict(seed=-1), "seed"), ("layer_norm", dict(seed=2 ** 64), "seed"),
    ("layer_norm", dict(offset=2 ** 63), "offset"), ("layer_norm", dict(offset_tensor=f(2, dtype=I64)), "offset_tensor"),
    ("layer_norm_backward", dict(dy=f(4, 16, dtype=B16)), "dy must be"), ("layer_norm_backward", dict(seed=-5), "seed"),
    ("dropout", dict(seed=2 ** 70), "seed"), ("dropout", dict(residual=f(16, 4)), "residual must have shape"),
    ("dropout", dict(out=f(4, 16, dtype=B16)), "out must be"),
    ("embed", dict(table=f(10, 16, 1)), r"\[T, d\]"), ("embed", dict(out=f(6, 16)), "out must have shape"),
    ("embed", dict(out=None, out_dtype=torch.float16), "out must be"), ("embed_backward", dict(V=0), "at least 1"),
    ("embed_backward", dict(V=2 ** 31), "not below"), ("embed_backward", dict(dy=f(6, 16)), "ids.shape"),
    ("embed_backward", dict(dy=f(3, 2, 16)), "dy must have shape"), ("embed_backward", dict(out=None, accumulate=True), "give out"),
    ("embed_backward", dict(out=f(11, 16)), "out must have shape"),
])
def test_python_refusals(moe, name, change, match):
    call, kw = good(moe)[name]
    with pytest.raises(ValueError, match=match):
        call(**{**kw, **change})
    assert not moe.made


def test_sizes_past_32_bits(moe):
    big = 2 ** 31
    with pytest.raises(ValueError, match="not below"):
        moe.route_scores(f(big, 8), 2)
    with pytest.raises(ValueError, match="not below"):
        moe.layer_norm(f(big, 8))
    with pytest.raises(ValueError, match="not below"):
        moe.embed(f(big, dtype=I32), f(4, 8))
    with pytest.raises(ValueError, match="not below"):
        moe.embed_backward(f(big, dtype=I32), f(big, 8), 4)
    assert not moe.made

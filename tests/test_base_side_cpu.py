"""The base side without a GPU: what its entry points and its binding refuse before any
device call, and the float64 forms that its GPU tests compare with."""
import ctypes as C

import numpy as np
import pytest
import torch

import base_ref as R
import segmented_gather_rank_amd as L

OK, INVALID, UNSUPPORTED, SPACE = L.LORA_OK, L.LORA_ERR_INVALID_ARG, L.LORA_ERR_UNSUPPORTED, L.LORA_ERR_WORKSPACE
_buf = (C.c_char * 65536)()
P = (C.addressof(_buf) + 255) // 256 * 256          # never read: every call below is refused, or has nothing to do


def meta(rows=8, keys=4, div=1, **kw):
    m = L.lora_meta(rows, keys, div, P, P, P, P, P, P, P)
    for k, v in kw.items():
        setattr(m, k, v)
    return C.byref(m)


def route(rt=None, logits=P, ld=None, T=0, dtype=0, ids=P, w=P, **kw):
    r = dict(num_experts=64, topk=8, score=0, num_groups=1, topk_groups=0, group_top=0, renormalize=1, scale=1.0, d_bias=None)
    r.update(kw)
    c = L.lora_routing(**r)
    return L._lib.lora_moe_route(C.byref(c) if rt is None else None, logits, r["num_experts"] if ld is None else ld, T, dtype, ids, w, None)


def test_route_refusals():
    assert route() == OK                            # no tokens: nothing is launched
    assert route(rt="none") == INVALID
    assert route(T=-1) == INVALID
    for kw in (dict(dtype=2), dict(dtype=7), dict(score=2), dict(score=-1), dict(num_experts=1025, ld=1025), dict(topk=33),
               dict(num_groups=65, num_experts=65)):
        assert route(**kw) == UNSUPPORTED, kw
    for kw in (dict(num_experts=0), dict(topk=0), dict(num_groups=0), dict(num_groups=3), dict(ld=63), dict(topk=9, num_experts=8),
               dict(d_bias=P + 2), dict(num_groups=4), dict(num_groups=4, topk_groups=5, group_top=2),
               dict(num_groups=4, topk_groups=2, group_top=0), dict(num_groups=4, topk_groups=2, group_top=3),
               dict(num_groups=64, topk_groups=8, group_top=2), dict(num_groups=16, topk_groups=1, group_top=2),
               dict(T=1, logits=None), dict(T=1, ids=None), dict(T=1, w=None), dict(T=1, logits=P + 2), dict(T=1, logits=P + 1, dtype=1),
               dict(T=1, ids=P + 2), dict(T=1, w=P + 1)):
        assert route(**kw) == INVALID, kw
    assert route(num_groups=4, topk_groups=2, group_top=2) == OK and route(num_groups=64, topk_groups=8, group_top=1) == OK


def quantize(x=P, ldx=64, rows=0, width=64, dtype=1, act=0, m=None, q=P, ldq=64, s=P, a=None, lda=0):
    return L._lib.lora_quantize(x, ldx, rows, width, dtype, act, m, q, ldq, s, a, lda, None)


def test_quantize_refusals():
    assert quantize() == OK and quantize(act=1, ldx=128, a=P, lda=64) == OK and quantize(m=meta(0)) == OK
    for kw in (dict(dtype=2), dict(act=2), dict(act=-1), dict(width=(1 << 24) + 16, ldx=1 << 25, ldq=1 << 25),
               dict(rows=(1 << 30) + 1)):
        assert quantize(**kw) == UNSUPPORTED, kw
    for kw in (dict(rows=-1), dict(width=0), dict(width=8), dict(width=24), dict(ldx=56), dict(ldx=68), dict(act=1), dict(ldq=48),
               dict(ldq=72), dict(act=1, ldx=128, a=P, lda=56), dict(act=1, ldx=128, a=P, lda=66), dict(x=P + 8), dict(q=P + 8),
               dict(s=P + 2), dict(a=P + 8, lda=64), dict(m=meta(8)), dict(m=meta(0, div=2)), dict(m=meta(0, sorted=None)),
               dict(m=meta(0, keys=0)), dict(rows=1, x=None), dict(rows=1, q=None), dict(rows=1, s=None), dict(rows=4, m=meta(8))):
        assert quantize(**kw) == INVALID, kw


def weight(**kw):
    f = dict(ptr=P, expert_stride=0, row_stride=64, scale=P, bias=None, d_in=64, d_out=32, num_experts=1, reserved=0)
    f.update(kw)
    return C.byref(L.lora_int8_weight(**f))


def matmul(m=None, x=P, ldx=64, xs=P, rows=0, w=None, y=P, ldy=32, dtype=1, ws=None, ws_bytes=0):
    return L._lib.lora_int8_matmul(m, x, ldx, xs, rows, weight() if w is None else w, y, ldy, dtype, ws, ws_bytes, None)


def test_int8_matmul_refusals():
    n = C.c_size_t(7)
    assert matmul() == OK and L._lib.lora_int8_matmul_workspace_bytes(0, weight(), C.byref(n)) == OK
    assert matmul(w=weight(num_experts=4, expert_stride=2048), m=meta(0)) == OK
    bad = [(dict(ptr=None), INVALID), (dict(ptr=P + 8), INVALID), (dict(scale=None), INVALID), (dict(scale=P + 2), INVALID),
           (dict(bias=P + 2), INVALID), (dict(reserved=1), INVALID), (dict(num_experts=0), INVALID), (dict(d_in=0), INVALID),
           (dict(d_in=72, row_stride=80), INVALID), (dict(d_out=0), INVALID), (dict(d_out=12), INVALID), (dict(row_stride=48), INVALID),
           (dict(row_stride=72), INVALID), (dict(num_experts=4, expert_stride=2040), INVALID),
           (dict(num_experts=4, expert_stride=2032), INVALID), (dict(num_experts=1024, expert_stride=2048), UNSUPPORTED),
           (dict(d_in=131072, row_stride=131072), UNSUPPORTED), (dict(d_out=(1 << 24) + 8), UNSUPPORTED), (dict(row_stride=1 << 23), UNSUPPORTED)]
    for kw, st in bad:
        assert L._lib.lora_int8_matmul_workspace_bytes(1, weight(**kw), C.byref(n)) == st, kw
        assert matmul(w=weight(**kw)) == st, kw
    assert L._lib.lora_int8_matmul_workspace_bytes(1, None, C.byref(n)) == INVALID
    assert L._lib.lora_int8_matmul_workspace_bytes(1, weight(), None) == INVALID
    assert L._lib.lora_int8_matmul_workspace_bytes(-1, weight(), C.byref(n)) == INVALID
    assert matmul(dtype=2) == UNSUPPORTED and matmul(rows=(1 << 24) + 1) == UNSUPPORTED
    many = weight(num_experts=4, expert_stride=2048)
    for kw in (dict(rows=-1), dict(ldx=48), dict(ldx=72), dict(ldy=24), dict(ldy=36), dict(x=P + 8), dict(y=P + 8), dict(xs=P + 2),
               dict(rows=1, x=None), dict(rows=1, xs=None), dict(rows=1, y=None), dict(w=many), dict(w=many, m=meta(8)),
               dict(w=many, m=meta(0, keys=3)), dict(m=meta(0)), dict(w=many, m=meta(0, info=None)), dict(w=many, m=meta(0, div=0))):
        assert matmul(**kw) == INVALID, kw


def combine(y=P, ldy=64, width=64, dtype=1, ids=P, w=P, T=0, K=4, E=8, local=8, emap=None, add=None, ldadd=0, out=P, ldout=64):
    return L._lib.lora_moe_combine(y, ldy, width, dtype, ids, w, T, K, E, local, emap, add, ldadd, out, ldout, None)


def test_combine_refusals():
    assert combine() == OK and combine(add=P, ldadd=64) == OK and combine(emap=P) == OK
    for kw in (dict(dtype=2), dict(K=65), dict(T=(1 << 24) + 1), dict(width=(1 << 24) + 8, ldy=1 << 25, ldout=1 << 25)):
        assert combine(**kw) == UNSUPPORTED, kw
    for kw in (dict(T=-1), dict(K=0), dict(E=0), dict(local=0), dict(width=0), dict(width=12), dict(ldy=56), dict(ldy=68), dict(ldout=56),
               dict(ldout=68), dict(add=P, ldadd=56), dict(add=P, ldadd=66), dict(add=P, ldadd=72), dict(y=P + 8), dict(out=P + 8),
               dict(add=P + 8, ldadd=64), dict(ids=P + 2), dict(w=P + 2), dict(emap=P + 2), dict(T=1, y=None), dict(T=1, ids=None),
               dict(T=1, w=None), dict(T=1, out=None)):
        assert combine(**kw) == INVALID, kw


def test_binding_refusals(monkeypatch):
    """Shapes, types and strides that the C entry points cannot see."""
    monkeypatch.setattr(L, "_dev", lambda t, name: P)
    monkeypatch.setattr(L, "_stream_handle", lambda stream: 0)
    i8, f32, bf = torch.int8, torch.float32, torch.bfloat16
    z = lambda *s, dtype=f32: torch.zeros(s, dtype=dtype)  # noqa: E731
    r = L.Routing(8, 2)
    bad = [lambda: L.Routing(8, 2, score="relu"), lambda: L.Routing(8, 2, bias=z(7)), lambda: L.Routing(8, 2, bias=z(8, dtype=bf)),
           lambda: L.lora_moe_route(z(4, 7), r), lambda: L.lora_moe_route(z(8), r), lambda: L.lora_moe_route(z(8, 4).t(), r),
           lambda: L.lora_moe_route(z(4, 8), r, topk_ids=z(4, 2, dtype=torch.int64)),
           lambda: L.lora_moe_route(z(4, 8), r, topk_ids=z(4, 3, dtype=torch.int32)),
           lambda: L.lora_moe_route(z(4, 8), r, topk_ids=z(4, 2, dtype=torch.int32), weights=z(4, 4)[:, ::2]),
           lambda: L.lora_quantize(z(4, 16), activation="relu"), lambda: L.lora_quantize(z(4, 16), act=z(4, 16)),
           lambda: L.lora_quantize(z(16, 4).t()), lambda: L.lora_quantize(z(4, 33), activation="silu_mul"),
           lambda: L.lora_quantize(z(4, 16), q=z(4, 16)), lambda: L.lora_quantize(z(4, 16), q=z(3, 16, dtype=i8)),
           lambda: L.lora_quantize(z(4, 16), q=z(4, 16, dtype=i8), scale=z(5)),
           lambda: L.lora_quantize(z(4, 32), q=z(4, 16, dtype=i8), scale=z(4), activation="silu_mul", act=z(4, 16, dtype=bf)),
           lambda: L.Int8Weight(z(8, 16), z(8)), lambda: L.Int8Weight(z(8, 16, dtype=i8), z(7)),
           lambda: L.Int8Weight(z(2, 8, 16, dtype=i8), z(8)), lambda: L.Int8Weight(z(16, 8, dtype=i8).t(), z(8)),
           lambda: L.Int8Weight(z(8, 16, dtype=i8), z(8), bias=z(8, dtype=bf))]
    w = L.Int8Weight(z(8, 16, dtype=i8), z(8))
    bad += [lambda: L.lora_int8_matmul(z(4, 16), z(4), w), lambda: L.lora_int8_matmul(z(4, 32, dtype=i8), z(4), w),
            lambda: L.lora_int8_matmul(z(4, 16, dtype=i8), z(3), w),
            lambda: L.lora_int8_matmul(z(4, 16, dtype=i8), z(4), w, out=z(4, 9)),
            lambda: L.lora_int8_matmul(z(4, 16, dtype=i8), z(4), w, out=z(5, 8)),
            lambda: L.lora_moe_combine(z(8, 16), z(4, 2), z(4, 3, dtype=torch.int32)),
            lambda: L.lora_moe_combine(z(8, 16), z(4, 3), z(4, 2, dtype=torch.int32)),
            lambda: L.lora_moe_combine(z(8, 16), z(4, 2), z(4, 2, dtype=torch.int64)),
            lambda: L.lora_moe_combine(z(8, 16), z(4, 2), z(4, 2, dtype=torch.int32), out=z(4, 16, dtype=bf)),
            lambda: L.lora_moe_combine(z(8, 16), z(4, 2), z(4, 2, dtype=torch.int32), add=z(3, 16)),
            lambda: L.lora_moe_combine(z(8, 16), z(4, 2), z(4, 2, dtype=torch.int32), expert_map=z(8, dtype=torch.int32)),
            lambda: L.lora_moe_combine(z(8, 16), z(4, 2), z(4, 2, dtype=torch.int32), num_experts=9, num_local_experts=2,
                                       expert_map=z(8, dtype=torch.int32))]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
            print("call", i, "was taken")
    with pytest.raises(TypeError):
        L.lora_int8_matmul(z(4, 16, dtype=i8), z(4), w, dtype=torch.float16)
    with pytest.raises(L.LoraError):                 # a width that the library refuses
        L.lora_quantize(z(4, 24), q=z(4, 24, dtype=i8), scale=z(4))


def test_reference_forms():
    """The float64 forms themselves, on cases small enough to see."""
    x = torch.tensor([[1.0, 3.0, 2.0, 3.0], [-torch.inf, 0.0, -torch.inf, -torch.inf]])
    ids, w = R.route(x, 2, "softmax")
    assert ids.tolist() == [[1, 3], [1, 0]] and np.allclose(w, [[0.5, 0.5], [1, 0]])
    ids, w = R.route(x, 2, "sigmoid", torch.tensor([9.0, 0.0, 0.0, 0.0]), renorm=False)
    assert ids.tolist() == [[0, 1], [1, 0]] and np.allclose(w, [[0.73105858, 0.95257413], [0.5, 0]])
    # groups (0, 1) and (2, 3): the second has the larger sum
    ids, _ = R.route(torch.tensor([[5.0, 0.0, 4.0, 4.0]]), 2, "sigmoid", None, 2, 1)
    assert ids.tolist() == [[2, 3]]
    q, s = R.quantize(np.array([[127.0, 0.5, 1.5, -2.5, -127.0], [0, 0, 0, 0, 0]]))
    assert q.tolist() == [[127, 0, 2, -2, -127], [0] * 5] and s.tolist() == [1.0, 0.0]


def test_an_activation_that_is_none_is_not_written():
    """Without an activation there is nothing that d_act could take: refused, whatever its stride."""
    for kw in (dict(a=P, lda=64), dict(a=P, lda=64, rows=1), dict(a=P, lda=128, m=meta(0))):
        assert quantize(**kw) == INVALID, kw
    assert quantize(act=1, ldx=128, a=P, lda=64) == OK


def test_experts_side_by_side():
    """Matrices in each other's gaps are taken, overlapping ones refused."""
    n = C.c_size_t(7)
    ask = lambda **kw: L._lib.lora_int8_matmul_workspace_bytes(1, weight(num_experts=4, **kw), C.byref(n))  # noqa: E731
    assert ask(expert_stride=64, row_stride=256) == OK and ask(expert_stride=80, row_stride=304) == OK
    assert ask(expert_stride=2048, row_stride=64) == OK
    for es, rs in ((48, 256), (64, 240), (80, 288), (0, 64), (0, 256), (64, 64), (-64, 256), (256, 256), (-2048, 64)):
        assert ask(expert_stride=es, row_stride=rs) == INVALID, (es, rs)

"""lora_moe_route against the float64 form: scores, bias, groups, masked and non-finite
logits, equal and nearly equal values, strides, every size of expert set."""
import numpy as np
import pytest
import torch

import base_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    import segmented_gather_rank_amd as lib
    return lib


def check(L, logits, bias=None, **kw):
    """The call's outputs, checked."""
    topk = kw.pop("topk")
    r = L.Routing(logits.shape[1], topk, bias=bias, **{{"groups": "num_groups", "kept": "topk_groups", "renorm": "renormalize"}.get(k, k): v
                                                       for k, v in kw.items()})
    ids, w = L.lora_moe_route(logits, r)
    torch.cuda.synchronize()
    want, weights = R.route(logits, topk, kw.pop("score", "softmax"), bias, **kw)
    assert ids.dtype == torch.int32 and ids.shape == want.shape
    got = ids.cpu().numpy()
    wrong = (got != want).any(1)
    assert not wrong.any(), f"{wrong.sum()} tokens, first {np.argmax(wrong)}: {got[wrong][0]} for {want[wrong][0]}"
    # float64, rounded once; without renormalising, the softmax's sum has 16 float32 terms a lane, each an
    # exponential (2 steps, and half a step of an argument up to 104)
    renorm = kw.get("renorm", True)
    R.near(w, weights, np.abs(weights) * (R.F32 * (2 if renorm else 130)) + 1e-45, "weights")
    return ids, w


FORMS = [dict(), dict(renorm=False, scale=2.5), dict(score="sigmoid"), dict(score="sigmoid", renorm=False),
         dict(score="sigmoid", biased=True, scale=2.5), dict(biased=True), dict(biased=True, renorm=False)]


@pytest.mark.parametrize("form", FORMS, ids=str)
@pytest.mark.parametrize("T,E,topk", [(1, 1, 1), (1, 256, 8), (3, 2, 2), (5, 16, 16), (67, 60, 4), (130, 64, 6), (33, 100, 32),
                                      (129, 128, 8), (65, 200, 7), (1001, 256, 8), (40, 257, 8), (19, 512, 32), (7, 1000, 3),
                                      (6, 1024, 10)])
def test_route(L, T, E, topk, form):
    form = dict(form)
    g = torch.Generator("cuda").manual_seed(T + E)
    bias = 0.1 * torch.randn(E, generator=g, device="cuda") if form.pop("biased", False) else None
    for dtype in (torch.float32, torch.bfloat16):
        logits = (2 * torch.randn((T, E), generator=g, device="cuda")).to(dtype)
        check(L, logits, bias, topk=topk, **form)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("T,E,topk,groups,kept,top", [(1, 256, 8, 8, 4, 2), (300, 256, 8, 8, 4, 2), (65, 256, 8, 8, 1, 1),
                                                      (50, 60, 4, 4, 2, 2), (50, 64, 6, 64, 7, 1), (50, 8, 2, 4, 2, 2),
                                                      (20, 1024, 32, 16, 3, 2), (20, 96, 3, 3, 3, 2), (9, 320, 10, 10, 9, 1)])
def test_groups(L, T, E, topk, groups, kept, top, biased, score):
    g = torch.Generator("cuda").manual_seed(E + groups)
    bias = 0.1 * torch.randn(E, generator=g, device="cuda") if biased else None
    for dtype in (torch.float32, torch.bfloat16):
        logits = (2 * torch.randn((T, E), generator=g, device="cuda")).to(dtype)
        check(L, logits, bias, topk=topk, score=score, groups=groups, kept=kept, group_top=top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups,kept", [(1, 1), (8, 3)])
def test_equal_values(L, score, biased, groups, kept):
    """Few different logits, so that most choices are between equal ones: the lowest ids."""
    g = torch.Generator("cuda").manual_seed(5)
    logits = torch.randint(-2, 3, (200, 256), generator=g, device="cuda").bfloat16()
    logits[0] = 0
    bias = torch.zeros(256, device="cuda") if biased else None
    if biased:
        bias[::7] = 0.25
    check(L, logits, bias, topk=8, score=score, groups=groups, kept=kept)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_values_that_32_bits_cannot_tell_apart(L, score, groups):
    """Biases that bring the leading experts' values within a float32 step of each other."""
    g = torch.Generator("cuda").manual_seed(6)
    logits = torch.randn((400, 64), generator=g, device="cuda")
    x = logits[0].double()
    s = torch.softmax(x, 0) if score == "softmax" else torch.sigmoid(x)
    bias = (0.7 - s).float()            # every value of token 0 is 0.7 up to the bias's rounding
    logits[200:] = logits[0] + 1e-6 * torch.randn((200, 64), generator=g, device="cuda")
    check(L, logits, bias, topk=8, score=score, groups=groups, kept=2)
    # without bias: large logits, whose sigmoids are 1 in any precision
    check(L, 30 + torch.rand((100, 64), generator=g, device="cuda") * 20, None, topk=8, score=score, groups=groups, kept=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups,top", [(1, 1), (4, 2), (4, 1)])
def test_masked_and_non_finite(L, score, biased, groups, top):
    g = torch.Generator("cuda").manual_seed(7)
    E, topk = 32, 6
    logits = torch.randn((40, E), generator=g, device="cuda")
    logits[1] = -torch.inf                                   # nothing left
    logits[2, 3:] = -torch.inf                               # fewer than topk left
    logits[3, ::2] = -torch.inf
    logits[4, 5] = torch.inf
    logits[5, [2, 30]] = torch.inf                           # they share the mass
    logits[6, 7] = torch.nan
    logits[7] = torch.nan
    logits[8] = torch.finfo(torch.float32).min               # a mask of the lowest value, everywhere
    logits[9, 4:] = torch.finfo(torch.float32).min
    logits[10] = -200.0                                      # sigmoids that float32 has no normal numbers for
    logits[11] = 1e-45
    logits[12] = torch.finfo(torch.float32).max
    logits[13:20] = logits[13:20].masked_fill(torch.rand((7, E), generator=g, device="cuda") < 0.7, -torch.inf)
    bias = 0.1 * torch.randn(E, generator=g, device="cuda") if biased else None
    for renorm in (True, False):
        ids, w = check(L, logits, bias, topk=topk, score=score, groups=groups, kept=2, group_top=top, renorm=renorm)
        assert (w[1] == 0).all() and w[6].isnan().all() and not w[:6].isnan().any()
    if biased:
        bias[9] = torch.nan
        bias[3] = torch.inf
        bias[4] = -torch.inf
        ids, _ = L.lora_moe_route(logits, L.Routing(E, topk, score=score, bias=bias, num_groups=groups, topk_groups=2, group_top=top))
        ids = ids.cpu().numpy()
        assert ((ids >= 0) & (ids < E)).all() and all(len(set(r)) == topk for r in ids.tolist())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides_and_streams(L, dtype):
    """Rows that are part of wider ones, at odd places; outputs on another stream."""
    g = torch.Generator("cuda").manual_seed(8)
    wide = torch.randn((70, 300), generator=g, device="cuda").to(dtype)
    for off, E in ((0, 256), (1, 256), (3, 60), (44, 256), (7, 17)):
        check(L, wide[:, off:off + E], None, topk=4)
    check(L, wide[::2, :64], None, topk=4)
    r = L.Routing(256, 8)
    want = L.lora_moe_route(wide[:, :256].contiguous(), r)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream):
        got = L.lora_moe_route(wide[:, :256], r, stream=stream)
        s.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # nothing to do
    ids, w = L.lora_moe_route(wide[:0, :256], r)
    assert ids.shape == (0, 8) and w.shape == (0, 8)


def test_outputs_end_where_they_should(L):
    """Only the batch's rows are written."""
    logits = torch.randn((37, 60), device="cuda")
    ids = torch.full((50, 4), -7, dtype=torch.int32, device="cuda")
    w = torch.full((50, 4), -7.0, device="cuda")
    L.lora_moe_route(logits, L.Routing(60, 4), topk_ids=ids[5:42], weights=w[5:42])
    assert (ids[:5] == -7).all() and (ids[42:] == -7).all() and (w[:5] == -7).all() and (w[42:] == -7).all()
    assert (ids[5:42] >= 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,kept", [(16, 8, 3), (64, 8, 3), (66, 11, 4), (512, 16, 5)])
def test_group_ranks_that_cancel(L, score, E, groups, kept):
    """The two largest of a group are far larger than their sum: c's rounding goes by their sizes, the rank does not."""
    g = torch.Generator("cuda").manual_seed(E)
    size = E // groups
    bias = torch.full((groups, size), -3000.0, device="cuda")
    bias[:, 0], bias[:, 1] = 1000.0, -1000.0
    bias = bias.reshape(-1).contiguous()
    logits = 0.02 * torch.randn((3000, E), generator=g, device="cuda")
    ids, _ = check(L, logits, bias, topk=min(4, kept * size), score=score, groups=groups, kept=kept, group_top=2)
    assert len(torch.unique(ids[:, 0] // size)) == groups


def test_many_launches(L):
    """More tokens than one launch takes: as the same tokens in two calls."""
    T, cut = (1 << 26) + 37, (1 << 26) - 5
    g = torch.Generator("cuda").manual_seed(1)
    logits = torch.randn((T, 3), generator=g, device="cuda").bfloat16()
    r = L.Routing(3, 1)
    ids, w = L.lora_moe_route(logits, r)
    for part in (slice(0, cut), slice(cut, T)):
        i, v = L.lora_moe_route(logits[part], r)
        assert torch.equal(i, ids[part]) and torch.equal(v, w[part])
    best = logits.float().argmax(1).int()  # (equal logits: any of them)
    assert bool((logits.gather(1, best.long()[:, None]) == logits.gather(1, ids.long())).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,kept", [(16, 8, 3), (64, 8, 3), (66, 11, 4), (256, 8, 1), (512, 16, 5)])
def test_infinite_bias_beside_masked_experts(L, score, E, groups, kept):
    """A group of one +inf and masked experts has no rank (inf - inf is no number): it counts as -inf, like a masked group."""
    g = torch.Generator("cuda").manual_seed(E + 1)
    size = E // groups
    logits = torch.randn((60, E), generator=g, device="cuda")
    bias = 0.1 * torch.randn(E, generator=g, device="cuda")
    bias[size], bias[3 * size + 1] = torch.inf, torch.inf          # groups 1 and 3
    logits[:20, size + 1:2 * size] = -torch.inf
    logits[10:40, 3 * size] = -torch.inf
    logits[10:40, 3 * size + 2:4 * size] = -torch.inf
    logits[30:40, 4 * size:] = -torch.inf                          # what is left may be masked groups alone
    logits[50:60, :] = -torch.inf
    logits[50:60, size] = 0
    with np.errstate(invalid="ignore"):
        check(L, logits, bias, topk=min(4, kept * size), score=score, groups=groups, kept=kept, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("E,groups,kept", [(16, 8, 3), (64, 8, 3), (66, 11, 4), (512, 16, 5)])
def test_group_ranks_beyond_32_bits(L, score, top, E, groups, kept):
    """Biases whose sum of two is past the largest float32: the ranks are those of 64 bits."""
    g = torch.Generator("cuda").manual_seed(E + 2)
    size = E // groups
    logits = torch.randn((40, E), generator=g, device="cuda")
    largest = torch.finfo(torch.float32).max
    for sign in (1, -1):
        bias = sign * largest * (0.6 + 0.4 * torch.rand((groups, size), generator=g, device="cuda"))
        some = logits.clone().view(40, groups, size)
        some[20:, ::2, 1:] = -torch.inf                            # -inf is below every sum
        check(L, some.view(40, E), bias.view(-1), topk=min(4, kept * size), score=score, groups=groups, kept=kept, group_top=top)
        bias[...] = sign * largest                                 # equal in 64 bits too
        check(L, logits, bias.view(-1), topk=min(4, kept * size), score=score, groups=groups, kept=kept, group_top=top)


@pytest.mark.parametrize("E,gap", [(256, 16), (64, 4), (1024, 16)])
def test_softmax_sum_of_many_small_terms(L, E, gap):
    """Without renormalising: terms of just under half a float32 step of 1 beside the 1 of the largest logit, every one of
    which a sum in float32 drops."""
    logits = torch.full((5, E), -16.64, device="cuda")             # exp(-16.64) = 0.9956 * 2^-24
    logits[:, ::gap] = 0
    topk = 4
    ids, w = L.lora_moe_route(logits, L.Routing(E, topk, renormalize=False))
    want, weights = R.route(logits, topk, "softmax", renorm=False)
    assert (ids.cpu().numpy() == want).all()
    # a small term is off by the exponential's step and the rounding of its argument, (2 + 17) * 2^-24 of itself, and they
    # are less than 2^-19 of the sum together; the sum and the quotient are taken in 64 bits, the weight is rounded once
    R.near(w, weights, weights * R.F32 * (1 + 19 * 2.0 ** -19) + 1e-45, "weights")

"""lora_quantize against the float64 form: every width's kernel, halves and near halves,
the gated activation, rows that hold nothing or too much, metadata, strides."""
import numpy as np
import pytest
import torch

import base_ref as R

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module")
def L():
    import segmented_gather_rank_amd as lib
    return lib


def check_plain(L, x, **kw):
    q, s = L.lora_quantize(x, **kw)
    torch.cuda.synchronize()
    want, scale = R.quantize(R.f64(x))
    assert (q.cpu().numpy() == want).all(), np.argwhere(q.cpu().numpy() != want)[:5]
    assert np.array_equal(s.cpu().numpy(), scale, equal_nan=True)
    return q, s


def check_act(q, s, act, x, rows=None):
    """Against the activation in float64.  In float32 it is off by the exponential (2 steps, and half a step of an
    argument up to 104 on its way), the sum, the division, the product."""
    v = R.silu_mul(x)
    rows = np.arange(len(v)) if rows is None else rows
    v, size = v[rows], 110 * R.F32
    m = np.abs(v).max(1)
    R.near(s[rows], m / 127, m / 127 * (size + 2 * R.F32) + 1e-44, "scale")
    step = np.where(m > 0, m / 127, 1.0)[:, None]
    got = R.f64(q)[rows]
    assert (np.abs(got - v / step) <= 0.5 + 127 * 3 * size).all()
    if act is not None:
        R.near(act[rows], v, np.abs(v) * (size + R.HALF[act.dtype]) + 1e-40, "act")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,width", [(1, 16), (3, 48), (9, 512), (5, 528), (7, 1024), (1, 2048), (6, 2032), (5, 4096), (3, 4112),
                                        (2, 8192), (3, 14336), (2, 16384), (2, 16400), (1, 40000), (260, 128), (1, 4096)])
def test_rows(L, rows, width, dtype):
    g = torch.Generator("cuda").manual_seed(rows + width)
    x = torch.randn((rows, width), generator=g, device="cuda").to(dtype)
    check_plain(L, x)
    both = torch.randn((rows, 2 * width), generator=g, device="cuda").to(dtype)
    act = torch.empty((rows, width), dtype=dtype, device="cuda")
    q, s = L.lora_quantize(both, activation="silu_mul", act=act)
    check_act(q, s, act, both)
    q2, s2 = L.lora_quantize(both, activation="silu_mul")
    assert torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("dtype", DTYPES)
def test_halves(L, dtype):
    """Values on and next to the border between two integers."""
    m = 127.0 * 8
    n = torch.arange(-126, 126, dtype=torch.float64)
    x = torch.zeros((40, 1024), dtype=torch.float64)
    x[:, 0] = m
    x[:, 1:253] = (n + 0.5) * 8
    for i in range(40):                             # neighbours at a few float32 steps, and other largest values
        x[i, 300:552] = (n + 0.5) * 8 * (1 + (i - 20) * 2.0 ** -23)
        x[i, 1:553] *= 1.0 if i < 10 else 2.0 ** (i - 25)
        x[i, 0] *= 1.0 if i < 10 else 2.0 ** (i - 25)
    x[30:, 0] *= torch.rand(10, generator=torch.Generator().manual_seed(1), dtype=torch.float64) + 1
    check_plain(L, x.to(dtype).cuda())


@pytest.mark.parametrize("dtype", DTYPES)
def test_extremes(L, dtype):
    g = torch.Generator("cuda").manual_seed(2)
    x = torch.randn((16, 320), generator=g, device="cuda").to(dtype)
    big = torch.finfo(dtype).max
    x[1] = 0
    x[2] = -0.0
    x[3, 5] = torch.inf
    x[4, 7] = -torch.inf
    x[5, 9] = torch.nan
    x[6, 11] = big
    x[7] = big
    x[8] = -big
    x[9] *= 1e-37                                   # 127 / m leaves float32
    x[10] = 0
    x[10, 3] = 1e-45 if dtype == torch.float32 else 9.2e-41    # the smallest there is
    x[11] *= 1e-39
    x[12] *= 1e-30
    q, s = check_plain(L, x)
    assert s[3:6].isnan().all() and (q[3:6] == 0).all() and (q[1:3] == 0).all() and (s[1:3] == 0).all()
    assert (q[7] == 127).all() and (q[8] == -127).all()
    both = torch.randn((6, 640), generator=g, device="cuda").to(dtype)
    both[1, 3] = torch.nan
    both[2, 400] = torch.inf
    both[3, 0], both[3, 1], both[3, 2] = -1e4, 200.0, -90.0
    both[4, :320] = 0
    both[5, 8] = -torch.inf                         # -inf * 0
    act = torch.empty((6, 320), dtype=dtype, device="cuda")
    q, s = L.lora_quantize(both, activation="silu_mul", act=act)
    assert s[1].isnan() and s[2].isnan() and s[5].isnan() and (q[[1, 2, 5]] == 0).all() and (q[4] == 0).all() and s[4] == 0
    check_act(q, s, act, both, np.array([0, 3, 4]))


@pytest.mark.parametrize("dtype", DTYPES)
def test_strides(L, dtype):
    """Parts of wider matrices: nothing but the rows is written."""
    g = torch.Generator("cuda").manual_seed(3)
    wide = torch.randn((33, 400), generator=g, device="cuda").to(dtype)
    x = wide[:, 16:16 + 256]
    q = torch.full((33, 320), 99, dtype=torch.int8, device="cuda")
    check_plain(L, x, q=q[:, 32:288])
    assert (q[:, :32] == 99).all() and (q[:, 288:] == 99).all()
    act = torch.full((33, 160), 7.0, dtype=dtype, device="cuda")
    q2, s2 = L.lora_quantize(x, activation="silu_mul", act=act[:, 16:144])
    check_act(q2, s2, act[:, 16:144], x)
    assert (act[:, :16] == 7).all() and (act[:, 144:] == 7).all()
    q3, s3 = L.lora_quantize(x[:0])
    assert q3.shape == (0, 256) and s3.shape == (0,)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,topk,local", [(1, 1, 1), (37, 4, 5), (300, 8, 2)])
def test_metadata(L, T, topk, local, dtype):
    """Only rows with a key are read and written."""
    g = torch.Generator("cuda").manual_seed(T)
    E, width = 16, 1040
    ids = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(t))[:topk] for t in range(T)]).int().cuda()
    emap = torch.full((E,), -1, dtype=torch.int32, device="cuda")
    emap[3:3 + local] = torch.arange(local, dtype=torch.int32, device="cuda")
    meta = L.lora_prepare_moe_meta(ids, torch.zeros(T, dtype=torch.int32, device="cuda"), 1, E, local, emap).with_x_row_div(1)
    here = ((ids >= 3) & (ids < 3 + local)).view(-1).cpu().numpy()
    x = torch.randn((T * topk, 2 * width), generator=g, device="cuda").to(dtype)
    x[torch.from_numpy(~here).cuda()] = torch.nan
    q = torch.full((T * topk, width), 99, dtype=torch.int8, device="cuda")
    s = torch.full((T * topk,), 7.0, device="cuda")
    act = torch.full((T * topk, width), 7.0, dtype=dtype, device="cuda")
    L.lora_quantize(x, q=q, scale=s, activation="silu_mul", act=act, meta=meta)
    away = torch.from_numpy(~here).cuda()
    assert (q[away] == 99).all() and (s[away] == 7).all() and (act[away] == 7).all()
    if here.any():
        check_act(q, s, act, x, np.nonzero(here)[0])


def test_many_launches(L):
    """More rows than one launch takes: as the same rows in two calls; with metadata, only its rows."""
    rows, cut = (1 << 23) + 37, (1 << 23) - 5
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn((rows, 16), generator=g, device="cuda").bfloat16()
    q, s = L.lora_quantize(x)
    for part in (slice(0, cut), slice(cut, rows)):
        a, b = L.lora_quantize(x[part])
        assert torch.equal(a, q[part]) and torch.equal(b, s[part])
    check_plain(L, x[-50:])
    slots = torch.randint(-1, 2, (rows,), generator=g, device="cuda", dtype=torch.int32)
    some, scale = torch.full_like(q, 5), torch.full_like(s, 5.0)
    L.lora_quantize(x, q=some, scale=scale, meta=L.lora_prepare_meta(slots, 2))
    here = slots >= 0
    assert torch.equal(some[here], q[here]) and torch.equal(scale[here], s[here])
    assert bool((some[~here] == 5).all()) and bool((scale[~here] == 5).all())


@pytest.mark.parametrize("gate", [(-87.0, 0.0), (0.0, 87.0), (-1.0, 1.0)])
def test_gate_in_32_bits(L, gate):
    """The gated activation in float32, where no part of it leaves the normal numbers."""
    g = torch.Generator("cuda").manual_seed(4)
    width = 4096
    both = torch.empty((32, 2 * width), device="cuda")
    both[:, :width] = gate[0] + (gate[1] - gate[0]) * torch.rand((32, width), generator=g, device="cuda")
    both[:, width:] = 0.5 + torch.rand((32, width), generator=g, device="cuda")
    act = torch.empty((32, width), device="cuda")
    q, s = L.lora_quantize(both, activation="silu_mul", act=act)
    v = R.silu_mul(both)
    # e = exp(-|x|) is a square of the hardware's exponential (a step, 2 * 2^-24, twice; the square's rounding), corrected
    # by what its argument's rounding left out (another rounding): 6 * 2^-24.  1 + e is rounded, its inverse is the
    # hardware's (a step); then three products.  Where e stands alone it is off in e / (1 + e) by 6, else by at most half
    # of that.
    R.near(act, v, np.abs(v) * 12 * R.F32 * (1 + 1e-5) + 1e-45, "act")
    m = np.abs(v).max(1)
    R.near(s, m / 127, m / 127 * 13 * R.F32 * (1 + 1e-5) + 1e-45, "scale")


@pytest.mark.parametrize("dtype", DTYPES)
def test_gate_of_values_that_are_not_finite(L, dtype):
    """act is the formula's value there: inf * u, and no number where the quotient is inf / inf."""
    both = torch.ones((1, 32), dtype=dtype, device="cuda")
    both[0, :7] = torch.tensor([torch.inf, torch.inf, torch.inf, -torch.inf, torch.nan, 3e38, -3e38])
    both[0, 16:23] = torch.tensor([2.0, -1.0, 0.0, 1.0, 1.0, 1.0, 1.0])
    act = torch.empty((1, 16), dtype=dtype, device="cuda")
    q, s = L.lora_quantize(both, activation="silu_mul", act=act)
    want = torch.tensor([torch.inf, -torch.inf, torch.nan, torch.nan, torch.nan, float(both[0, 5]), 0.0], dtype=dtype)
    assert torch.equal(act[0, :7].cpu().nan_to_num(nan=7.0, posinf=1e3, neginf=-1e3), want.nan_to_num(nan=7.0, posinf=1e3, neginf=-1e3))
    assert bool(s.isnan().all()) and not q.any()

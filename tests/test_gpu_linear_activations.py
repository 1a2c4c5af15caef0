"""zero_linear's activations and their slopes over every finite 16-bit number, against float64.

A layer with one input that is 1 and weights that are the numbers: z is exactly the number, y its activation; the
bias gradient of one row with dy = 1 is the slope, rounded once.

Tolerances.  One rounding to 16 bits: u16 of the value (2^-25 for fp16's subnormal numbers).  fp32: an
exponential's argument below 2^7 that carries 4 roundings makes 2^-24 4 2^7 = 2^-15 of its value; every term of a
value or a slope has that much of its own magnitude.  A logistic or exponential below 2^-126 becomes 0: at most 2^-126 times
the polynomial beside it, |z| (1 + z^2) with |z| below 100 where the functions are not 0 or 1 to the last
place, so less than 2^-105.
"""
import math

import pytest
import torch

import zero_sharded_mixed_03_gb300 as Z

pytestmark = pytest.mark.gpu
ACTS = {"none": Z.ZERO_ACT_NONE, "relu": Z.ZERO_ACT_RELU, "gelu_tanh": Z.ZERO_ACT_GELU_TANH,
        "gelu": Z.ZERO_ACT_GELU, "silu": Z.ZERO_ACT_SILU}
DTYPES = {"bf16": (torch.bfloat16, Z.ZERO_BF16, 2.0 ** -8, 2.0 ** -105),
          "fp16": (torch.float16, Z.ZERO_FP16, 2.0 ** -11, 2.0 ** -25)}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    Z.lib()
    yield
    Z.zero_operators_check()


def numbers(t):
    v = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(t)
    return v[torch.isfinite(v)].cuda()


def value64(z, act):
    """(value, slope, magnitudes of the slope's terms)"""
    one = torch.ones_like(z)
    if act == "none":
        return z, one, one
    if act == "relu":
        return torch.where(z > 0, z, 0.0), (z > 0).double(), one
    if act == "gelu":
        cdf = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        bell = z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        return z * cdf, cdf + bell, cdf + bell.abs()
    u = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3) if act == "gelu_tanh" else z
    du = 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z) if act == "gelu_tanh" else one
    s = torch.sigmoid(u)
    rest = z * s * torch.sigmoid(-u) * du
    return z * s, s + rest, s + rest.abs()


def near(got, want, magnitude, u16, floor):
    bound = u16 * want.abs() + 2.0 ** -15 * magnitude + floor
    # what rounds beyond the type's largest number becomes infinite: none of these do
    off = (got.double() - want).abs()
    assert bool((off <= bound).all()), [(float(a), float(b)) for a, b in zip(got[~(off <= bound)][:4], want[~(off <= bound)][:4])]


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,shift", [(1, 0), (1, 1), (5, 0), (5, 1)])
def test_values(act, dtype, rows, shift):
    """By the few rows' kernel, by tiles, and by tiles whose rows do not start on 16 bytes."""
    t, kind, u16, floor = DTYPES[dtype]
    z = numbers(t)
    n = z.numel() - shift                          # a multiple of eight columns, and one less
    w = torch.zeros(n, 8, dtype=t, device="cuda")
    w[:, 0] = z[:n]
    x = torch.zeros(rows, 8, dtype=t, device="cuda")
    x[:, 0] = 1.0
    y, pre = (torch.full((rows, n), 3.0, dtype=t, device="cuda") for _ in range(2))
    a = Z.zero_linear_t(rows=rows, in_features=8, out_features=n, dtype16=kind, layout=Z.ZERO_WEIGHT_OUT_IN,
                        activation=ACTS[act], x=x.data_ptr(), w=w.data_ptr(), y=y.data_ptr(), pre=pre.data_ptr())
    size = Z.zero_linear_workspace(a)
    ws = torch.empty(max(16, size), dtype=torch.uint8, device="cuda")
    Z.zero_linear(a, ws.data_ptr(), size, torch.cuda.current_stream().cuda_stream)
    z64 = z[:n].double()
    want = value64(z64, act)[0]
    for r in range(rows):
        near(pre[r], z64, z64.abs(), 0.0, floor)
        near(y[r], want, want.abs(), u16, floor)


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shift", [0, 1])
def test_slopes(act, dtype, shift):
    t, kind, u16, floor = DTYPES[dtype]
    z = numbers(t)
    n = z.numel()
    storage = torch.zeros(n + 8, dtype=t, device="cuda")
    pre = storage[shift:shift + n]
    pre.copy_(z)
    dy, db = torch.ones(n, dtype=t, device="cuda"), torch.empty(n, dtype=t, device="cuda")
    dw = torch.empty(n, 8, dtype=t, device="cuda")
    x = torch.zeros(1, 8, dtype=t, device="cuda")
    x[0, 3] = 1.0
    a = Z.zero_linear_t(rows=1, in_features=8, out_features=n, dtype16=kind, layout=Z.ZERO_WEIGHT_OUT_IN, activation=ACTS[act],
                        x=x.data_ptr(), pre=pre.data_ptr(), dy=dy.data_ptr(), dw=dw.data_ptr(), dbias=db.data_ptr())
    size = Z.zero_linear_workspace(a, True)
    ws = torch.empty(max(16, size), dtype=torch.uint8, device="cuda")
    Z.zero_linear_backward(a, ws.data_ptr(), size, torch.cuda.current_stream().cuda_stream)
    _, slope, magnitude = value64(z.double(), act)
    near(db, slope, magnitude, u16, floor)
    near(dw[:, 3], slope, magnitude, u16, floor)           # dz itself, through a product with 1
    assert not bool(dw[:, [0, 1, 2, 4, 5, 6, 7]].any())


@pytest.mark.parametrize("act", list(ACTS))
def test_not_a_number_stays_so(act):
    """NaN's own value and slope are NaN, its neighbours' their own."""
    t = torch.bfloat16
    pre = torch.tensor([1.0, math.nan, -1.0, 2.0, -2.0, 0.5, -0.5, 0.25], dtype=t, device="cuda").repeat(2)
    n = pre.numel()
    dy, db = torch.ones(n, dtype=t, device="cuda"), torch.empty(n, dtype=t, device="cuda")
    a = Z.zero_linear_t(rows=1, in_features=8, out_features=n, dtype16=Z.ZERO_BF16, layout=Z.ZERO_WEIGHT_OUT_IN, activation=ACTS[act],
                        pre=pre.data_ptr(), dy=dy.data_ptr(), dbias=db.data_ptr())
    size = Z.zero_linear_workspace(a, True)
    ws = torch.empty(max(16, size), dtype=torch.uint8, device="cuda")
    Z.zero_linear_backward(a, ws.data_ptr(), size, torch.cuda.current_stream().cuda_stream)
    assert torch.equal(torch.isnan(db), torch.isnan(pre) if act != "none" else torch.zeros_like(db, dtype=torch.bool))


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,cols", [(1000, 264), (257, 101), (5, 4096)])
def test_bias_gradients_sum_what_is_not_rounded(act, dtype, rows, cols):
    """dbias adds dz in fp32, before the rounding that the products' operand takes: random signs leave a sum far below its
    terms, of which that rounding would be 2^-8.  A term's fp32 part is 2^-17 of its magnitudes (arguments
    below 2^5), the sum's rows + 64 roundings."""
    t, kind, u16, _ = DTYPES[dtype]
    gen = torch.Generator(device="cuda").manual_seed(rows)
    pre, dy = (torch.randn(rows, cols, generator=gen, device="cuda").to(t) for _ in range(2))
    pre[:, 0] = pre[:, 0].sign() * 3                       # a column whose slopes are alike, with signs in turn
    dy[:, 0] = 1 - 2.0 * (torch.arange(rows, device="cuda") % 2).to(t)
    db = torch.empty(cols, dtype=t, device="cuda")
    a = Z.zero_linear_t(rows=rows, in_features=8, out_features=cols, dtype16=kind, layout=Z.ZERO_WEIGHT_OUT_IN, activation=ACTS[act],
                        pre=pre.data_ptr(), dy=dy.data_ptr(), dbias=db.data_ptr())
    size = Z.zero_linear_workspace(a, True)
    ws = torch.empty(max(16, size), dtype=torch.uint8, device="cuda")
    Z.zero_linear_backward(a, ws.data_ptr(), size, torch.cuda.current_stream().cuda_stream)
    _, slope, magnitude = value64(pre.double(), act)
    want, mag = (dy.double() * slope).sum(0), (dy.double().abs() * magnitude).sum(0)
    bound = (2.0 ** -17 + (rows + 64) * 2.0 ** -24) * mag + u16 * want.abs() + 2.0 ** -25
    off = (db.double() - want).abs()
    assert bool((off <= bound).all()), float((off / bound).max())

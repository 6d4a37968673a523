"""moe_linear_w4 on the GPU against the fp64 oracle, within the bound of its fp32 sums."""
import math

import numpy as np
import pytest
import torch

import bit_quantized_grouped_router_amd as M
from oracle import kv4_oracle as K
from oracle.moe_oracle import bf16_to_f64, round_to_bf16_bits
from parity_util import host_bits, say

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M.lib()
    yield
    torch.cuda.synchronize()


def rounded(a):
    return bf16_to_f64(round_to_bf16_bits(np.asarray(a, dtype=np.float64)))


def make_w(rng, rows, cols, general=False):
    """Quantised normal weights; general: random codes, scales of both signs and any bias."""
    if general:
        codes = rng.integers(0, 256, (rows, cols // 2), dtype=np.uint8)
        s = round_to_bf16_bits(rng.standard_normal((rows, cols // 64)) * np.exp2(rng.integers(-12, 3, (rows, cols // 64))))
        b = round_to_bf16_bits(rng.standard_normal((rows, cols // 64)) * np.exp2(rng.integers(-30, 3, (rows, cols // 64))))
    else:
        q, s, b = K.quantise(rng.standard_normal((rows, cols)) * cols ** -0.5)
        codes = K.pack(q)
    up = lambda a: torch.from_numpy(a[None].view(np.int16) if a.dtype == np.uint16 else a[None]).cuda()  # noqa: E731
    return M.W4Matrix(up(codes), up(s), up(b)), K.weights(codes, s, b)


def bound(x, w, z, y, dtype):
    """cols + 8 roundings of at most 2^-24 of the sum of the products' magnitudes, through an
    activation of slope at most 1.13; a few ulp for its own arithmetic (exp and erf of hardware
    to 2^-20) and the final rounding."""
    return (1.13 * (x.shape[1] + 8) * 2.0 ** -24 * (np.abs(x) @ np.abs(w).T) + 2.0 ** -20 * (np.abs(z) + np.abs(y))
            + (2.0 ** -8 if dtype == BF16 else 2.0 ** -23) * np.abs(y) + 1e-30)


def check(got, want, tol, what):
    got = got.float().cpu().numpy().astype(np.float64)
    off = np.abs(got - want)
    say(f"  {what}: worst {float((off / tol).max()):.3f} of the bound")
    assert np.isfinite(got).all() and (off <= tol).all(), what


CASES = [  # T, rows, cols, bias, act, residual, dtype
    (1, 1, 64, False, "none", False, F32),
    (1, 16, 64, True, "none", False, BF16),
    (1, 1003, 2048, True, "silu", True, BF16),
    (2, 17, 128, False, "relu", False, F32),
    (15, 64, 192, True, "gelu", True, F32),
    (16, 33, 4096, False, "none", True, F32),
    (17, 100, 512, True, "silu", False, BF16),
    (33, 256, 1024, False, "gelu", False, BF16),
    (64, 130, 320, True, "none", True, BF16),
    (65, 48, 704, False, "relu", True, F32),
    (127, 257, 256, True, "none", False, F32),
    (128, 256, 2048, False, "none", False, BF16),
    (129, 255, 64, True, "silu", True, F32),
    (300, 512, 576, True, "gelu", True, BF16),
    (513, 769, 1088, False, "none", True, F32),
    (1000, 77, 640, True, "relu", False, BF16),
    (2, 300, 6400, True, "none", False, F32),                # more columns than a fused expert takes
    # narrow tiles (more than 256 blocks of 32 tokens by 16 rows): groups left over by four
    # teams, fewer groups than teams, more than one table of 8 a team
    (70, 2100, 704, True, "gelu", True, BF16),
    (400, 520, 64, False, "none", True, F32),
    (257, 777, 128, True, "silu", False, F32),
    (90, 2200, 1216, False, "none", False, F32),
    (333, 1000, 2048, True, "relu", True, BF16),
    (170, 2100, 704, True, "gelu", True, BF16),
    (700, 520, 64, False, "none", True, F32),
    (450, 777, 128, True, "silu", False, F32),
    (170, 2200, 1216, False, "none", False, F32),
    (100, 2100, 2240, True, "silu", False, BF16),
    (64, 2049, 512, False, "none", False, BF16),             # 258 blocks, and 256 below
    (64, 2048, 512, False, "none", False, BF16),
    # middle tiles (more than 256 narrow ones): an odd number of groups, one, two, and more
    # than one table of 8 a team
    (1100, 1100, 704, True, "gelu", True, BF16),
    (1300, 900, 64, False, "none", True, F32),
    (1030, 1090, 128, True, "silu", False, F32),
    (1200, 1000, 1216, False, "none", False, F32),
    (1025, 1000, 256, False, "none", False, BF16),           # 272 narrow tiles, and 256 below
    (1024, 1000, 256, False, "none", False, BF16),
    # large tiles (220 of 128 x 256 and more): tails in both directions, few and many groups
    (2100, 3400, 64, True, "none", True, BF16),
    (3700, 2050, 576, False, "silu", False, F32),
    (1900, 3900, 1152, True, "none", False, BF16),
]


@pytest.mark.parametrize("general", [False, True])
@pytest.mark.parametrize("T,rows,cols,bias,act,residual,dtype", CASES)
def test_linear(T, rows, cols, bias, act, residual, dtype, general):
    rng = np.random.default_rng(T * 31 + rows + cols)
    w, w64 = make_w(rng, rows, cols, general)
    x = rounded(rng.standard_normal((T, cols)))
    b = rounded(rng.standard_normal(rows)) if bias else None
    r = rng.standard_normal((T, rows)).astype(np.float32)
    r = rounded(r) if dtype == BF16 else r.astype(np.float64)
    xd = torch.from_numpy(x).cuda().to(BF16)
    got = M.moe_linear_w4(xd, w, bias=None if b is None else torch.from_numpy(b).cuda().to(BF16), act=act,
                          residual=torch.from_numpy(r).cuda().to(dtype) if residual else None, out_dtype=dtype)
    assert got.dtype == dtype
    z = x @ w64.T + (0 if b is None else b)
    want = K.linear(x, w64, b, act, r if residual else None)
    tol = bound(x, w64, z, want, dtype) + (2.0 ** -23 * np.abs(r) if residual else 0)
    check(got, want, tol, f"{T}x{rows}x{cols} {act}")


@pytest.mark.parametrize("T", [1, 20, 200])
def test_strides_and_in_place(T):
    """Rows of x, residual and y inside wider tensors; y onto the residual; the rest untouched."""
    rng = np.random.default_rng(T)
    w, w64 = make_w(rng, 50, 128)
    wide = torch.from_numpy(rounded(rng.standard_normal((T, 192)))).cuda().to(BF16)
    x = wide[:, 64:]
    room = torch.from_numpy(rng.standard_normal((T, 61)).astype(np.float32)).cuda()
    before = room.cpu().numpy().astype(np.float64)
    y = room[:, :50]
    assert M.moe_linear_w4(x, w, residual=y, y=y) is y
    xs = x.float().cpu().numpy().astype(np.float64)
    want = K.linear(xs, w64, residual=before[:, :50])
    check(y, want, bound(xs, w64, want, want, F32) + 2.0 ** -23 * np.abs(before[:, :50]), "in place")
    assert (room[:, 50:].cpu().numpy() == before[:, 50:].astype(np.float32)).all()


@pytest.mark.parametrize("T", [1, 40, 300])
def test_activation_extremes(T):
    """Saturated activations stay finite; infinities and NaN of a token stay with it."""
    rng = np.random.default_rng(3)
    w, w64 = make_w(rng, 64, 64)
    x = rounded(rng.standard_normal((T, 64)) * 500)
    xd = torch.from_numpy(x).cuda().to(BF16)
    for act in ("relu", "silu", "gelu"):
        z = x @ w64.T
        with np.errstate(over="ignore"):
            want = K.linear(x, w64, act=act)
        check(M.moe_linear_w4(xd, w, act=act, out_dtype=F32), want, bound(x, w64, z, want, F32) + 1e-6, act)
    if T > 1:
        clean = M.moe_linear_w4(xd, w, out_dtype=F32)
        xd[1, 5], xd[T - 1, 6] = float("nan"), float("inf")
        got = M.moe_linear_w4(xd, w, out_dtype=F32)
        keep = [t for t in range(T) if t not in (1, T - 1)]
        assert torch.equal(got[keep], clean[keep])
        assert torch.isnan(got[1]).all() and not torch.isfinite(got[T - 1]).any()


TILES = [(200, 2100), (1100, 1100), (2100, 3300)]  # narrow, middle and large tiles


@pytest.mark.parametrize("T,rows", TILES)
@pytest.mark.parametrize("dtype,pad", [(F32, 11), (BF16, 8), (BF16, 3)])
def test_tiles_inside_wider_tensors_and_in_place(T, rows, dtype, pad):
    rng = np.random.default_rng(T + pad)
    w, w64 = make_w(rng, rows, 128)
    wide = torch.from_numpy(rounded(rng.standard_normal((T, 192)))).cuda().to(BF16)
    x = wide[:, 64:]
    room = torch.from_numpy(rng.standard_normal((T, rows + pad)).astype(np.float32)).cuda().to(dtype)
    before = room.double().cpu().numpy()
    y = room[:, :rows]
    M.moe_linear_w4(x, w, residual=y, y=y, act="relu")
    xs = x.double().cpu().numpy()
    z = xs @ w64.T
    want = K.linear(xs, w64, act="relu", residual=before[:, :rows])
    check(y, want, bound(xs, w64, z, want, dtype) + 2.0 ** -23 * np.abs(before[:, :rows]), f"{T} in place")
    assert (room[:, rows:].double().cpu().numpy() == before[:, rows:]).all()


@pytest.mark.parametrize("T,rows", TILES)
def test_tiles_keep_tokens_apart(T, rows):
    rng = np.random.default_rng(T)
    w, w64 = make_w(rng, rows, 128)
    x = rounded(rng.standard_normal((T, 128)) * 500)
    xd = torch.from_numpy(x).cuda().to(BF16)
    z = x @ w64.T
    clean = M.moe_linear_w4(xd, w, act="silu", out_dtype=F32)
    with np.errstate(over="ignore"):
        check(clean, K.linear(x, w64, act="silu"), bound(x, w64, z, z, F32) + 1e-6, "silu")
    xd[1, 5], xd[T - 1, 6] = float("nan"), float("inf")
    got = M.moe_linear_w4(xd, w, act="silu", out_dtype=F32)
    keep = [t for t in range(T) if t not in (1, T - 1)]
    assert torch.equal(got[keep], clean[keep])
    assert torch.isnan(got[1]).all() and not torch.isfinite(got[T - 1]).all()


def test_matches_the_dequantised_matrix_and_repeats():
    rng = np.random.default_rng(8)
    w, w64 = make_w(rng, 96, 256, general=True)
    assert (bf16_to_f64(host_bits(M.moe_dequant_w4(w))) == w64).all()
    x = torch.randn((70, 256), device="cuda").to(BF16)
    a = M.moe_linear_w4(x, w)
    for _ in range(3):
        assert torch.equal(a, M.moe_linear_w4(x, w))


def test_binding_refusals():
    rng = np.random.default_rng(9)
    w, _ = make_w(rng, 32, 128)
    x = torch.zeros((4, 128), dtype=BF16, device="cuda")
    ok = torch.zeros((4, 32), device="cuda")
    for bad in (dict(x=x.float()), dict(x=x[:, :64]), dict(x=x.t()), dict(x=x.cpu()), dict(act="swish"),
                dict(residual=ok[:3]), dict(residual=ok, out_dtype=BF16), dict(y=ok.half()), dict(y=ok, residual=ok.to(BF16)),
                dict(bias=torch.zeros(32, device="cuda")), dict(bias=torch.zeros(31, dtype=BF16, device="cuda")),
                dict(y=torch.zeros((32, 4), device="cuda").t()), dict(y=ok[:1].expand(4, 32)),
                dict(x=torch.zeros((4, 132), dtype=BF16, device="cuda")[:, :128])):
        a = dict(x=x)
        a.update(bad)
        with pytest.raises(M.MoeError):
            M.moe_linear_w4(a.pop("x"), w, **a)
    assert M.moe_linear_w4(x[:0], w).shape == (0, 32)


@pytest.mark.parametrize("T,rows", [(1, 20), (40, 20)] + TILES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gelu_keeps_its_digits_far_from_zero(T, rows, dtype):
    """z erfc(-z / sqrt 2) / 2 for z down to -12, relative to itself: the argument is off by 2^-23
    of itself (its product and the constant), which z^2 + 1 takes into erfc, and erfc and the two
    products by 16 steps of 2^-24 together; z itself is exact (one product of ones)."""
    z = rounded(np.linspace(-12.0, 6.0, T) if T > 1 else np.array([-6.5]))
    x = np.zeros((T, 64))
    x[:, 5] = z
    ones = M.W4Matrix(torch.zeros((1, rows, 32), dtype=torch.uint8, device="cuda"),
                      torch.zeros((1, rows, 1), dtype=BF16, device="cuda"),
                      torch.ones((1, rows, 1), dtype=BF16, device="cuda"))
    got = M.moe_linear_w4(torch.from_numpy(x).cuda().to(BF16), ones, act="gelu", out_dtype=dtype)
    got = got.double().cpu().numpy()
    want = np.array([v * math.erfc(-v / math.sqrt(2.0)) / 2.0 for v in z])[:, None]
    tol = ((z ** 2 + 1) * 2.0 ** -23 + 2.0 ** -20)[:, None] + (2.0 ** -8 if dtype == BF16 else 0)
    worst = float((np.abs(got - want) / (tol * np.abs(want) + 1e-300)).max())
    say(f"  gelu {T}: worst {worst:.3f} of the bound")
    assert worst <= 1

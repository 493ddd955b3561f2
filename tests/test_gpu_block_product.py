"""The frozen product over E4M3 codes with 128-blocks, and its quantisation, against float64.

Codes and scales are decided in fp32 on both sides and must be bit-exact. A product's value is
rounded to bf16 once (2^-9 relative) from sums whose terms the tensor cores may align before
adding; 2^-12 of the sum of the terms' magnitudes is allowed for that, element by element, and the
2-norm of the error over the 2-norm of the result stays under 3e-3 (a uniformly distributed bf16
rounding alone gives 1.7e-3).
"""
import numpy as np
import pytest
import torch

from oracle import sublayer_oracle as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_adapter_adamw_gb300 import binding
    return binding


def _bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16)


def _weight(rng, out_d, in_d):
    w = rng.standard_normal((out_d, in_d)) / np.sqrt(in_d)
    # neighbouring blocks of very different size, so that a scale of the wrong block shows
    grow = np.exp(rng.uniform(-3, 3, (-(-out_d // 128), -(-in_d // 128))))
    w *= np.repeat(np.repeat(grow, 128, 0), 128, 1)[:out_d, :in_d]
    return S.quantize_blocks(_bf16(w).float().numpy(), 128, 128)


def _acts(rng, T, K):
    x = rng.standard_normal((T, K))
    x *= np.repeat(np.exp(rng.uniform(-3, 3, (T, -(-K // 128)))), 128, 1)[:, :K]
    return _bf16(x)


def _run(L, X, c, s, out_d, in_d, dx, Y=None, stream=None):
    T = X.shape[0]
    if Y is None:
        Y = torch.full((T, in_d if dx else out_d), float("nan"), dtype=torch.bfloat16, device="cuda")
    n = L.lora_block_product_workspace_size(T, out_d, in_d, dx)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    L.lora_block_product(T, out_d, in_d, X, c, s, Y, dx, ws, stream=stream)
    return Y


def _check(Y, ref, mag):
    y = Y.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(y).all()
    assert np.all(np.abs(y - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -12 * mag)
    assert np.linalg.norm(y - ref) <= 3e-3 * np.linalg.norm(ref)


@pytest.mark.parametrize("rows,K", [(1, 16), (7, 128), (33, 144), (5, 4112), (260, 1536)])
def test_activation_blocks_bit_exact(L, rows, K):
    rng = np.random.default_rng(rows * 7 + K)
    X = _acts(rng, rows, K)
    X[0, :16] = 0.0
    codes = torch.empty((rows, K), dtype=torch.uint8, device="cuda")
    scales = torch.empty((rows, -(-K // 128)), device="cuda")
    L.lora_block_quantize(X.cuda(), rows, K, codes, scales)
    torch.cuda.synchronize()
    c, s = S.quantize_blocks(X.float().numpy(), 1, 128)
    assert np.array_equal(codes.cpu().numpy(), c)
    assert np.array_equal(scales.cpu().numpy(), s)


@pytest.mark.parametrize("out_d,in_d", [(16, 16), (128, 128), (144, 272), (256, 1536)])
def test_weight_blocks_bit_exact(L, out_d, in_d):
    rng = np.random.default_rng(out_d + in_d)
    W = _bf16(rng.standard_normal((out_d, in_d)) * 1e-2)
    W[:128, :128] = 0.0
    codes = torch.empty((out_d, in_d), dtype=torch.uint8, device="cuda")
    scales = torch.empty((-(-out_d // 128), -(-in_d // 128)), device="cuda")
    L.lora_block_quantize_weight(W.cuda(), out_d, in_d, codes, scales)
    torch.cuda.synchronize()
    c, s = S.quantize_blocks(W.float().numpy(), 128, 128)
    assert np.array_equal(codes.cpu().numpy(), c)
    assert np.array_equal(scales.cpu().numpy(), s)


# one token to several tiles; odd token counts; widths below, at and past the block and the tile;
# contractions of one partial block, of whole blocks, of many blocks
SHAPES = [(1, 16, 16), (1, 1024, 2560), (3, 144, 128), (8, 256, 4096), (17, 400, 272),
          (33, 128, 1040), (64, 640, 640), (65, 272, 528), (100, 1552, 896), (128, 128, 256),
          (129, 256, 128), (200, 384, 1552), (257, 512, 784), (300, 1040, 400), (513, 272, 1296)]


@pytest.mark.parametrize("dx", [False, True])
@pytest.mark.parametrize("T,out_d,in_d", SHAPES)
def test_product(L, T, out_d, in_d, dx):
    rng = np.random.default_rng(T * 1009 + out_d * 31 + in_d + dx)
    c, s = _weight(rng, out_d, in_d)
    X = _acts(rng, T, out_d if dx else in_d)
    Y = _run(L, X.cuda(), torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), out_d, in_d, dx)
    torch.cuda.synchronize()
    ref, mag = S.block_product(X.float().numpy(), c, s, dx)
    _check(Y, ref, mag)
    assert L.lora_device_error() == 0


@pytest.mark.parametrize("T,K,N", [(1, 256, 160), (40, 400, 272), (300, 256, 512)])
def test_nonfinite_rows_stay_in_their_rows(L, T, K, N):
    rng = np.random.default_rng(T)
    c, s = _weight(rng, N, K)
    cd, sd = torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda()
    X = _acts(rng, T, K)
    clean = _run(L, X.cuda(), cd, sd, N, K, False)
    bad = X.clone()
    rows = sorted({0, T // 2, T - 1})
    for r, v in zip(rows, [float("nan"), float("inf"), float("-inf")]):
        bad[r, (r * 37 + 5) % K] = v
    Y = _run(L, bad.cuda(), cd, sd, N, K, False)
    torch.cuda.synchronize()
    hit = torch.zeros(T, dtype=torch.bool, device="cuda")
    hit[rows] = True
    assert torch.isnan(Y[hit].float()).all()
    assert torch.equal(Y[~hit], clean[~hit])


def test_zero_rows_zero_weight_and_extreme_scales(L):
    T, N, K = 20, 144, 272
    rng = np.random.default_rng(5)
    c, s = _weight(rng, N, K)
    X = _acts(rng, T, K)
    X[3] = 0.0
    X[4] *= 1e30                 # block maxima near the top and the bottom of the range
    X[5] *= 1e-30
    cd, sd = torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda()
    Y = _run(L, X.cuda(), cd, sd, N, K, False)
    Z = _run(L, X.cuda(), torch.zeros_like(cd), sd, N, K, False)
    torch.cuda.synchronize()
    ref, mag = S.block_product(X.float().numpy(), c, s, False)
    y = Y.float().cpu().numpy().astype(np.float64)
    assert np.all(y[3] == 0.0)
    assert np.all(np.abs(y - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -12 * mag)
    assert torch.equal(Z, torch.zeros_like(Z))


@pytest.mark.parametrize("T,dx", [(1, False), (40, True), (300, False), (1000, True)])
def test_reruns_and_streams_bitwise_equal_and_nothing_past_the_output(L, T, dx):
    out_d, in_d = 528, 1040
    rng = np.random.default_rng(9)
    c, s = _weight(rng, out_d, in_d)
    cd, sd = torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda()
    X = _acts(rng, T, out_d if dx else in_d).cuda()
    N = in_d if dx else out_d
    guard = torch.full((T + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    first = _run(L, X, cd, sd, out_d, in_d, dx)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    _run(L, X, cd, sd, out_d, in_d, dx, Y=guard[1:T + 1], stream=st)
    torch.cuda.synchronize()
    assert torch.equal(guard[1:T + 1], first)
    assert (guard[0] == 7.0).all() and (guard[T + 1] == 7.0).all()


def test_input_gradient_is_the_forwards(L):
    """<Y(X), dY> is linear in the dequantised X: its central difference along D equals
    <D, dX(dY)> to the two results' bf16 and E4M3 rounding of dY (2^-4 per element, averaged over
    the 400 x 272 terms, measured against the product of the norms)."""
    T, out_d, in_d = 40, 400, 272
    rng = np.random.default_rng(11)
    c, s = _weight(rng, out_d, in_d)
    dY = _bf16(rng.standard_normal((T, out_d)))
    dX = _run(L, dY.cuda(), torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), out_d, in_d, True)
    w = S.dequantize_blocks(c, s, 128, 128)
    X, D = rng.standard_normal((T, in_d)), rng.standard_normal((T, in_d))
    f = lambda x: float(np.sum((x @ w.T) * dY.double().numpy()))   # noqa: E731
    diff = (f(X + 1e-3 * D) - f(X - 1e-3 * D)) / 2e-3
    got = float(np.sum(D * dX.double().cpu().numpy()))
    scale = np.linalg.norm(D @ w.T) * np.linalg.norm(dY.double().numpy())
    assert abs(got - diff) <= 2.0 ** -4 * scale / np.sqrt(T)

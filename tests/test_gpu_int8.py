"""8-bit products against exact integers.

The integers of a row are those of 127 x / amax rounded to the nearest, ties to even:
float64 decides every case (127 x has at most 31 bits, and a quotient of 24-bit
numbers below 128 is on a border or at least 2^-32 away from it), so they are compared
for equality.  Sums are exact; y is the sum as float32, times two scales: 2^-24 each
for the sum, the two products and the two scales, 5 in all, and where rows are scaled
by their root mean square the mean (K / 256 + 10 additions of squares, half of whose
error a root passes on), the root, the quotient and one more: K / 256 + 20 at most.
A bfloat16 y is rounded once more, 2^-8 of itself.
"""

import numpy as np
import pytest

from _gpu_common import log, require_gpu
from distilled_modal_ssm_amd import HMError, Int8Dense
from distilled_modal_ssm_amd import binding as hb

pytestmark = pytest.mark.gpu


def quantized64(x):
    amax = abs(x).max(-1, keepdims=True)
    return np.rint(x * 127 / np.where(amax > 0, amax, 1)), amax[:, 0] / 127


def _rows_of(q, M, K):
    """The rows that blocks hold, up to the next multiple of 64 columns."""
    KB = -(-K // 64)
    q = q.cpu().numpy().reshape(-1, KB, 16, 4, 16)
    turn = np.array([0, 2, 3, 1])[np.arange(16) // 4][:, None] ^ np.arange(4)[None]  # where chunk c of row r is
    q = np.take_along_axis(q, turn[None, None, :, :, None], 3)
    return q.transpose(0, 2, 1, 3, 4).reshape(-1, KB * 64)[:M]


def _quantize(torch, x, rms_eps=None):
    M, K = x.shape
    q = torch.full((hb.hyena_int8_bytes(M, K),), 99, dtype=torch.int8, device="cuda")
    s = torch.empty(M, device="cuda")
    hb.hyena_quantize_rows(M, K, hb.HM_BF16 if x.dtype == torch.bfloat16 else hb.HM_F32, x, x.stride(0),
                           rms_eps is not None, rms_eps or 0.0, q, s)
    if M % 16:  # rows past the last are left as they are
        assert (_rows_of(q, -(-M // 16) * 16, K)[M:] == 99).all()
    return _rows_of(q, M, K), s


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("M,K,pad", [(1, 1, 0), (3, 64, 0), (5, 515, 0), (2, 2048, 8), (300, 100, 3), (1, 20000, 1),
                                     (7, 8191, 0), (1, 131072, 0)])
def test_rows(act, M, K, pad):
    torch = require_gpu()
    log(f"rows {act} {M} {K} {pad}")
    g = torch.Generator().manual_seed(M + K)
    x = (torch.randn(M, K + pad, generator=g) * torch.exp(3 * torch.randn(M, 1, generator=g)))
    x = x.to(torch.bfloat16 if act == "bf16" else torch.float32).cuda()[:, :K]
    ref, scale = quantized64(x.double().cpu().numpy())
    for eps in (None, 1e-6):
        q, s = _quantize(torch, x, eps)
        assert (q[:, :K] == ref).all()
        assert (q[:, K:] == 0).all()
        want = scale
        if eps is not None:
            want = scale / np.sqrt((x.double().cpu().numpy() ** 2).mean(-1) + eps)
        assert (abs(s.cpu().numpy() - want) <= (2 if eps is None else K / 256 + 18) * 2.0 ** -24 * want).all()


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("M,K", [(2, 32771), (3, 16387), (1, 40961), (5, 7), (1030, 1023)])
def test_rows_between_words(act, M, K):
    """Odd rows that begin anywhere, the largest value the last one, and NaN right before and behind them."""
    torch = require_gpu()
    log(f"rows between words {act} {M} {K}")
    g = torch.Generator().manual_seed(M + K)
    x = torch.full((M, K + 2), float("nan"))
    x[:, 1:K + 1] = torch.randn(M, K, generator=g)
    x[:, K] = 9.0
    x = x.to(torch.bfloat16 if act == "bf16" else torch.float32).cuda()[:, 1:K + 1]
    ref, scale = quantized64(x.double().cpu().numpy())
    q, s = _quantize(torch, x)
    assert (q[:, :K] == ref).all() and (q[:, K:] == 0).all()
    assert (abs(s.cpu().numpy() - scale) <= 2 * 2.0 ** -24 * scale).all()


def test_rows_at_borders():
    """Ties, values next to them, the smallest and largest numbers, rows of zeros and rows that are not finite."""
    torch = require_gpu()
    log("borders")
    n = torch.arange(-127, 127, dtype=torch.float32)
    ties = torch.cat([n + 0.5, torch.tensor([127.0])])
    up = torch.nextafter(ties, torch.full_like(ties, 1e9)).clamp(-127, 127)
    down = torch.nextafter(ties, torch.full_like(ties, -1e9))
    down[-1] = 127.0
    third = ties / 3.0
    rows = torch.stack([ties, up, down, third, ties * 2.0 ** -140, ties * 2.0 ** 120, ties * 1e-30, ties * 0.0])
    x = rows.cuda()
    q, s = _quantize(torch, x)
    ref, scale = quantized64(x.double().cpu().numpy())
    assert (q[:, :255] == ref).all()
    assert (abs(s.cpu().numpy() - scale) <= 2.0 ** -24 * scale + 2.0 ** -150).all()
    assert float(s[7]) == 0 and not q[7].any()
    g = torch.Generator().manual_seed(5)
    x = torch.randn(3, 700, generator=g)
    x[0, 3], x[1, 600], x[1, 2] = float("nan"), float("inf"), -float("inf")
    q, s = _quantize(torch, x.cuda(), 1e-6)
    assert torch.isnan(s[:2]).all() and not q[:2].any() and torch.isfinite(s[2])
    y = Int8Dense(torch.randn(40, 700, generator=g).cuda())(x.cuda())
    assert torch.isnan(y[:2]).all() and torch.isfinite(y[2]).all()


SHAPES = [(1, 1, 1), (1, 17, 64), (5, 6144, 2048), (3, 33, 65), (16, 100, 515), (17, 64, 128), (64, 2048, 2048),
          (65, 129, 200), (100, 1001, 1000), (130, 256, 64), (255, 255, 255), (256, 256, 256), (257, 511, 320),
          (513, 770, 2048), (1000, 300, 77), (2, 40, 131072), (1, 70000, 100), (2049, 300, 192)]


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_products(act, M, N, K):
    torch = require_gpu()
    log(f"dense {act} {M} {N} {K}")
    g = torch.Generator().manual_seed(M + 3 * N + K)
    dt = torch.bfloat16 if act == "bf16" else torch.float32
    x = (torch.randn(M, K + 3, generator=g) * torch.exp(torch.randn(M, 1, generator=g))).to(dt).cuda()[:, 2:K + 2]
    w = torch.randn(N, K + 1, generator=g).to(dt).cuda()[:, :K]
    op = Int8Dense(w)
    X, sx = quantized64(x.double().cpu().numpy())
    W, sw = quantized64(w.double().cpu().numpy())
    sums = (torch.from_numpy(X).cuda() @ torch.from_numpy(W).cuda().t()).cpu().numpy()  # exact: below 2^53
    wide = torch.full((M, N + 6), 5.0, dtype=dt, device="cuda")
    for eps, out in ((None, None), (1e-6, wide[:, 3:N + 3])):
        y = op(x, out=out, rms_eps=eps).double().cpu().numpy()
        s = sx if eps is None else sx / np.sqrt((x.double().cpu().numpy() ** 2).mean(-1) + eps)
        ref = sums * s[:, None] * sw
        tol = (5 if eps is None else K / 256 + 20) * 2.0 ** -24 + (2.0 ** -8 if act == "bf16" else 0)
        bad = abs(y - ref) - tol * abs(ref) - 2.0 ** -126
        assert bad.max() <= 0, (np.unravel_index(bad.argmax(), bad.shape), bad.max())
    assert (wide[:, :3] == 5).all() and (wide[:, N + 3:] == 5).all()


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("M,N", [(70, 90), (1100, 3001), (2100, 6210)])  # tiles of 64 x 64, 128 x 128 and larger
def test_products_in_tiles(act, M, N):
    """Numbers of stages of 64 inputs around every turn of the loop, and the long K of the largest tiles."""
    torch = require_gpu()
    dt = torch.bfloat16 if act == "bf16" else torch.float32
    tol = 5 * 2.0 ** -24 + (2.0 ** -8 if act == "bf16" else 0)
    g = torch.Generator(device="cuda").manual_seed(M)
    stages = [*range(1, 19), 64, 65] if M < 1000 else [1, 2, 3, 4, 5, 7, 12, 13, 16, 17, 64, 65]
    for s in stages:
        K = 64 * s - (s * 7) % 64
        log(f"tiles {act} {M} {N} {K}")
        x, w = (torch.randn(r, K, generator=g, device="cuda").to(dt) for r in (M, N))
        y = Int8Dense(w)(x).double()

        def quantized(a):
            a = a.double()
            top = a.abs().amax(-1, keepdim=True)
            return torch.round(a * 127 / top), top[:, 0] / 127

        (X, sx), (W, sw) = quantized(x), quantized(w)
        ref = (X @ W.t()) * sx[:, None] * sw
        bad = (y - ref).abs() - tol * ref.abs()
        assert float(bad.max()) <= 0, (K, int(bad.argmax()) // N, int(bad.argmax()) % N)
        wide = torch.full((M, N + 10), 5.0, dtype=dt, device="cuda")  # rows of even stride, then of whole pieces
        for at, cols in ((3, N), (8, N // 8 * 8)):
            part = Int8Dense(w[:cols])(x, out=wide[:, at:at + cols])
            assert torch.equal(part.double(), y[:, :cols])
            assert (wide[:, :at] == 5).all() and (wide[:, at + cols:] == 5).all()
            wide.fill_(5.0)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("M", [1, 3, 4, 5, 8, 9])
@pytest.mark.parametrize("K", [4, 64, 130, 512, 1000, 2048, 2050])
def test_few_rows_in_one_launch(act, M, K):
    """Up to 8 rows of up to 2048 inputs are brought to 8 bits by the product itself: as the two calls do."""
    torch = require_gpu()
    log(f"few {act} {M} {K}")
    g = torch.Generator(device="cuda").manual_seed(M + K)
    dt = torch.bfloat16 if act == "bf16" else torch.float32
    x = (torch.randn(M, K, generator=g, device="cuda") * torch.exp(torch.randn(M, 1, generator=g, device="cuda"))).to(dt)
    if M > 2:
        x[1] = 0
        x[2, K // 2] = float("inf") if M == 4 else 3.0
    op = Int8Dense(torch.randn(77, K, generator=g, device="cuda").to(dt))
    for eps in (None, 1e-6):
        q = torch.empty(hb.hyena_int8_bytes(M, K), dtype=torch.int8, device="cuda")
        s = torch.empty(M, device="cuda")
        hb.hyena_quantize_rows(M, K, hb.HM_BF16 if act == "bf16" else hb.HM_F32, x, K, eps is not None, eps or 0.0, q, s)
        for ot in (torch.float32, torch.bfloat16):
            want = torch.empty(M, 77, dtype=ot, device="cuda")
            hb.hyena_dense_int8(M, 77, K, q, s, op.weight8, op.weight_scale, hb.HM_BF16 if ot == torch.bfloat16 else hb.HM_F32,
                                want, 77)
            got = op(x, out=torch.empty_like(want), rms_eps=eps)
            # (a row's sum of squares may be added in another order: K / 256 + 18 roundings of the scale)
            tol = 0 if eps is None else (K / 256 + 18) * 2.0 ** -24 + (2.0 ** -7 if ot == torch.bfloat16 else 0)
            a, b = got.double(), want.double()
            assert torch.equal(torch.isnan(a), torch.isnan(b)) and (M < 3 or bool(torch.isnan(a[2]).all()) == (M == 4))
            a, b = torch.nan_to_num(a), torch.nan_to_num(b)
            assert bool(((a - b).abs() <= tol * b.abs()).all())


def test_largest_sums():
    """All products 127^2 of 131072 inputs: 2.11e9, below 2^31."""
    torch = require_gpu()
    K = 131072
    x, w = torch.ones(3, K, device="cuda"), -torch.ones(20, K, device="cuda")
    y = Int8Dense(w)(x)
    assert (abs(y + K) <= 5 * 2.0 ** -24 * K).all()


def test_types_rows_and_refusals():
    torch = require_gpu()
    g = torch.Generator().manual_seed(1)
    w, x = torch.randn(50, 130, generator=g).cuda(), torch.randn(9, 130, generator=g).cuda()
    op = Int8Dense(w)
    y = op(x)
    assert torch.equal(op(x, out=torch.empty(9, 50, dtype=torch.bfloat16, device="cuda")), y.bfloat16())
    assert op(x[:0]).shape == (0, 50)
    assert torch.equal(op(x[4:5]), y[4:5]) and torch.equal(op(x[::2]), y[::2])
    assert torch.equal(Int8Dense(w[:0])(x), y[:, :0])
    for bad in (x[:, :129], x.half(), x.t(), x[0], x[:, None], x.cpu(), x[:1].expand(9, 130)):
        with pytest.raises(ValueError):
            op(bad)
    with pytest.raises(ValueError):
        op(x, out=y[:8])
    with pytest.raises(HMError):
        op(x, rms_eps=-1.0)
    with pytest.raises(ValueError):
        Int8Dense(torch.randn(3, 131073, device="cuda"))


def test_captured_products_replay():
    torch = require_gpu()
    log("graph")
    g = torch.Generator(device="cuda").manual_seed(1)
    op = Int8Dense(torch.randn(500, 300, generator=g, device="cuda"))
    x = torch.randn(40, 300, generator=g, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        op(x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = op(x, rms_eps=1e-6)
    for _ in range(4):
        x.copy_(torch.randn(40, 300, generator=g, device="cuda"))
        graph.replay()
        got = y.clone()
        torch.cuda.synchronize()
        op(torch.randn(90, 300, generator=g, device="cuda"))
        assert torch.equal(got, op(x, rms_eps=1e-6))


SIZES = [0.0, 1.0, 1e-12, 1e-19, 1e-25, 1e-40, 1e18, 1e20, 1e37]


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("eps", [0.0, 1e-37, 1e-6])
@pytest.mark.parametrize("M,K", [(9, 33), (9, 515), (9, 4001), (9, 16385), (9, 40000), (1026, 513)])
def test_root_mean_squares_of_any_size(act, eps, M, K):
    """Rows whose squares leave float32's range at either end, rows of zeros without eps, a large value among small
    ones; in every kernel that brings rows to 8 bits.  A scale formed in float64 is rounded once (a subnormal one to
    2^-150), others as in the module's text."""
    torch = require_gpu()
    log(f"rms {act} {eps} {M} {K}")
    g = torch.Generator().manual_seed(K)
    size = torch.tensor([SIZES[m % 9] for m in range(M)], dtype=torch.float64)
    x = torch.randn(M, K, generator=g).double() * size[:, None]
    x[5, K // 2], x[6, K - 1] = 1.0, 3e38
    x = x.to(torch.bfloat16 if act == "bf16" else torch.float32).cuda()
    x64 = x.double().cpu().numpy()
    ref, scale = quantized64(x64)
    with np.errstate(invalid="ignore"):
        want = np.nan_to_num(scale / np.sqrt((x64 ** 2).mean(-1) + float(np.float32(eps))))
    q, s = _quantize(torch, x, eps)
    assert (q[:, :K] == ref).all()
    tol = (K / 256 + 18) * 2.0 ** -24 * want + 2.0 ** -150
    assert (abs(s.cpu().numpy() - want) <= tol).all(), (s, want)
    op = Int8Dense(torch.randn(50, K, generator=g).cuda())
    for rows in (slice(0, 8), slice(0, M)):  # in one launch where K is short, and in two
        y = op(x[rows], rms_eps=eps, out=torch.empty(len(want[rows]), 50, device="cuda"))
        sums = (torch.from_numpy(ref[rows]) @ torch.from_numpy(_rows_of(op.weight8, 50, K)[:, :K].astype(np.float64)).t()).numpy()
        exact = sums * want[rows, None] * op.weight_scale.double().cpu().numpy()
        bad = abs(y.double().cpu().numpy() - exact) - (K / 256 + 20) * 2.0 ** -24 * abs(exact) - 2.0 ** -126
        assert bad.max() <= 0, np.unravel_index(bad.argmax(), bad.shape)


@pytest.mark.parametrize("M", [1, 5, 8, 20])
def test_outputs_that_take_the_inputs_place(M):
    """x and the outputs in one memory: the same rows, columns of wider rows that meet or not, rows of another width."""
    torch = require_gpu()
    log(f"in place {M}")
    g = torch.Generator(device="cuda").manual_seed(M)
    for K, N, width, at, to in ((512, 512, 512, 0, 0), (300, 9000, 9000, 100, 0), (300, 500, 800, 0, 300),
                                (300, 500, 800, 500, 0), (300, 500, 799, 290, 299)):
        op = Int8Dense(torch.randn(N, K, generator=g, device="cuda"))
        buf = torch.randn(M, width, generator=g, device="cuda")
        want = op(buf[:, at:at + K].clone())
        y = op(buf[:, at:at + K], out=buf[:, to:to + N])
        assert torch.equal(y, want) and y.data_ptr() == buf[:, to:].data_ptr()
    op = Int8Dense(torch.randn(200, 600, generator=g, device="cuda"))  # bfloat16 outputs at the front of float32 rows
    x = torch.randn(M, 600, generator=g, device="cuda")
    want = op(x.clone(), out=torch.empty(M, 200, dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(op(x, out=x.view(torch.bfloat16).view(-1)[:200 * M].view(M, 200)), want)


@pytest.mark.parametrize("M,N,K", [(5, 8192, 2048), (5, 8193, 2048), (4, 16384, 2048), (8, 16384, 1024), (8, 16385, 64),
                                   (1, 32003, 2048), (8, 32003, 512)])
def test_few_rows_of_many_outputs(M, N, K):
    """On both sides of the border between one launch and two, and in the largest of one."""
    torch = require_gpu()
    log(f"many outputs {M} {N} {K}")
    g = torch.Generator(device="cuda").manual_seed(N + K)
    x, w = (torch.randn(r, K, generator=g, device="cuda") for r in (M, N))
    op = Int8Dense(w)
    X, sx = quantized64(x.double().cpu().numpy())
    W, sw = quantized64(w.double().cpu().numpy())
    ref = X @ W.T * sx[:, None] * sw
    assert (abs(op(x).double().cpu().numpy() - ref) <= 5 * 2.0 ** -24 * abs(ref)).all()

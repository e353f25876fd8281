"""The 8-bit head on the GPU (norm and quantisation to codes, the integer
product, sampling from it) against oracle.decode.

Tolerances. Codes are rounded exact quotients and integer sums are exact: both
have to be equal. Scales are fp64 values rounded to fp32 once: half a step,
2^-24, and 2^-48 for the order of the fp64 sum. fp32 outputs of the product are
two fp32 products of one exact sum: equal; bf16 outputs are those, rounded to
the nearest: equal.
"""
import numpy as np
import pytest

import oracle
from oracle import decode
from tests._util import check_parity

pytestmark = pytest.mark.gpu

SCALE_TOL = 2.0 ** -24 + 2.0 ** -48


@pytest.fixture(scope="module")
def fs():
    import torch
    assert torch.cuda.is_available()
    from lm_head_gemm_amd import flashsample
    return flashsample


def _t(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def _vals(rng, shape, bf16, sigma=1.0):
    x = (rng.standard_normal(shape) * sigma).astype(np.float32)
    return decode.bf16_round(x) if bf16 else x


def _check_codes(q, scales, want_q, want_s):
    q, scales = q.cpu().numpy(), scales.cpu().numpy().astype(np.float64)
    assert np.array_equal(q, want_q)
    nan = np.isnan(want_s)
    assert np.array_equal(np.isnan(scales), nan)
    s, w = scales[~nan], want_s[~nan]
    assert np.all(np.abs(s - w) <= np.maximum(w * SCALE_TOL, 2.0 ** -150))


# rows of one piece to the longest, around every change of the thread layout
BF16_D = [8, 64, 504, 512, 520, 2048, 2056, 4096, 4104, 8192, 8200, 16384, 16392, 32768, 32776, 81408]
F32_D = [4, 252, 256, 260, 1024, 1028, 2048, 2052, 4096, 4100, 8192, 8196, 16384, 16388, 40704]


@pytest.mark.parametrize("bf16,D", [(True, d) for d in BF16_D] + [(False, d) for d in F32_D])
def test_quantize(fs, bf16, D):
    import torch
    rng = np.random.default_rng(D)
    for M in (1, 5):
        x = _vals(rng, (M, D), bf16, 0.02)
        q, s = fs.quantize_i8(_t(x, torch.bfloat16 if bf16 else torch.float32))
        _check_codes(q, s, *decode.quantize(x))


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("gain_bf16", [False, True])
@pytest.mark.parametrize("bf16,D", [(True, d) for d in BF16_D] + [(False, d) for d in F32_D])
def test_norm(fs, bf16, D, gain_bf16, residual):
    import torch
    if gain_bf16 and not bf16:
        pytest.skip("fp32 rows take fp32 gains")
    rng = np.random.default_rng(D + 1)
    t = torch.bfloat16 if bf16 else torch.float32
    g = _vals(rng, (D,), gain_bf16, 0.2) + np.float32(1)
    g = decode.bf16_round(g) if gain_bf16 else g
    for M in (1, 6):
        x = _vals(rng, (M, D), bf16)
        r = _vals(rng, (M, D), bf16, 3.0) if residual else None
        want_q, want_s, want_h = decode.rms_norm(x, g, 1e-5, r, bf16)
        got = fs.rms_norm_i8(_t(x, t), _t(g, torch.bfloat16 if gain_bf16 else torch.float32), 1e-5,
                             residual=None if r is None else _t(r, t))
        _check_codes(got[0], got[1], want_q, want_s)
        if residual:
            assert np.array_equal(got[2].float().cpu().numpy(), want_h)
        else:
            assert len(got) == 2


@pytest.mark.parametrize("M", [1, 3, 4, 5, 1000])
def test_norm_many_rows(fs, M):
    import torch
    rng = np.random.default_rng(M)
    for D in (128, 264, 1032):
        x, r = _vals(rng, (M, D), True), _vals(rng, (M, D), True)
        g = _vals(rng, (D,), True)
        want = decode.rms_norm(x, g, 1e-6, r, True)
        q, s, h = fs.rms_norm_i8(_t(x, torch.bfloat16), _t(g, torch.bfloat16), residual=_t(r, torch.bfloat16))
        _check_codes(q, s, want[0], want[1])
        assert np.array_equal(h.float().cpu().numpy(), want[2])


@pytest.mark.parametrize("bf16,D", [(True, d) for d in (2048, 2056, 4096, 4104, 6144, 6152, 8192, 8200)] +
                         [(False, d) for d in (1028, 2048, 2052, 3076, 4096)])
def test_norm_more_rows_than_cus(fs, bf16, D):
    """The layouts for many rows (those for few rows are the ones above)."""
    import torch
    M = 257
    rng = np.random.default_rng(D + 2)
    t = torch.bfloat16 if bf16 else torch.float32
    x, r = _vals(rng, (M, D), bf16), _vals(rng, (M, D), bf16, 2.0)
    g = _vals(rng, (D,), True, 0.2) + np.float32(1)
    for gt in (torch.bfloat16, torch.float32) if bf16 else (torch.float32,):
        gain = decode.bf16_round(g) if gt is torch.bfloat16 else g * np.float32(1.0000123)
        for res in (None, r):
            want = decode.rms_norm(x, gain, 1e-5, res, bf16)
            got = fs.rms_norm_i8(_t(x, t), _t(gain, gt), 1e-5, residual=None if res is None else _t(res, t))
            _check_codes(got[0], got[1], want[0], want[1])
    q, s = fs.quantize_i8(_t(x, t))
    _check_codes(q, s, *decode.quantize(x))


@pytest.mark.parametrize("bf16", [False, True])
def test_rounded_products_with_fp32_gains(fs, bf16):
    """Products that fp32 rounds: the largest one among others that fp32 cannot
    tell from it, and quotients beside the middle between two codes of it."""
    import torch
    rng = np.random.default_rng(77)
    D, M = 1024, 40
    t = torch.bfloat16 if bf16 else torch.float32
    for i in range(M):
        x = np.ones(D, dtype=np.float32)
        g = (rng.random(D) * 0.5).astype(np.float32)
        big = _vals(rng, (1,), bf16, 0.2)[0] % np.float32(0.5) + np.float32(1.25)
        big = decode.bf16_round(np.array([big]))[0] if bf16 else big
        base = np.float32(1.5 + 0.25 * rng.random())
        x[:4] = big
        g[:4] = base
        g[1], g[2] = np.nextafter(base, np.float32(0)), np.nextafter(base, np.float32(9))
        x[3], g[3] = -base if not bf16 else -big, big if not bf16 else base
        a = np.abs(x.astype(np.float64) * g).max()
        k = rng.integers(-126, 126, 600)
        g[100:700] = ((k + 0.5) * a / 127.0).astype(np.float32)
        g[100:300] = np.nextafter(g[100:300], np.float32(9))
        g[300:500] = np.nextafter(g[300:500], np.float32(-9))
        want = decode.rms_norm(x[None], g, 1e-5)
        q, s = fs.rms_norm_i8(_t(x[None], t), _t(g), 1e-5)
        _check_codes(q, s, want[0], want[1])


def test_codes_in_the_middle(fs):
    """Quotients at, and one bit beside, the middle between two codes."""
    import torch
    rows = []
    for top in (1.0, 3.0, 254.0, 127.0, 0.7):
        k = np.arange(-127, 127)
        u = ((k + 0.5) * top / 127.0).astype(np.float32)
        rows.append(np.concatenate([u, np.nextafter(u, np.float32(9e9)), np.nextafter(u, np.float32(-9e9)),
                                    np.array([top, -top], dtype=np.float32), np.zeros(4, np.float32)]))
    x = np.stack(rows)
    assert x.shape[1] % 8 == 0
    for bf16 in (False, True):
        v = decode.bf16_round(x) if bf16 else x
        q, s = fs.quantize_i8(_t(v, torch.bfloat16 if bf16 else torch.float32))
        _check_codes(q, s, *decode.quantize(v))


def test_extreme_and_bad_rows(fs):
    """Zero rows, NaN and infinity, the smallest and the largest values, sums
    and squares past fp32's range: none touches another row."""
    import torch
    D = 256
    rng = np.random.default_rng(0)
    x = _vals(rng, (14, D), True)
    x[0] = 0
    x[1, 7] = np.nan
    x[2, 255] = np.inf
    x[3, 0] = -np.inf
    x[4] *= np.float32(2.0 ** 100)
    x[5] = decode.bf16_round(np.sign(x[5]) * np.float32(3.3e38))
    x[6] *= np.float32(2.0 ** -120)
    x[7] = 0
    x[7, 3] = np.float32(2.0 ** -133)      # the smallest bf16
    x[8] = -0.0
    x[9, :] = 0
    x[9, 5] = 1
    x = decode.bf16_round(x)
    q, s = fs.quantize_i8(_t(x, torch.bfloat16))
    _check_codes(q, s, *decode.quantize(x))
    for g in (np.full(D, 2.0, np.float32), np.full(D, 2.0 ** -30, np.float32), np.zeros(D, np.float32)):
        for gt in (torch.bfloat16, torch.float32):
            for eps in (1e-6, 0.0):
                want_q, want_s, _ = decode.rms_norm(x, g, eps)
                # eps 0 and a zero row: 0 / 0 in the norm's factor is NaN whatever the gain
                q, s = fs.rms_norm_i8(_t(x, torch.bfloat16), _t(g, gt), eps)
                _check_codes(q, s, want_q, want_s)
    # a residual that overflows the type
    r = np.where(np.arange(14)[:, None] == 5, x, np.float32(0))
    r = np.where(np.isfinite(r), r, np.float32(0))
    want_q, want_s, want_h = decode.rms_norm(x, np.ones(D, np.float32), 1e-6, r, True)
    q, s, h = fs.rms_norm_i8(_t(x, torch.bfloat16), _t(np.ones(D, np.float32)), residual=_t(r, torch.bfloat16))
    assert np.isnan(want_s[5])
    _check_codes(q, s, want_q, want_s)
    assert np.array_equal(h.float().cpu().numpy(), want_h, equal_nan=True)


def test_norm_in_place_and_strided(fs):
    import torch
    rng = np.random.default_rng(5)
    M, D = 33, 264
    x, r, g = _vals(rng, (M, D), True), _vals(rng, (M, D), True), _vals(rng, (D,), True)
    want_q, want_s, want_h = decode.rms_norm(x, g, 1e-6, r, True)
    gd = _t(g, torch.bfloat16)
    for into in ("x", "residual"):
        xd, rd = _t(x, torch.bfloat16), _t(r, torch.bfloat16)
        h = fs.rms_norm_i8(xd, gd, residual=rd, sum_out=xd if into == "x" else rd)[2]
        assert h is (xd if into == "x" else rd)
        assert np.array_equal(h.float().cpu().numpy(), want_h)
        other, same = (rd, r) if into == "x" else (xd, x)
        assert np.array_equal(other.float().cpu().numpy(), same)
    wide = torch.full((M, 3 * 272), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + D] = _t(x, torch.bfloat16)
    wide[:, 280:280 + D] = _t(r, torch.bfloat16)
    codes = torch.full((M, 304), 99, dtype=torch.int8, device="cuda")
    q, s, h = fs.rms_norm_i8(wide[:, 8:8 + D], gd, residual=wide[:, 280:280 + D], sum_out=wide[:, 552:552 + D],
                             q=codes[:, 16:16 + D])
    _check_codes(q, s, want_q, want_s)
    assert np.array_equal(h.float().cpu().numpy(), want_h)
    assert int((codes[:, :16] != 99).sum()) == 0 and int((codes[:, 16 + D:] != 99).sum()) == 0
    assert bool((wide[:, :8] == 7).all()) and bool((wide[:, 552 + D:] == 7).all())


# ------------------------------------------------------------------ product
def _codes(rng, shape, full=False):
    if full:
        return rng.integers(-128, 128, shape).astype(np.int8)
    return np.clip(np.rint(rng.standard_normal(shape) * 30), -127, 127).astype(np.int8)


def _product_case(rng, M, N, K, full=False):
    q, w = _codes(rng, (M, K), full), _codes(rng, (N, K), full)
    qs = (0.01 + 0.03 * rng.random(M)).astype(np.float32)
    ws = (1e-4 + 1e-3 * rng.random(N)).astype(np.float32)
    return q, qs, w, ws


def _check_product(fs, q, qs, w, ws, **kw):
    import torch
    want = decode.product(q, qs, w, ws)
    d = [_t(a) for a in (q, qs, w, ws)]
    got = fs.matmul_i8(*d, out_dtype=torch.float32, **kw)
    assert np.array_equal(got.cpu().numpy(), want)
    got = fs.matmul_i8(*d, **kw)
    assert got.dtype == torch.bfloat16 and np.array_equal(got.float().cpu().numpy(), decode.bf16_round(want))


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 31, 33, 64, 65, 127, 128, 129, 200, 256, 257, 300, 513])
@pytest.mark.parametrize("N,K", [(1, 16), (17, 64), (255, 272), (1000, 2320), (4097, 512)])
def test_product(fs, M, N, K):
    _check_product(fs, *_product_case(np.random.default_rng(M * 7 + N + K), M, N, K))


@pytest.mark.parametrize("K", [16, 32, 48, 112, 128, 144, 240, 256, 496, 528, 1040, 4096, 8208])
@pytest.mark.parametrize("M", [1, 40, 150, 600])
def test_product_k(fs, M, K):
    """Every remainder of the K loops."""
    _check_product(fs, *_product_case(np.random.default_rng(M + K), M, 700, K, full=True))


@pytest.mark.parametrize("K", [16, 144, 400, 768, 1040, 1360])
@pytest.mark.parametrize("M,N", [(3, 16400), (20, 33001), (33, 33001), (64, 74001), (100, 50001), (129, 25001),
                                 (300, 9001), (300, 25001), (500, 25001), (850, 12001)])
def test_product_many_channels(fs, M, N, K):
    """Enough channels for each of the larger tiles, the last one ragged."""
    _check_product(fs, *_product_case(np.random.default_rng(M + N + K), M, N, K))


def test_product_large_sums(fs):
    """Sums past 2^24 (rounded once, to fp32) and the largest there are."""
    rng = np.random.default_rng(1)
    K = 131056
    q, w = np.full((3, K), -128, np.int8), np.full((35, K), -128, np.int8)
    w[1] = 127
    w[2] = _codes(rng, (K,), True)
    q[1] = _codes(rng, (K,), True)
    one = np.ones(35, np.float32)
    _check_product(fs, q, one[:3], w, one)
    _check_product(fs, np.repeat(q, 100, 0), np.repeat(one[:3], 100), w, one)


def test_product_strided_and_unaligned_output(fs):
    import torch
    rng = np.random.default_rng(2)
    for M, N, K in ((5, 300, 96), (70, 1001, 320), (300, 515, 256)):
        q, qs, w, ws = _product_case(rng, M, N, K)
        want = decode.product(q, qs, w, ws)
        qd = torch.zeros((M, K + 48), dtype=torch.int8, device="cuda")
        wd = torch.zeros((N, 2 * K + 16), dtype=torch.int8, device="cuda")
        qd[:, 16:16 + K] = _t(q)
        wd[:, K:2 * K] = _t(w)
        for dtype in (torch.float32, torch.bfloat16):
            for off in (0, 1, 3):
                out = torch.full((M, N + 5 + off), 5.0, dtype=dtype, device="cuda")
                fs.matmul_i8(qd[:, 16:16 + K], _t(qs), wd[:, K:2 * K], _t(ws), out=out[:, off:off + N])
                got = out.float().cpu().numpy()
                assert np.array_equal(got[:, off:off + N], want if dtype == torch.float32 else decode.bf16_round(want))
                assert np.all(got[:, :off] == 5) and np.all(got[:, off + N:] == 5)


def test_product_scales_that_are_not_numbers(fs):
    rng = np.random.default_rng(3)
    q, qs, w, ws = _product_case(rng, 20, 70, 64)
    qs[3], qs[5], ws[11], ws[12] = np.nan, 0, np.inf, 0
    import torch
    with np.errstate(invalid="ignore", over="ignore"):
        want = decode.product(q, qs, w, ws)
    got = fs.matmul_i8(*[_t(a) for a in (q, qs, w, ws)], out_dtype=torch.float32).cpu().numpy()
    assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("M,N,K", [(2, 2**20 + 17, 64), (5000, 300, 128), (70000, 33, 32)])
def test_product_long_sides(fs, M, N, K):
    _check_product(fs, *_product_case(np.random.default_rng(4), M, N, K))


def test_product_past_32_bit_offsets(fs):
    """W and the output longer than 2^32 bytes: rows at the end."""
    import torch
    K, N = 8192, 2**19 + 300
    w = torch.zeros((N, K), dtype=torch.int8, device="cuda")
    rng = np.random.default_rng(5)
    tail = _codes(rng, (260, K))
    w[-260:] = _t(tail)
    for M in (4, 300):
        q, qs, _, _ = _product_case(rng, M, 1, K)
        ws = np.full(N, 1e-3, np.float32)
        got = fs.matmul_i8(_t(q), _t(qs), w, _t(ws), out_dtype=torch.float32)
        assert np.array_equal(got[:, -260:].cpu().numpy(), decode.product(q, qs, tail, ws[-260:]))
        assert int((got[:, :-260] != 0).sum()) == 0


# ----------------------------------------------------------------- sampling
@pytest.mark.parametrize("B,D,V", [(1, 64, 1000), (7, 272, 2053), (70, 512, 4099), (300, 128, 1111)])
def test_sample_i8(fs, B, D, V):
    """Tokens from the 8-bit head against the sampler's oracle on its logits
    (an identity head hands the oracle exactly those)."""
    rng = np.random.default_rng(B + V)
    q, qs, w, ws = _product_case(rng, B, V, D)
    logits = decode.product(q, qs, w, ws)
    d = [_t(a) for a in (q, qs, w, ws)]
    eye = np.eye(V, dtype=np.float32)
    for T, seed, step in ((1.0, 3, 0), (0.6, 2**40 + 1, 2**33)):
        tok = fs.sample_i8(*d, T, seed, step).cpu().numpy()
        check_parity(logits, eye, T, seed, step, np.arange(B), tok)
    assert np.array_equal(fs.sample_i8(*d, 0.0, 0, 0).cpu().numpy(), logits.argmax(1))


def test_sample_i8_bad_row(fs):
    rng = np.random.default_rng(9)
    q, qs, w, ws = _product_case(rng, 6, 500, 64)
    qs[2] = np.nan
    tok = fs.sample_i8(*[_t(a) for a in (q, qs, w, ws)], 1.0, 1, 2).cpu().numpy()
    assert tok[2] == -1 and (tok[[0, 1, 3, 4, 5]] >= 0).all()


def test_norm_product_sample(fs):
    """The decode step: residual and norm to codes, a quantised head, tokens."""
    import torch
    rng = np.random.default_rng(11)
    B, D, V = 9, 512, 3001
    x, r, g = _vals(rng, (B, D), True), _vals(rng, (B, D), True), _vals(rng, (D,), True) + np.float32(1)
    g = decode.bf16_round(g)
    W = _vals(rng, (V, D), True, 0.05)
    bt = torch.bfloat16
    wq, wsc = fs.quantize_i8(_t(W, bt))
    q, s, h = fs.rms_norm_i8(_t(x, bt), _t(g, bt), residual=_t(r, bt))
    oq, osc, oh = decode.rms_norm(x, g, 1e-6, r, True)
    ow, ows = decode.quantize(W)
    assert np.array_equal(wq.cpu().numpy(), ow) and np.array_equal(q.cpu().numpy(), oq)
    logits = decode.product(oq, s.cpu().numpy(), ow, wsc.cpu().numpy())
    tok = fs.sample_i8(q, s, wq, wsc, 0.8, 5, 6).cpu().numpy()
    check_parity(logits, np.eye(V, dtype=np.float32), 0.8, 5, 6, np.arange(B), tok)
    # and the codes stand for the norm: each side off by at most half a code
    y = oh.astype(np.float64) / np.sqrt((oh.astype(np.float64) ** 2).mean(1, keepdims=True) + 1e-6) * g
    exact = y @ W.astype(np.float64).T
    bound = (0.5 * osc[:, None]) * np.abs(W).sum(1)[None] + np.abs(y).sum(1)[:, None] * (0.5 * ows)[None] \
        + D * 0.25 * osc[:, None] * ows[None]
    assert np.all(np.abs(logits - exact) <= bound * (1 + 1e-5))


# ------------------------------------------------- streams, graphs, devices
def test_other_stream_and_graph(fs):
    import torch
    rng = np.random.default_rng(12)
    M, N, K = 20, 3000, 512
    x, r, g = _vals(rng, (M, K), True), _vals(rng, (M, K), True), _vals(rng, (K,), True)
    w = _codes(rng, (N, K))
    ws = (1e-3 * rng.random(N)).astype(np.float32)
    bt = torch.bfloat16
    xd, rd, gd, wd, wsd = _t(x, bt), _t(r, bt), _t(g, bt), _t(w), _t(ws)

    def step(**kw):
        q, s, h = fs.rms_norm_i8(xd, gd, residual=rd, **kw)
        out = fs.matmul_i8(q, s, wd, wsd, out_dtype=torch.float32, **kw)
        tok = fs.sample_i8(q, s, wd, wsd, 0.9, 1, 2, **kw)
        return h, out, tok

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for i in range(4):
        xd.copy_(_t(_vals(np.random.default_rng(100 + i), (M, K), True), bt))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured]
        assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_stream_of_nothing_else(fs):
    """A stream that is not of the tensors' device is refused."""
    import torch
    q = torch.zeros((2, 64), dtype=torch.bfloat16, device="cuda")

    class Elsewhere:
        device = torch.device("cuda", 7)
    with pytest.raises(ValueError, match="stream"):
        fs.quantize_i8(q, stream=Elsewhere())


def test_refusals_reach_python(fs):
    import torch
    q = torch.zeros((2, 24), dtype=torch.int8, device="cuda")
    s = torch.ones(2, device="cuda")
    with pytest.raises(fs.FlashSampleError, match="FS_ERR_UNSUPPORTED"):
        fs.matmul_i8(q, s, q, s)
    x = torch.zeros((2, 12), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(fs.FlashSampleError, match="FS_ERR_UNSUPPORTED"):
        fs.quantize_i8(x)
    with pytest.raises(fs.FlashSampleError, match="FS_ERR_WORKSPACE_TOO_SMALL"):
        c = torch.zeros((2, 32), dtype=torch.int8, device="cuda")
        fs.sample_i8(c, s, c, s, 1.0, 0, 0, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))

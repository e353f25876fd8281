"""Beam search on the GPU (selection, reordering) against oracle.decode.

Tolerances. A row's logarithm of the sum is off by at most 1e-5: each of the
terms that matter (within 30 of the maximum) carries two fp32 roundings of its
exponent (30 * 2^-23) and two of the exponential (2^-22), and a thread adds up
to 64 of them in fp32 (64 * 2^-24): below 9e-6 in all. Scores are rounded to
fp32 once more (2^-24). Places have to be equal wherever the oracle's best
n + 1 scores lie further apart than 2e-5 (equal ones within a row, and of equal
rows, are decided by their place and have to be equal too)."""
import numpy as np
import pytest

from oracle import decode

pytestmark = pytest.mark.gpu
LSE_TOL = 1e-5


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


def _run(fs, logits, scores, n, bf16, finished=None, pad=0, **kw):
    import torch
    l = _t(logits.astype(np.float32), torch.bfloat16 if bf16 else torch.float32)
    return fs.beam_select(l, _t(scores.astype(np.float32)), n,
                          finished=None if finished is None else _t(finished), pad_token=pad, **kw)


def _check(fs, logits, scores, n, bf16=False, finished=None, pad=0, least=0.8, got=None, **kw):
    got = _run(fs, logits, scores, n, bf16, finished, pad, **kw) if got is None else got
    s, p, t = (a.cpu().numpy() for a in got)
    scores = scores.astype(np.float32)
    logits = decode.bf16_round(logits) if bf16 else logits.astype(np.float32)
    ws, wp, wt, margin = decode.beam_select(logits, scores, n, finished, pad)
    none = ws == -np.inf
    assert np.array_equal(s == -np.inf, none)
    assert np.all(p[none] == -1) and np.all(t[none] == -1)
    assert np.all(np.abs(s[~none] - ws[~none]) <= LSE_TOL + np.abs(ws[~none]) * 2.0 ** -24)
    firm = margin > 2 * LSE_TOL
    assert np.array_equal(p[firm], wp[firm]) and np.array_equal(t[firm], wt[firm])
    assert firm.mean() >= least
    return s, p, t


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("B,K,V,n", [
    (1, 1, 1, 1), (1, 1, 5, 8), (2, 3, 7, 4), (1, 4, 100, 8), (3, 5, 2047, 5), (2, 4, 2048, 8), (2, 4, 2049, 16),
    (5, 2, 5003, 3), (1, 12, 16385, 24), (1, 4, 50257, 8), (4, 8, 33000, 16), (1, 64, 3001, 64), (2, 33, 1000, 33),
    (40, 4, 4099, 8), (1, 2, 151936, 64), (300, 2, 300, 4), (64, 5, 9001, 10),
    (30, 8, 33003, 16), (64, 8, 40001, 8), (1, 64, 20011, 64)])
def test_selection(fs, bf16, B, K, V, n):
    rng = np.random.default_rng(B * 100 + K * 10 + V + n)
    logits = rng.standard_normal((B * K, V)) * 2
    scores = -5 - 3 * rng.random((B, K))
    # groups of many candidates have close neighbours now and then
    _check(fs, logits, scores, n, bf16, least=0.5 if n * B < 20 else 0.8)


@pytest.mark.parametrize("bf16", [False, True])
def test_masks_and_states_of_beams(fs, bf16):
    rng = np.random.default_rng(1)
    B, K, V, n = 6, 4, 3001, 8
    low = float(np.finfo(np.float32).min) if not bf16 else -3.3895313892515355e38
    logits = rng.standard_normal((B * K, V)) * 2
    logits[rng.random((B * K, V)) < 0.3] = -np.inf
    logits[0:4] = -np.inf                         # group 0: nothing may follow
    logits[4:7] = -np.inf                         # group 1: one beam left, three tokens
    logits[7] = -np.inf
    logits[7, [5, 2999, 17]] = [0.5, 0.25, 1.5]
    logits[8] = low                               # a row of the lowest value only
    logits[9, 100:] = low
    logits[12, 40] = np.nan
    logits[13] = np.nan
    logits[14, 3] = np.inf                        # no continuation
    logits[15, ::2] = np.nan
    scores = -rng.random((B, K))
    scores[4, 1:] = -np.inf                       # one beam in use
    scores[5] = -np.inf                           # none
    scores[3, 2] = np.nan
    finished = np.zeros((B, K), dtype=bool)
    finished[2, 1] = True
    finished[2, 3] = True
    finished[0, 0] = True
    finished[5, 0] = True                         # finished, but not in use
    s, p, t = _check(fs, logits, scores, n, bf16, finished, pad=2999, least=0.5)
    assert p[0].tolist() == [0] + [-1] * 7 and t[0, 0] == 2999 and s[0, 0] == np.float32(scores[0, 0])
    assert sorted(t[1, :3].tolist()) == [5, 17, 2999] and p[1, 3] == -1
    assert (p[5] == -1).all() and set(p[4].tolist()) == {0}
    assert not np.isin(2, p[3])
    # finished as bytes
    again = _run(fs, logits, scores, n, bf16, finished.astype(np.uint8) * 7, 2999)
    assert all(np.array_equal(a, b.cpu().numpy()) for a, b in zip((s, p, t), again))


@pytest.mark.parametrize("n", [1, 4, 16, 64])
def test_ties(fs, n):
    """Equal logits go to the lowest place: whole rows of one value, rows of a
    few values, equal rows at different alignments."""
    B, K = 2, 3
    for V in (500, 2048, 20001, 40007):
        for levels in (1, 2, 3):
            rng = np.random.default_rng(V + levels)
            row = rng.integers(0, levels, V).astype(np.float64)
            logits = np.tile(row, (B * K, 1))
            scores = np.full((B, K), -1.5)
            scores[1, 0] = -9.0
            _check(fs, logits, scores, n, least=1.0)
            _check(fs, logits, scores, n, True, least=1.0)


def test_equal_rows_give_equal_scores(fs):
    """Rows that start at every alignment hold the same random values: the
    first n are beam 0's, and each score appears once per beam."""
    rng = np.random.default_rng(3)
    for V in (1001, 30011):
        row = rng.standard_normal(V) * 2
        K, n = 8, 24
        s, p, t = _check(fs, np.tile(row, (K, 1)), np.zeros((1, K)), n, least=1.0)
        assert p[0].tolist() == list(range(8)) * 3
        assert all(len(set(t[0, 8 * i: 8 * i + 8].tolist())) == 1 for i in range(3))


def test_zero_signs_are_equal(fs):
    logits = np.full((1, 3000), -5.0)
    logits[0, 10:2000:2], logits[0, 11:2001:2] = -0.0, 0.0
    s, p, t = _check(fs, logits, np.zeros((1, 1)), 6, least=1.0)
    assert t[0].tolist() == [10, 11, 12, 13, 14, 15]


def test_sorted_rows(fs):
    """Increasing, decreasing, and all large values side by side."""
    for V in (3000, 70001):
        up = np.linspace(-8, 8, V)
        block = np.full(V, -3.0) + np.linspace(0, 1e-3, V)
        block[V // 2: V // 2 + 64] = 5 + np.linspace(0, 1, 64)
        for row in (up, up[::-1], block):
            for n in (4, 32, 64):
                _check(fs, row[None], np.zeros((1, 1)), n, least=0.0)
                s, p, t = (a.cpu().numpy() for a in _run(fs, row[None], np.zeros((1, 1)), n, False))
                want = np.lexsort((np.arange(V), -row.astype(np.float32)))[:n]
                assert np.array_equal(t[0], want)   # order within a row is exact whatever the gaps


def test_strided_logits_and_given_outputs(fs):
    import torch
    rng = np.random.default_rng(4)
    B, K, V, n = 2, 3, 2500, 6
    logits = (rng.standard_normal((B * K, V)) * 2).astype(np.float32)
    scores = (-rng.random((B, K))).astype(np.float32)
    for dtype in (torch.float32, torch.bfloat16):
        want = fs.beam_select(_t(logits, dtype), _t(scores), n)
        for off in (1, 2, 7):
            wide = torch.full((B * K, V + 37), 1e9, dtype=dtype, device="cuda")
            wide[:, off:off + V] = _t(logits, dtype)
            out = (torch.zeros((B, n), device="cuda"), torch.zeros((B, n), dtype=torch.int32, device="cuda"),
                   torch.zeros((B, n), dtype=torch.int32, device="cuda"))
            work = torch.empty(fs.beam_select_workspace_bytes(B, K, V, n, dtype), dtype=torch.uint8, device="cuda")
            got = fs.beam_select(wide[:, off:off + V], _t(scores), n, out=out, workspace=work)
            assert all(a is b for a, b in zip(got, out))
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(fs.FlashSampleError, match="FS_ERR_WORKSPACE_TOO_SMALL"):
        fs.beam_select(_t(logits), _t(scores), n, workspace=work[:64])
    with pytest.raises(ValueError, match="workspace"):
        fs.beam_select(_t(logits), _t(scores), n, workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda")[::2])
    with pytest.raises(fs.FlashSampleError, match="FS_ERR_INVALID_ARGUMENT"):
        fs.beam_select(_t(logits), _t(scores), 65)
    with pytest.raises(fs.FlashSampleError, match="FS_ERR_INVALID_ARGUMENT"):
        fs.beam_select(_t(logits), _t(scores), n, pad_token=V)


def test_scores_in_place_in_a_replayed_graph(fs):
    """Scores written over the ones read, as a loop captured once keeps them;
    two graphs with a workspace of their own, replayed in turn."""
    import torch
    rng = np.random.default_rng(12)
    B, K, V = 3, 8, 9001
    logits = [_t((rng.standard_normal((B * K, V)) * 2).astype(np.float32)) for _ in range(2)]
    start = _t((-rng.random((B, K))).astype(np.float32))
    scores = [start.clone() for _ in range(2)]
    outs = [[s, torch.zeros((B, K), dtype=torch.int32, device="cuda"),
             torch.zeros((B, K), dtype=torch.int32, device="cuda")] for s in scores]
    for l, o in zip(logits, outs):
        fs.beam_select(l, o[0], out=o)            # eager, in place
    want = [fs.beam_select(l, start) for l in logits]
    assert all(torch.equal(a, b) for o, w in zip(outs, want) for a, b in zip(o, w))
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, l, o in zip(graphs, logits, outs):
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            fs.beam_select(l, o[0], out=o)
    for s in scores:
        s.copy_(start)
    state = [start, start]
    for step in range(4):
        for i, g in enumerate(graphs):
            g.replay()
            want = fs.beam_select(logits[i], state[i])
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs[i], want))
            state[i] = want[0]


def test_rows_past_32_bit_offsets(fs):
    import torch
    V, K = 2**20 + 3, 2
    B = 520                                        # over 2^32 bytes of fp32 logits
    logits = torch.zeros((B * K, V), device="cuda")
    rng = np.random.default_rng(6)
    tail = (rng.standard_normal((2 * K, V)) * 2).astype(np.float32)
    logits[-2 * K:] = _t(tail)
    scores = np.zeros((B, K), dtype=np.float32)
    got = fs.beam_select(logits, _t(scores), 5)
    _check(fs, tail, scores[:2], 5, got=[a[-2:] for a in got], least=0.5)
    # all scores of the other groups are equal: in order of (beam, token)
    assert bool((got[2][:-2] == torch.arange(5, dtype=torch.int32, device="cuda")).all()) and not got[1][:-2].any()


# --------------------------------------------------------------- reordering
def _state(rng, shape, dtype):
    import torch
    if dtype == "i8":
        return torch.from_numpy(rng.integers(-128, 128, shape).astype(np.int8)).cuda()
    t = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda()
    return t.to({"bf16": torch.bfloat16, "f32": torch.float32}[dtype])


def _np(t):
    import torch
    return (t.view(torch.int16) if t.dtype == torch.bfloat16 else t).cpu().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "f32", "i8"])
@pytest.mark.parametrize("B,K", [(1, 1), (1, 2), (2, 3), (3, 4), (2, 5), (1, 8), (2, 9), (1, 16), (2, 17), (1, 40),
                                 (1, 64)])
def test_reordering(fs, dtype, B, K):
    rng = np.random.default_rng(B * 100 + K)
    parents = rng.integers(0, K, (B, K)).astype(np.int32)
    parents[0, 0] = -1
    if K > 2:
        parents[B - 1, 2] = K
    for heads, T, length, d in ((2, 9, 7, 64), (1, 5, 5, 20), (3, 4, 1, 3), (2, 300, 290, 8)):
        state = _state(rng, (3, B * K, heads, T, d), dtype)
        want = _np(state).copy()
        want[:, :, :, :length] = decode.beam_reorder(want[:, :, :, :length], parents, 1)
        other = _state(rng, state.shape, dtype)
        want_other = _np(other).copy()
        moved = decode.beam_reorder(_np(state)[:, :, :, :length], parents, 1)
        for b in range(B):
            for i in range(K):
                if 0 <= parents[b, i] < K:
                    want_other[:, b * K + i, :, :length] = moved[:, b * K + i]
        got = fs.beam_reorder(state[:, :, :, :length], _t(parents), dim=1, out=other[:, :, :, :length])
        assert got.data_ptr() == other.data_ptr()
        assert np.array_equal(_np(other), want_other)
        compact = _state(rng, moved.shape, dtype)      # an output of other strides
        want_compact = _np(compact).copy()
        fs.beam_reorder(state[:, :, :, :length], _t(parents), dim=1, out=compact)
        for b in range(B):
            for i in range(K):
                if 0 <= parents[b, i] < K:
                    want_compact[:, b * K + i] = moved[:, b * K + i]
        assert np.array_equal(_np(compact), want_compact)
        fs.beam_reorder(state[:, :, :, :length], _t(parents), dim=1)
        assert np.array_equal(_np(state), want)


def test_reordering_of_a_list(fs):
    """Keys and values of many layers, as tensors of their own and as views
    that interleave in one buffer."""
    import torch
    rng = np.random.default_rng(7)
    parents = np.array([[1, 0, 1], [2, 2, 0]], dtype=np.int32)
    states = [_state(rng, (6, 2, 11, 16), "bf16") for _ in range(192)]
    want = [decode.beam_reorder(_np(t), parents, 0) for t in states]
    assert fs.beam_reorder(states, _t(parents)) is states
    assert all(np.array_equal(_np(t), w) for t, w in zip(states, want))
    with pytest.raises(ValueError, match="192"):
        fs.beam_reorder(states + states[:1], _t(parents))
    whole = _state(rng, (6, 5, 2, 3, 8), "f32")            # rows, layers, keys/values, ...
    want = decode.beam_reorder(_np(whole), parents, 0)
    fs.beam_reorder([whole[:, l, k] for l in range(5) for k in range(2)], _t(parents))
    assert np.array_equal(_np(whole), want)
    with pytest.raises(fs.FlashSampleError, match="FS_ERR_INVALID_ARGUMENT"):
        fs.beam_reorder([whole[:, 0], whole[:, 0]], _t(parents))
    out = [torch.empty_like(t) for t in states[:3]]
    with pytest.raises(fs.FlashSampleError, match="FS_ERR_INVALID_ARGUMENT"):
        fs.beam_reorder(states[:3], _t(parents), out=[out[0], out[1], out[0]])
    with pytest.raises(fs.FlashSampleError, match="FS_ERR_INVALID_ARGUMENT"):
        fs.beam_reorder(states[:2], _t(parents), out=[out[0], states[0]])


def test_reordering_nothing_and_one(fs):
    import torch
    parents = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    empty = torch.zeros((2, 3, 0, 4), device="cuda")
    assert fs.beam_reorder(empty, parents) is empty
    one = torch.tensor([3.0, 4.0], device="cuda")
    fs.beam_reorder(one, parents)
    assert one.tolist() == [3.0, 3.0]
    same = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    fs.beam_reorder(one, same)
    assert one.tolist() == [3.0, 3.0]
    two = torch.zeros(2, device="cuda")
    assert fs.beam_reorder(one, same, out=two) is two and two.tolist() == [3.0, 3.0]
    assert fs.beam_reorder(one, same, out=one) is one


def test_reordering_past_32_bit_offsets(fs):
    import torch
    cache = torch.zeros((4, 1 << 30), dtype=torch.int32, device="cuda")   # 16 GiB, rows of 4 GiB
    for i in range(4):
        cache[i, -5:] = i + 1
        cache[i, :5] = 10 * i
    parents = torch.tensor([[3, 1, 0, 0]], dtype=torch.int32, device="cuda")
    fs.beam_reorder(cache, parents)
    assert cache[:, -1].tolist() == [4, 2, 1, 1] and cache[:, 0].tolist() == [30, 10, 0, 0]
    assert int(cache.count_nonzero()) == 5 * 4 + 5 * 2


# ------------------------------------------------------------ a decode loop
def test_beam_search_over_the_8bit_head(fs):
    """Three steps of beam search: norm, 8-bit head, selection, reordering of
    a cache and of the hidden states, on the default stream, on another one,
    and replayed from a graph; every step against the oracle."""
    import torch
    rng = np.random.default_rng(8)
    B, K, D, V, T = 3, 4, 256, 2003, 8
    bt = torch.bfloat16
    gain = _t(decode.bf16_round((1 + 0.1 * rng.standard_normal(D)).astype(np.float32)), bt)
    W = _t(decode.bf16_round(rng.standard_normal((V, D)).astype(np.float32)), bt)
    wq, ws = fs.quantize_i8(W)
    x = _t(decode.bf16_round(rng.standard_normal((B * K, D)).astype(np.float32)), bt)
    res = _t(decode.bf16_round(rng.standard_normal((B * K, D)).astype(np.float32)), bt)
    cache = _state(rng, (2, B * K, 2, T, 8), "bf16")
    start = torch.full((B, K), -float("inf"), device="cuda")
    start[:, 0] = 0

    def step(scores, finished, res, cache, length, **kw):
        q, s, res = fs.rms_norm_i8(x, gain, residual=res, **kw)
        logits = fs.matmul_i8(q, s, wq, ws, out_dtype=torch.float32, **kw)
        new = fs.beam_select(logits, scores, finished=finished, pad_token=1, **kw)
        fs.beam_reorder(cache[:, :, :, :length], new[1], dim=1, **kw)
        fs.beam_reorder(res, new[1], **kw)
        return logits, res, new

    def loop(check=False, **kw):
        scores, finished, r, c = start, torch.zeros((B, K), dtype=torch.bool, device="cuda"), res, cache.clone()
        tokens = []
        for i in range(3):
            before = (_np(c).copy(), scores.cpu().numpy(), finished.cpu().numpy()) if check else None
            logits, r, (scores, parents, tok) = step(scores, finished, r, c, i + 2, **kw)
            if check:
                old, s0, f0 = before
                p = _check(fs, logits.cpu().numpy(), s0, K, finished=f0, pad=1, got=(scores, parents, tok))[1]
                old[:, :, :, :i + 2] = decode.beam_reorder(old[:, :, :, :i + 2], p, 1)
                assert np.array_equal(_np(c), old)
            finished = tok % 3 == 0
            tokens.append(tok)
        return torch.stack(tokens), scores, c, r

    want = loop(check=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = loop()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = loop()
    for i in range(4):
        x.copy_(_t(decode.bf16_round(np.random.default_rng(50 + i).standard_normal((B * K, D)).astype(np.float32)), bt))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured]
        assert all(torch.equal(a, b) for a, b in zip(got, loop()))


def test_two_calls_at_once(fs):
    """Calls on two streams with workspaces of their own do not touch each
    other, with and without graphs."""
    import torch
    rng = np.random.default_rng(9)
    K, V, n = 4, 60001, 8
    inputs = [(_t((rng.standard_normal((K, V)) * 2).astype(np.float32)), _t(np.zeros((1, K), np.float32)))
              for _ in range(2)]
    want = [fs.beam_select(l, s, n) for l, s in inputs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        got = [fs.beam_select(l, s, n, stream=st) for (l, s), st in zip(inputs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))

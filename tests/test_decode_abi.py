"""Refusals of the 8-bit head's and beam search's entry points: documented
status codes, synchronously, with nothing enqueued (no device is needed)."""
import ctypes
import random

import pytest

OK, INVALID, UNSUPPORTED, WS_SMALL = 0, 1, 2, 3
BF16, F32 = 0, 1
FAKE = 0x1000000   # aligned, never dereferenced: every call below fails validation first
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def fs():
    from lm_head_gemm_amd import flashsample
    return flashsample


def _call(fn, defaults, **kw):
    assert not set(kw) - set(defaults)
    return fn(*{**defaults, **kw}.values(), None)


QUANT = dict(X=FAKE, ldx=64, dtype=BF16, M=4, D=64, codes=FAKE, ldc=64, scales=FAKE)


@pytest.mark.parametrize("kw,status", [
    (dict(X=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
    (dict(M=0), INVALID), (dict(D=0), INVALID), (dict(M=2**31), INVALID), (dict(D=-8), INVALID),
    (dict(ldx=56), INVALID), (dict(ldc=56), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(X=FAKE + 8), UNSUPPORTED),
    (dict(D=60), UNSUPPORTED), (dict(ldx=68), UNSUPPORTED), (dict(codes=FAKE + 4), UNSUPPORTED),
    (dict(ldc=68), UNSUPPORTED), (dict(scales=FAKE + 2), UNSUPPORTED),
    (dict(D=81416, ldx=81416, ldc=81416), UNSUPPORTED),
    (dict(dtype=F32, D=40708, ldx=40708, ldc=40708), UNSUPPORTED),
    (dict(dtype=F32, D=62, ldx=64), UNSUPPORTED), (dict(dtype=F32, ldc=66), UNSUPPORTED),
])
def test_quantize_refusals(fs, kw, status):
    assert _call(fs._lib.fs_quantize_i8, QUANT, **kw) == status


NORM = dict(X=FAKE, ldx=64, residual=FAKE, ldr=64, gain=FAKE, gain_dtype=BF16, dtype=BF16, M=4, D=64, eps=1e-6,
            sum=FAKE, lds=64, codes=FAKE, ldc=64, scales=FAKE)


@pytest.mark.parametrize("kw,status", [
    (dict(X=None), INVALID), (dict(gain=None), INVALID), (dict(residual=None), INVALID), (dict(sum=None), INVALID),
    (dict(eps=-1e-6), INVALID), (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID), (dict(ldr=63), INVALID),
    (dict(lds=32), INVALID), (dict(dtype=F32), UNSUPPORTED), (dict(gain_dtype=5), UNSUPPORTED),
    (dict(gain=FAKE + 4), UNSUPPORTED), (dict(residual=FAKE + 2), UNSUPPORTED), (dict(sum=FAKE + 8), UNSUPPORTED),
    (dict(ldr=68), UNSUPPORTED), (dict(lds=68), UNSUPPORTED), (dict(D=81416), INVALID),
])
def test_norm_refusals(fs, kw, status):
    assert _call(fs._lib.fs_rms_norm_i8, NORM, **kw) == status


PRODUCT = dict(Q=FAKE, ldq=64, qs=FAKE, W=FAKE, ldw=64, ws=FAKE, M=4, N=100, K=64, out=FAKE, ldo=100, dtype=BF16)


@pytest.mark.parametrize("kw,status", [
    (dict(Q=None), INVALID), (dict(qs=None), INVALID), (dict(W=None), INVALID), (dict(ws=None), INVALID),
    (dict(out=None), INVALID), (dict(M=0), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID),
    (dict(N=2**31), INVALID), (dict(M=2**31), INVALID), (dict(N=2**31 - 1, ldo=2**31), INVALID),
    (dict(M=2**31 - 1), INVALID), (dict(ldq=48), INVALID), (dict(ldw=48), INVALID),
    (dict(ldo=99), INVALID), (dict(K=56), UNSUPPORTED), (dict(ldq=72), UNSUPPORTED), (dict(ldw=72), UNSUPPORTED),
    (dict(K=131072, ldq=131072, ldw=131072), UNSUPPORTED), (dict(Q=FAKE + 8), UNSUPPORTED),
    (dict(ldq=2**24), UNSUPPORTED), (dict(ldw=2**24), UNSUPPORTED),
    (dict(W=FAKE + 4), UNSUPPORTED), (dict(qs=FAKE + 1), UNSUPPORTED), (dict(ws=FAKE + 2), UNSUPPORTED),
    (dict(out=FAKE + 1), UNSUPPORTED), (dict(out=FAKE + 2, dtype=F32), UNSUPPORTED), (dict(dtype=9), UNSUPPORTED),
])
def test_product_refusals(fs, kw, status):
    assert _call(fs._lib.fs_matmul_i8, PRODUCT, **kw) == status


SAMPLE = dict(Q=FAKE, ldq=64, qs=FAKE, W=FAKE, ldw=64, ws=FAKE, B=4, V=100, D=64, T=1.0, seed=0, step=0, work=FAKE,
              bytes=1 << 20, out=FAKE)


@pytest.mark.parametrize("kw,status", [
    (dict(work=None), INVALID), (dict(out=None), INVALID), (dict(T=-1.0), INVALID), (dict(T=NAN), INVALID),
    (dict(T=INF), INVALID), (dict(B=65537), INVALID), (dict(Q=None), INVALID), (dict(D=56), UNSUPPORTED),
    (dict(work=FAKE + 8), UNSUPPORTED), (dict(bytes=4 * 104 * 4), WS_SMALL),
])
def test_sample_refusals(fs, kw, status):
    a = {**SAMPLE, **kw}
    b, v, d = a.pop("B"), a.pop("V"), a.pop("D")
    head = [a.pop(k) for k in ("Q", "ldq", "qs", "W", "ldw", "ws")]
    assert fs._lib.fs_sample_i8(*head, b, d, v, *a.values(), None) == status


def test_sample_workspace(fs):
    need = fs.sample_i8_workspace_bytes(4, 64, 100)
    assert need >= 4 * 104 * 4 + 4 * 8 and need % 256 == 0
    for bad in ((0, 64, 100), (4, 0, 100), (4, 64, 0), (65537, 64, 100), (4, 131072, 100), (4, 64, 2**31), (4, 64, 2**31 - 1)):
        assert fs.sample_i8_workspace_bytes(*bad) == 0


SELECT = dict(logits=FAKE, ld=1000, dtype=BF16, scores=FAKE, finished=None, pad=0, B=2, beams=4, V=1000, n=8,
              ws=FAKE, bytes=1 << 20, s=FAKE, p=FAKE, t=FAKE)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), INVALID), (dict(scores=None), INVALID), (dict(ws=None), INVALID), (dict(s=None), INVALID),
    (dict(p=None), INVALID), (dict(t=None), INVALID), (dict(B=0), INVALID), (dict(B=65537), INVALID),
    (dict(beams=0), INVALID), (dict(beams=65), INVALID), (dict(V=0), INVALID), (dict(V=2**31), INVALID),
    (dict(V=2**31 - 1, ld=2**31), INVALID), (dict(n=0), INVALID), (dict(n=65), INVALID), (dict(ld=999), INVALID), (dict(pad=-1), INVALID),
    (dict(pad=1000), INVALID), (dict(dtype=3), UNSUPPORTED), (dict(logits=FAKE + 1), UNSUPPORTED),
    (dict(logits=FAKE + 2, dtype=F32), UNSUPPORTED), (dict(ws=FAKE + 8), UNSUPPORTED),
    (dict(scores=FAKE + 2), UNSUPPORTED), (dict(s=FAKE + 1), UNSUPPORTED), (dict(p=FAKE + 2), UNSUPPORTED),
    (dict(t=FAKE + 3), UNSUPPORTED), (dict(bytes=100), WS_SMALL),
    (dict(), INVALID), (dict(s=FAKE + 28), INVALID), (dict(s=FAKE - 60), INVALID),   # scores overwritten in part
    (dict(n=4, s=FAKE + 4), INVALID),
])
def test_select_refusals(fs, kw, status):
    assert _call(fs._lib.fs_beam_select, SELECT, **kw) == status


def test_select_workspace(fs):
    need = fs.beam_select_workspace_bytes(2, 4, 1000, 8)
    assert need >= 8 * 8 * 8 + 8 * 12 and need % 256 == 0
    for bad in ((0, 4, 1000, 8), (2, 65, 1000, 8), (2, 4, 0, 8), (2, 4, 1000, 0), (2, 4, 1000, 65)):
        assert fs.beam_select_workspace_bytes(*bad) == 0


def _reorder(fs, states=(FAKE,), out=None, layout=(2, 4096, 256, 4, 64, 32), out_layout=None, parents=FAKE, B=2,
             beams=4, n=None):
    def table(ptrs):
        return (ctypes.c_void_p * max(len(ptrs), 1))(*ptrs)
    lay = None if layout is None else ctypes.byref(fs.FsBeamLayout(*layout))
    olay = None if out_layout is None else ctypes.byref(fs.FsBeamLayout(*out_layout))
    return fs._lib.fs_beam_reorder(None if states is None else table(states), None if out is None else table(out),
                                   len(states or ()) if n is None else n, lay, olay, parents, B, beams, None)


@pytest.mark.parametrize("kw", [
    dict(states=None, n=1), dict(layout=None), dict(parents=None), dict(states=(None,)), dict(n=0), dict(n=193),
    dict(B=0), dict(B=65537), dict(beams=0), dict(beams=65), dict(out=(None,)),
    dict(out_layout=(2, 4096, 256, 4, 64, 32)),                                  # a layout without buffers
    dict(layout=(-1, 4096, 256, 4, 64, 32)), dict(layout=(2, -4096, 256, 4, 64, 32)),
    dict(layout=(2, 4096, 256, 4, 64, -1)), dict(layout=(1 << 40, 1 << 40, 256, 4, 64, 32)),
    dict(layout=(2, 4096, 256, 4, 64, 65)),                                      # blocks overlap
    dict(layout=(2, 4096, 200, 4, 64, 32)),                                      # rows overlap
    dict(layout=(2, 1000, 256, 4, 64, 32)),                                      # slabs overlap
    dict(layout=(2, 4096, 0, 4, 64, 32)),                                        # one row for all
    dict(states=(FAKE, FAKE)),
    dict(states=(FAKE, FAKE + 4096 + 16)),                                       # a slab later, half a block off
    dict(states=(FAKE, FAKE + 16)), dict(states=(FAKE + 256 * 3, FAKE)),
    dict(out=(FAKE,)), dict(out=(FAKE + 256,)), dict(out=(FAKE + 31,)),
    dict(out=(FAKE + 64,), out_layout=(2, 8192, 512, 4, 64, 32)),
    dict(out=(FAKE + 65536,), out_layout=(2, 4096, 256, 4, 64, 16)),             # rows of another size
    dict(out=(FAKE + 65536,), out_layout=(1, 4096, 256, 4, 64, 32)),
])
def test_reorder_refusals(fs, kw):
    assert _reorder(fs, **kw) == INVALID


def _bytes(at, layout, rows):
    outer, os, rs, blocks, bs, size = layout
    return [at + o * os + r * rs + b * bs + i for o in range(outer) for r in range(rows) for b in range(blocks)
            for i in range(size)]


def test_reorder_overlaps_against_bytes():
    """Random layouts and places: refused just where two buffers, or one with
    itself, share a byte. Without a device an accepted call ends in a launch
    error; where there is one, the made-up addresses are not offered."""
    from concurrent.futures import ThreadPoolExecutor

    import torch
    if torch.cuda.device_count():
        pytest.skip("accepted calls would be launched")
    from lm_head_gemm_amd import flashsample as fs
    with ThreadPoolExecutor(1) as thread:     # the last launch error is kept per thread
        thread.submit(_overlaps_against_bytes, fs).result()


def _overlaps_against_bytes(fs):
    rng = random.Random(5)
    seen = {True: 0, False: 0}
    for _ in range(6000):
        B, beams = rng.randint(1, 2), rng.randint(1, 3)
        rows = B * beams
        size = rng.randint(1, 4)
        counts = [rng.randint(1, 3), rows, rng.randint(1, 3)]
        strides, span = [0, 0, 0], size
        for i in rng.sample(range(3), 3):         # dimensions in any order of their strides, mostly apart
            strides[i] = max(span - (rng.random() < 0.1), 0) + rng.choice([0, 0, 1, 3, 9])
            span += (counts[i] - 1) * strides[i]
        layout = (counts[0], strides[0], strides[1], counts[2], strides[2], size)
        states = [FAKE + rng.randint(0, 3 * span) for _ in range(rng.randint(1, 2))]
        out = [FAKE + rng.randint(0, 6 * span) for _ in states] if rng.random() < 0.5 else None
        sets = [_bytes(a, layout, rows) for a in (out or states)]
        itself = len(set(sets[0])) < len(sets[0])
        meet = len(sets) > 1 and bool(set(sets[0]) & set(sets[1]))
        if out:
            meet = meet or any(set(w) & set(_bytes(a, layout, rows)) for w in sets for a in states)
        got = _reorder(fs, states, out, layout, B=B, beams=beams)
        if itself or meet:
            assert got == INVALID, (layout, rows, states, out)
        elif got == INVALID:
            # strides that interleave (no order of dimensions in which each step clears the ones below)
            order = sorted((s, c) for s, c in zip(strides, counts) if c > 1)
            below, nested = size, True
            for s, c in order:
                nested = nested and s >= below
                below += (c - 1) * s
            assert not nested, (layout, rows, states, out)
        seen[got == INVALID] += 1
    assert min(seen.values()) > 500


def test_reorder_parents_alignment(fs):
    assert _reorder(fs, parents=FAKE + 2) == UNSUPPORTED


@pytest.mark.parametrize("layout", [(0, 4096, 256, 4, 64, 32), (2, 4096, 256, 0, 64, 32), (2, 4096, 256, 4, 64, 0)])
def test_reorder_of_nothing(fs, layout):
    assert _reorder(fs, layout=layout) == OK


@pytest.mark.parametrize("shape,dim,index", [
    ((2, 6, 3, 10, 8), 1, (slice(None), slice(None), slice(None), slice(0, 7))),
    ((6, 3, 10, 8), 0, (slice(None), slice(None), slice(0, 4))),
    ((6, 5), 0, ()), ((4, 3, 6), 2, ()), ((2, 3, 6, 4), 2, (slice(None), slice(1, 3))), ((6,), 0, ()),
    ((6, 1, 8), 0, ()), ((1, 6, 2, 4), 1, (slice(None), slice(None), slice(0, 1))),
])
def test_layouts_name_every_byte_once(fs, shape, dim, index):
    """The bytes that a state's layout reaches are the view's own, row by row."""
    import torch
    base = torch.arange(int(torch.tensor(shape).prod()), dtype=torch.int16).reshape(shape)
    view = base[index]
    (layout, starts), = fs._beam_layouts(dim, view)
    rows = view.shape[dim]
    seen = {}
    for s in starts:
        for o in range(layout.outer):
            for r in range(rows):
                for k in range(layout.blocks):
                    at = s + o * layout.outer_stride + r * layout.row_stride + k * layout.block_stride
                    for byte in range(layout.block_bytes):
                        assert at + byte not in seen
                        seen[at + byte] = r
    offset = 2 * view.storage_offset()
    want = {}
    for r in range(rows):
        for v in view.select(dim, r).reshape(-1).tolist():
            want[2 * v - offset] = want[2 * v + 1 - offset] = r
    assert seen == want


def test_layouts_of_two_tensors_split_alike(fs):
    import torch
    view = torch.zeros(2, 6, 3, 10, 8, dtype=torch.int16)[:, :, :, :7]
    (a, sa), (b, sb) = fs._beam_layouts(1, view, torch.empty(2, 6, 3, 7, 8, dtype=torch.int16))
    assert (a.outer, a.blocks, a.block_bytes) == (b.outer, b.blocks, b.block_bytes) == (2, 3, 112)
    assert (a.block_stride, b.block_stride, a.row_stride, b.row_stride) == (160, 112, 480, 336) and sa == sb == [0]


def test_layouts_that_are_refused(fs):
    import torch
    t = torch.zeros(6, 4, 5, 6, dtype=torch.int16)[:, :3, :4, :5]    # two runs of blocks
    with pytest.raises(ValueError, match="blocks"):
        fs._beam_layouts(0, t)


def test_host_tensors_are_refused(fs):
    import torch
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    q = torch.zeros(2, 64, dtype=torch.int8)
    s = torch.zeros(2)
    for call in (lambda: fs.quantize_i8(x), lambda: fs.rms_norm_i8(x, x[0]), lambda: fs.matmul_i8(q, s, q, s),
                 lambda: fs.sample_i8(q, s, q, s, 1.0, 0, 0), lambda: fs.beam_select(x, s[:, None]),
                 lambda: fs.beam_reorder(x, torch.zeros(1, 2, dtype=torch.int32))):
        with pytest.raises(ValueError, match="device tensors"):
            call()


def test_shapes_and_types_are_refused(fs):
    import torch
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    q = torch.zeros(2, 64, dtype=torch.int8)
    s, i = torch.zeros(2), torch.zeros(1, 2, dtype=torch.int32)
    for call, error in (
            (lambda: fs.quantize_i8(x.half()), TypeError), (lambda: fs.quantize_i8(x[0]), ValueError),
            (lambda: fs.quantize_i8(x.t()), ValueError),
            (lambda: fs.rms_norm_i8(x, x[0, :32]), ValueError), (lambda: fs.rms_norm_i8(x, x[0], sum_out=x), ValueError),
            (lambda: fs.rms_norm_i8(x, x[0], residual=x.float()), ValueError),
            (lambda: fs.matmul_i8(q, s, q[:, :32], s), ValueError), (lambda: fs.matmul_i8(x, s, q, s), ValueError),
            (lambda: fs.matmul_i8(q, s[:1], q, s), ValueError), (lambda: fs.matmul_i8(q, s, q, s.double()), ValueError),
            (lambda: fs.beam_select(x, s), ValueError), (lambda: fs.beam_select(x, torch.zeros(3, 1)), ValueError),
            (lambda: fs.beam_select(x, torch.zeros(2, 1).double()), ValueError),
            (lambda: fs.beam_select(x, torch.zeros(2, 1), finished=torch.zeros(2, 1)), ValueError),
            (lambda: fs.beam_select(x, torch.zeros(2, 1), pad_token=2**32), ValueError),
            (lambda: fs.beam_reorder(x, i.long()), ValueError), (lambda: fs.beam_reorder([x, x.float()], i), ValueError),
            (lambda: fs.beam_reorder([], i), ValueError), (lambda: fs.beam_reorder(x, i, dim=1), ValueError),
            (lambda: fs.beam_reorder(x, i, out=[x, x]), ValueError)):
        with pytest.raises(error):
            call()

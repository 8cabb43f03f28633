"""The norms around a block (mole_block_norm_forward / _backward) against plain
fp64 forms; the bounds count the roundings (train_ops_ref)."""
import numpy as np
import pytest
import torch

import train_ops_ref as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-5


def _rand(rng, *shape, dtype=F32, std=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).to(dtype).cuda()


def _layer(rng, T, D, tx, tf, post=True, gate=True):
    x, f = _rand(rng, T, D, dtype=tx, std=2.0), _rand(rng, T, D, dtype=tf, std=0.3)
    w_post = _rand(rng, D) if post else None
    g = _rand(rng, T) if gate else None
    return x, f, w_post, g, _rand(rng, D)


def _check_forward(mole, x, f, w_post, gate, res_scale, w_pre, th, in_place=False):
    x0 = x.clone()
    x_out, h = mole.mole_block_norm_forward(x, f, w_post, gate, res_scale, w_pre, EPS, h_dtype=th,
                                            x_out=x if in_place else None)
    assert mole.mole_check() == 0
    r32 = float(np.float32(res_scale))
    xo, hh, bx, bh = ref.norm_forward(ref.f64(x0), ref.f64(f), ref.f64(w_post), ref.f64(gate), r32, ref.f64(w_pre),
                                      float(np.float32(EPS)))
    ref.assert_within(ref.f64(x_out), xo, bx + ref.HALF[x.dtype] * (np.abs(xo) + bx), "x'")
    if w_pre is not None:
        assert h.dtype == th
        ref.assert_within(ref.f64(h), hh, bh + ref.HALF[th] * (np.abs(hh) + bh), "h")
    return x_out, h


@pytest.mark.parametrize("tx,tf,th", [(F32, F32, BF16), (BF16, BF16, BF16), (F32, BF16, F32), (BF16, F32, F32)])
@pytest.mark.parametrize("T,D", [(1, 1), (1, 2048), (3, 7), (9, 64), (10, 20), (130, 256), (65, 264), (37, 1001), (20, 2056),
                                 (11, 4097), (6, 8192), (2000, 128), (5000, 512), (41, 2048), (300, 384), (200, 768), (70, 1576), (8, 4100), (9, 3001), (300, 301), (6, 7680)])
def test_forward(mole, T, D, tx, tf, th):
    rng = np.random.default_rng(T + D)
    _check_forward(mole, *_layer(rng, T, D, tx, tf)[:4], 0.8, _rand(rng, D), th)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [False, True])
def test_forward_parts(mole, post, gate):
    rng = np.random.default_rng(5)
    x, f, w_post, g, w_pre = _layer(rng, 45, 320, F32, F32, post, gate)
    _check_forward(mole, x.clone(), f, w_post, g, 1.0, None, BF16)         # the last block: no h
    _check_forward(mole, x.clone(), f, w_post, g, -0.5, w_pre, BF16, in_place=True)
    x_out, h = _check_forward(mole, x, None, None, None, 1.0, w_pre, F32)  # the first: no f
    assert x_out is x
    x_out, _ = _check_forward(mole, x, None, None, None, 2.0, w_pre, F32)  # a scaled stream
    assert x_out is not x


def test_forward_h_alone(mole):
    # h without x' (the C entry allows it): the same h
    rng = np.random.default_rng(6)
    x, f, w_post, g, w_pre = _layer(rng, 33, 136, F32, F32)
    _, want = mole.mole_block_norm_forward(x, f, w_post, g, 0.8, w_pre, EPS, h_dtype=F32)
    h = torch.empty_like(x)
    st = mole.lib.mole_block_norm_forward(x.data_ptr(), 0, f.data_ptr(), 0, w_post.data_ptr(), g.data_ptr(), 0.8,
                                          w_pre.data_ptr(), EPS, 33, 136, None, h.data_ptr(), 0,
                                          torch.cuda.current_stream().cuda_stream)
    assert st == 0 and mole.mole_check() == 0 and torch.equal(h, want)


def test_forward_special_rows(mole):
    # zero rows give zero rows (eps), NaN and infinities stay in their rows
    rng = np.random.default_rng(7)
    x, f, w_post, g, w_pre = _layer(rng, 40, 96, F32, F32)
    x[3], f[3] = 0, 0
    x[5, 7], f[9, 2], g[11] = float("nan"), float("inf"), float("nan")
    x_out, h = mole.mole_block_norm_forward(x, f, w_post, g, 0.8, w_pre, EPS, h_dtype=F32)
    assert mole.mole_check() == 0
    assert not x_out[3].any() and not h[3].any()
    assert torch.isnan(h[5]).all() and torch.isnan(h[9]).any() and torch.isnan(h[11]).all()
    rest = torch.ones(40, dtype=torch.bool, device="cuda")
    rest[[5, 9, 11]] = False
    assert torch.isfinite(h[rest]).all() and torch.isfinite(x_out[rest]).all()


def _check_backward(mole, x, f, w_post, gate, res_scale, w_pre, dx_out, dh, alias=False):
    T, D = x.shape
    rng = np.random.default_rng(99)
    dw_pre = _rand(rng, D) if dh is not None else None
    dw_post = _rand(rng, D) if w_post is not None else None
    p0, q0 = ref.f64(dw_pre), ref.f64(dw_post)
    want = ref.norm_backward(ref.f64(x), ref.f64(f), ref.f64(w_post), ref.f64(gate), float(np.float32(res_scale)),
                             ref.f64(w_pre), float(np.float32(EPS)), ref.f64(dx_out), ref.f64(dh))
    kw = dict(dx=dx_out, df=dh if f is not None else None) if alias else {}
    args = (x, dx_out, dh, f, w_post, gate, res_scale, w_pre, EPS)
    if not alias:
        again = [None if t is None else t.clone() for t in (dw_pre, dw_post)]
        first = mole.mole_block_norm_backward(*args, dw_pre=again[0], dw_post=again[1])
    dx, df, dgate = mole.mole_block_norm_backward(*args, dw_pre=dw_pre, dw_post=dw_post, **kw)
    assert mole.mole_check() == 0
    got = {"dx": dx, "df": df, "dgate": dgate, "dw_pre": dw_pre, "dw_post": dw_post}
    if not alias:
        for a, b in zip([*first, *again], got.values()):
            assert (a is None and b is None) or torch.equal(a, b), "two runs differ"
    for name, t in got.items():
        if t is None:
            continue
        value, bound = want[name]
        if name in ("dw_pre", "dw_post"):
            value = value + (p0 if name == "dw_pre" else q0)
            bound = bound + 2 * ref.U * np.abs(value)
        ref.assert_within(ref.f64(t), value, bound, name)


@pytest.mark.parametrize("tx,tf", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("T,D", [(1, 1), (1, 2048), (3, 7), (9, 64), (10, 20), (130, 256), (65, 264), (37, 1001), (20, 2056),
                                 (11, 4097), (6, 8192), (3000, 128), (5001, 72), (700, 512), (41, 2048), (9, 4096), (300, 384), (200, 768), (70, 1576), (8, 4100), (9, 3001), (300, 301), (6, 7680)])
def test_backward(mole, T, D, tx, tf):
    rng = np.random.default_rng(T + D)
    x, f, w_post, g, w_pre = _layer(rng, T, D, tx, tf)
    _check_backward(mole, x, f, w_post, g, 0.8, w_pre, _rand(rng, T, D), _rand(rng, T, D))


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("stream", ["both", "dx_out", "dh"])
def test_backward_parts(mole, post, gate, stream):
    rng = np.random.default_rng(8)
    x, f, w_post, g, w_pre = _layer(rng, 45, 320, F32, F32, post, gate)
    dx_out = _rand(rng, 45, 320) if stream != "dh" else None
    dh = _rand(rng, 45, 320) if stream != "dx_out" else None
    _check_backward(mole, x, f, w_post, g, -0.5, w_pre, dx_out, dh)
    _check_backward(mole, x, None, None, None, 1.0, w_pre, dx_out, dh)  # before the first block
    if stream == "both":
        _check_backward(mole, x, f, w_post, g, 0.8, w_pre, dx_out, dh, alias=True)


def test_backward_gate_without_f(mole):
    # y = f: df = gate G needs no f (the C entry; dx, dgate not asked for)
    rng = np.random.default_rng(9)
    dx_out, g = _rand(rng, 21, 40), _rand(rng, 21)
    df = torch.empty_like(dx_out)
    st = mole.lib.mole_block_norm_backward(None, 0, None, 0, None, g.data_ptr(), 0.8, None, EPS, 21, 40,
                                           dx_out.data_ptr(), None, None, df.data_ptr(), None, None, None, None, 0,
                                           torch.cuda.current_stream().cuda_stream)
    assert st == 0 and mole.mole_check() == 0
    assert torch.equal(df, g[:, None] * dx_out)


def test_backward_special_rows(mole):
    # zero rows have finite gradients; a NaN row reaches the weights' sums and no other row
    rng = np.random.default_rng(10)
    x, f, w_post, g, w_pre = _layer(rng, 40, 96, F32, F32)
    dx_out, dh = _rand(rng, 40, 96), _rand(rng, 40, 96)
    x[3], f[3] = 0, 0
    dx, df, dg = mole.mole_block_norm_backward(x, dx_out, dh, f, w_post, g, 0.8, w_pre, EPS)
    assert all(torch.isfinite(t).all() for t in (dx, df, dg))
    dh[5, 1] = float("nan")
    dx2, df2, dg2 = mole.mole_block_norm_backward(x, dx_out, dh, f, w_post, g, 0.8, w_pre, EPS)
    assert mole.mole_check() == 0
    keep = torch.arange(40, device="cuda") != 5
    assert torch.isnan(dx2[5]).all() and torch.isnan(df2[5]).all() and torch.isnan(dg2[5])
    for a, b in ((dx, dx2), (df, df2), (dg, dg2)):
        assert torch.equal(a[keep], b[keep])


def test_unaligned_rows(mole):
    # rows that start inside a buffer take the scalar kernels; what lies around is left alone
    rng = np.random.default_rng(11)
    T, D = 30, 64
    x, f, w_post, g, w_pre = _layer(rng, T, D, BF16, F32)
    _check_forward(mole, _rand(rng, T * D + 1, dtype=BF16)[1:].view(T, D), f, w_post, g, 0.8, w_pre, BF16)
    buf = torch.full((T * D + 2,), 3.0, device="cuda")
    dx_out, dh = _rand(rng, T, D), _rand(rng, T, D)
    mole.mole_block_norm_backward(x, dx_out, dh, f, w_post, g, 0.8, w_pre, EPS, dx=buf[1:-1].view(T, D))
    want = ref.norm_backward(ref.f64(x), ref.f64(f), ref.f64(w_post), ref.f64(g), float(np.float32(0.8)),
                             ref.f64(w_pre), float(np.float32(EPS)), ref.f64(dx_out), ref.f64(dh))
    ref.assert_within(ref.f64(buf[1:-1]).reshape(T, D), *want["dx"], "dx")
    assert float(buf[0]) == 3.0 and float(buf[-1]) == 3.0


# Rows that start anywhere in a unit of 4: every width mod 4, widths around a
# thread's or a unit's end, more rows than CTAs (each shift takes its own ones),
# and widths whose rows are too long for the shifted units.
@pytest.mark.parametrize("T,D", [(6, 125), (9, 126), (7, 127), (4, 383), (5, 767), (3, 1534), (4, 1535), (3, 2046),
                                 (4, 2047), (5, 4093), (3, 4095), (2, 5633), (2, 7041), (2, 8189), (2, 8190), (3, 8191),
                                 (4001, 61), (3000, 130), (2600, 131), (1700, 641), (1501, 1153)])
@pytest.mark.parametrize("tx,tf", [(F32, BF16), (BF16, F32)])
def test_shifted_rows(mole, T, D, tx, tf):
    rng = np.random.default_rng(D)
    x, f, w_post, g, w_pre = _layer(rng, T + 1, D, tx, tf)
    x[T], f[T], g[T] = float("nan"), float("nan"), float("nan")  # behind the batch: must not get in
    x, f, g = x[:T], f[:T], g[:T]
    dx_out, dh = _rand(rng, T, D), _rand(rng, T, D)
    _check_backward(mole, x, f, w_post, g, 0.7, w_pre, dx_out, dh)
    _check_backward(mole, x, f, w_post, None, 0.7, w_pre, None, dh)
    _check_forward(mole, x, f, w_post, g, 0.8, w_pre, BF16)
    _check_forward(mole, x, f, w_post, g, 0.8, w_pre, F32, in_place=True)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [False, True])
def test_shifted_rows_parts(mole, post, gate):
    rng = np.random.default_rng(15)
    T, D = 2700, 323
    x, f, w_post, g, w_pre = _layer(rng, T, D, F32, BF16, post, gate)
    dx_out, dh = _rand(rng, T, D), _rand(rng, T, D)
    _check_forward(mole, x.clone(), f, w_post, g, 1.0, None, BF16)
    _check_forward(mole, x.clone(), f, w_post, g, -0.5, w_pre, BF16, in_place=True)
    _check_forward(mole, x, None, None, None, 1.0, w_pre, F32)
    _check_backward(mole, x, f, w_post, g, 0.6, None, dx_out, None)
    _check_backward(mole, x, f, w_post, g, 0.6, w_pre, None, dh)
    _check_backward(mole, x, f, w_post, g, 0.6, w_pre, dx_out.clone(), dh.clone(), alias=True)
    _check_backward(mole, x, None, None, None, 0.6, w_pre, dx_out, dh)


def test_shifted_rows_alone(mole):
    # a unit that two rows share: NaN in one stays there, and nothing is written behind the last row
    rng = np.random.default_rng(13)
    T, D = 2500, 67
    x, f, w_post, g, w_pre = _layer(rng, T, D, F32, F32)
    dx_out, dh = _rand(rng, T, D), _rand(rng, T, D)
    bad = torch.arange(1, T, 2, device="cuda")
    good = torch.arange(0, T, 2, device="cuda")
    want = (*mole.mole_block_norm_forward(x, f, w_post, g, 0.8, w_pre, EPS, h_dtype=F32),
            *mole.mole_block_norm_backward(x, dx_out, dh, f, w_post, g, 0.8, w_pre, EPS))
    for t in (x, f, dx_out, dh):
        t[bad] = float("nan")
    bufs = [torch.full((T + 1, D), 5.0, device="cuda") for _ in range(4)]
    mole.mole_block_norm_forward(x, f, w_post, g, 0.8, w_pre, EPS, x_out=bufs[0][:T], h=bufs[1][:T])
    _, _, dgate = mole.mole_block_norm_backward(x, dx_out, dh, f, w_post, g, 0.8, w_pre, EPS, dx=bufs[2][:T],
                                                df=bufs[3][:T])
    assert mole.mole_check() == 0
    for got, w in zip((*bufs, dgate), want):
        assert torch.equal(got[good], w[good])
    assert all(bool((b[T] == 5.0).all()) for b in bufs)


@pytest.mark.parametrize("T,D", [(30, 301), (20, 1001), (5, 3001)])
def test_element_rows(mole, T, D):
    # tensors that start inside a unit, rows of every kind of width
    rng = np.random.default_rng(14)
    _, f, w_post, g, w_pre = _layer(rng, T, D, BF16, F32)
    x = _rand(rng, T * D + 1, dtype=BF16)[1:].view(T, D)
    _check_forward(mole, x, f, w_post, g, 0.8, w_pre, BF16)
    _check_backward(mole, x, f, w_post, g, 0.8, w_pre, _rand(rng, T, D), _rand(rng, T, D))


def test_graph_and_stream(mole):
    rng = np.random.default_rng(12)
    T, D = 500, 256
    x, f, w_post, g, w_pre = _layer(rng, T, D, F32, F32)
    dx_out, dh = _rand(rng, T, D), _rand(rng, T, D)
    dw_pre, dw_post = torch.zeros(D, device="cuda"), torch.zeros(D, device="cuda")
    h, x_out = torch.empty(T, D, device="cuda", dtype=BF16), torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mole.mole_block_norm_forward(x, f, w_post, g, 0.8, w_pre, EPS, x_out=x_out, h=h)
        dx, df, dg = mole.mole_block_norm_backward(x_out, dx_out, dh, f, w_post, g, 0.8, w_pre, EPS, dw_pre=dw_pre,
                                                   dw_post=dw_post)
    for seed in (1, 2):
        rng = np.random.default_rng(seed)
        for t in (x, f, dx_out, dh):
            t.copy_(_rand(rng, T, D))
        dw_pre.zero_()
        dw_post.zero_()
        graph.replay()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        xo, hh = mole.mole_block_norm_forward(x, f, w_post, g, 0.8, w_pre, EPS, stream=side)
        p, q = torch.zeros(D, device="cuda"), torch.zeros(D, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        want = mole.mole_block_norm_backward(xo, dx_out, dh, f, w_post, g, 0.8, w_pre, EPS, dw_pre=p, dw_post=q,
                                             stream=side)
        side.synchronize()
        for a, b in zip((x_out, h, dx, df, dg, dw_pre, dw_post), (xo, hh, *want, p, q)):
            assert torch.equal(a, b)
    assert mole.mole_check() == 0


def test_empty_batch(mole):
    x = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    x_out, h = mole.mole_block_norm_forward(x, x.clone(), w, None, 1.0, w)
    assert x_out.shape == (0, 64) and h.shape == (0, 64)
    dw = torch.ones(64, device="cuda")
    mole.mole_block_norm_backward(x, x, x, x, w, None, 1.0, w, dw_pre=dw, dw_post=dw.clone())
    assert mole.mole_check() == 0 and bool((dw == 1).all())


# Rows for three turns of every CTA (as many as fit the GPU at once) in the forms
# that the lists above give one turn: single elements of 4, 8 and 16 columns a
# thread, over 4096 columns by units and by shifted ones, and backward rows too
# long for the stages or for shifted units.
@pytest.mark.parametrize("T,D,offset,tx,tf", [
    (9400, 301, 1, BF16, F32), (7200, 1001, 1, F32, BF16), (4500, 3001, 1, BF16, BF16), (1900, 4100, 1, F32, F32),
    (1900, 4100, 0, F32, F32), (1900, 4101, 0, BF16, F32), (1000, 5633, 0, F32, F32), (1000, 6656, 0, F32, F32),
    (1000, 7680, 0, F32, F32), (1000, 8191, 0, F32, F32), (1000, 8192, 0, BF16, BF16), (1000, 8192, 0, F32, F32)])
def test_many_rows(mole, T, D, offset, tx, tf):
    rng = np.random.default_rng(D)
    buf = torch.full((offset + (T + 1) * D,), float("nan"), dtype=tx, device="cuda")
    x = buf[offset:offset + T * D].view(T, D)
    x.copy_(_rand(rng, T, D, dtype=tx, std=2.0))
    _, f, w_post, g, w_pre = _layer(rng, T, D, tx, tf)
    _check_forward(mole, x, f, w_post, g, 0.8, w_pre, BF16)
    _check_backward(mole, x, f, w_post, g, 0.8, w_pre, _rand(rng, T, D), _rand(rng, T, D))
    # parts: one sum a row in place of two
    _check_forward(mole, x, None, None, None, 1.0, w_pre, F32)
    _check_backward(mole, x, None, None, None, 0.7, w_pre, None, _rand(rng, T, D))
    assert bool(buf[offset + T * D:].isnan().all())


def test_binding_backward_gate_without_f(mole):
    # df = gate G needs no f where there is no post-norm; dgate, which does, is not made
    rng = np.random.default_rng(16)
    x, _, _, g, w_pre = _layer(rng, 21, 40, F32, F32)
    dx_out, dh = _rand(rng, 21, 40), _rand(rng, 21, 40)
    f = _rand(rng, 21, 40)
    want = mole.mole_block_norm_backward(x, dx_out, dh, f, None, g, 0.8, w_pre, EPS)
    df = torch.empty_like(dx_out)
    dx, got, dgate = mole.mole_block_norm_backward(x, dx_out, dh, None, None, g, 0.8, w_pre, EPS, df=df)
    assert mole.mole_check() == 0 and got is df and dgate is None
    assert torch.equal(dx, want[0]) and torch.equal(df, want[1])


@pytest.mark.parametrize("T,D", [(1, 24), (45, 320), (2700, 323), (3000, 1024)])
def test_backward_one_weight_for_both_norms(mole, T, D):
    # w_pre is w_post and so are their gradients: both sums, dw_pre's first
    rng = np.random.default_rng(17)
    x, f, w, g, _ = _layer(rng, T, D, F32, F32)
    dx_out, dh, start = _rand(rng, T, D), _rand(rng, T, D), _rand(rng, D)
    pre, post = start.clone(), torch.zeros(D, device="cuda")
    want = mole.mole_block_norm_backward(x, dx_out, dh, f, w, g, 0.8, w, EPS, dw_pre=pre, dw_post=post)
    for _ in range(3):
        dw = start.clone()
        got = mole.mole_block_norm_backward(x, dx_out, dh, f, w, g, 0.8, w, EPS, dw_pre=dw, dw_post=dw)
        assert mole.mole_check() == 0
        assert torch.equal(dw, pre + post) and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T,D", [(1048600, 2056), (2200000, 981)])
def test_rows_beyond_2_31_elements(mole, T, D):
    # the last rows and some at 2^31 elements: the bits of a call on them alone
    rng = np.random.default_rng(D)
    part = 3000                                          # (rows that take the same kernels)
    at = [0, (1 << 31) // D // 4 * 4 - 2000, T // 4 * 4 - part]  # (rows and their shifts)
    x, f, w_post, g, w_pre = _layer(rng, part, D, BF16, BF16)
    dx_out, dh = _rand(rng, part, D), _rand(rng, part, D)
    want = (*mole.mole_block_norm_forward(x, f, w_post, g, 0.8, w_pre, EPS),
            *mole.mole_block_norm_backward(x, dx_out, dh, f, w_post, g, 0.8, w_pre, EPS))
    big = [torch.zeros(T, *t.shape[1:], dtype=t.dtype, device="cuda") for t in (x, f, g, dx_out, dh)]
    for i in at:
        for b, t in zip(big, (x, f, g, dx_out, dh)):
            b[i:i + part] = t
    X, F, G, DX, DH = big
    backward = mole.mole_block_norm_backward(X, DX, DH, F, w_post, G, 0.8, w_pre, EPS, dx=DX, df=DH)
    forward = mole.mole_block_norm_forward(X, F, w_post, G, 0.8, w_pre, EPS, x_out=X)
    assert mole.mole_check() == 0
    for got, w in zip((*forward, *backward), want):
        for i in at:
            assert torch.equal(got[i:i + part], w), i
        assert not got[part:at[1]].any() and not got[at[1] + part:at[2]].any()

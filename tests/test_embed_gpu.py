"""The embedding lookup and its gradient (mole_embed_forward / _backward)
against plain fp64 forms.  Bounds: a lookup is one product and one rounding to
the output's type; a gradient row of c tokens is c additions, a product and the
addition to dE (train_ops_ref)."""
import numpy as np
import pytest
import torch

import train_ops_ref as ref
from helpers import dev
from mixture_lookup_experts_b200 import inputs

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _rand(rng, *shape, dtype=F32, std=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).to(dtype).cuda()


def _check_forward(mole, rng, T, V, D, tin, tout, ids=None, scale=3.7):
    E = _rand(rng, V, D, dtype=tin)
    ids = inputs.uniform_ids(rng, T, V) if ids is None else ids
    out = mole.mole_embed_forward(dev(ids), E, scale, out_dtype=tout)
    assert out.dtype == tout and mole.mole_check() == 0
    want = float(np.float32(scale)) * ref.f64(E)[ids]
    ref.assert_within(ref.f64(out), want, (ref.U + ref.HALF[tout]) * (1 + 2.0 ** -7) * np.abs(want))


@pytest.mark.parametrize("tin", [F32, BF16])
@pytest.mark.parametrize("tout", [F32, BF16])
@pytest.mark.parametrize("T,V,D", [(1, 1, 1), (1, 50304, 2048), (7, 3, 8), (19, 40, 20), (33, 100, 1001), (300, 50, 72),
                                   (513, 1000, 2056), (5, 9, 4099)])
def test_forward(mole, T, V, D, tin, tout):
    _check_forward(mole, np.random.default_rng(T + D), T, V, D, tin, tout)


def test_forward_ids_at_both_ends_and_bad(mole):
    rng = np.random.default_rng(1)
    V, D = 77, 136
    E = _rand(rng, V, D, dtype=BF16)
    ids = np.array([0, V - 1, -1, V, 2 ** 31 - 1, -2 ** 31, 5], np.int32)
    out = mole.mole_embed_forward(dev(ids), E, 1.0)
    assert mole.mole_check() == 5
    bad = np.array([False, False, True, True, True, True, False])
    assert torch.isnan(out[dev(bad)]).all()
    assert torch.equal(out[dev(~bad)], E[dev(ids[~bad]).long()])
    assert mole.mole_check() == 0


def test_forward_from_unaligned_rows(mole):
    # a table and an output that start inside a buffer take the scalar kernel
    rng = np.random.default_rng(2)
    V, D, T = 40, 64, 50
    buf = _rand(rng, V * D + 3)
    E = buf[3:].view(V, D)
    out_buf = torch.full((T * D + 1,), 7.0, dtype=BF16, device="cuda")
    out = out_buf[1:].view(T, D)
    ids = inputs.uniform_ids(rng, T, V)
    mole.mole_embed_forward(dev(ids), E, 2.0, out=out)
    assert mole.mole_check() == 0
    assert torch.equal(out, (E[dev(ids).long()] * 2.0).to(BF16)) and float(out_buf[0]) == 7.0


# Widths that are no multiple of 4: rows of the table and of the output start at
# different places in a unit; one row a thread and four; a table that ends
# inside a unit, its last row and its first one among the ids.
@pytest.mark.parametrize("tin", [F32, BF16])
@pytest.mark.parametrize("tout", [F32, BF16])
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("T,V,D", [(50, 5, 1), (40, 7, 2), (61, 3, 5), (10001, 51, 67), (12000, 31, 130), (6001, 7, 301),
                                   (700, 9, 2045), (300, 5, 2046), (211, 3, 2047)])
def test_forward_shifted_rows(mole, T, V, D, offset, tin, tout):
    rng = np.random.default_rng(D)
    buf = _rand(rng, offset + V * D, dtype=tin)  # (offset 1: single columns)
    E = buf[offset:].view(V, D)
    ids = rng.integers(0, V, T).astype(np.int32)
    ids[0], ids[-1], ids[T // 2] = 0, V - 1, -3
    out = torch.full((T + 1, D), 7.0, dtype=tout, device="cuda")
    mole.mole_embed_forward(dev(ids), E, 2.0, out=out[:T])
    assert mole.mole_check() == 5
    keep = torch.from_numpy(ids >= 0).cuda()
    assert torch.equal(out[:T][keep], (E[dev(ids).long()[keep]] * 2.0).to(tout))
    assert torch.isnan(out[T // 2]).all() and bool((out[T] == 7.0).all())


def test_forward_table_beyond_2_31_elements(mole):
    # row offsets pass 32 bits: 2^31 + elements of bf16
    V, D = 1048600, 2056
    E = torch.empty((V, D), dtype=BF16, device="cuda")
    ids = torch.tensor([0, 1, V - 1, V - 2, 1044500], dtype=torch.int32, device="cuda")
    E[ids.long()] = torch.arange(5, device="cuda", dtype=BF16)[:, None] + 1
    out = mole.mole_embed_forward(ids, E, 1.0)
    assert mole.mole_check() == 0
    assert torch.equal(out, E[ids.long()])


def _check_backward(mole, rng, T, V, D, dtype, ids, scale=1.3, dout=None):
    dout = _rand(rng, T, D, dtype=dtype) if dout is None else dout
    dE = _rand(rng, V, D)
    start = dE.clone()
    again = dE.clone()
    mole.mole_embed_backward(dev(ids), dout, dE, scale)
    mole.mole_embed_backward(dev(ids), dout, again, scale)
    bad = bool(((ids < 0) | (ids >= V)).any())
    assert mole.mole_check() == (5 if bad else 0)
    want, bound = ref.embed_backward(ids, ref.f64(dout), ref.f64(start), float(np.float32(scale)), V)
    ref.assert_within(ref.f64(dE), want, bound)
    assert torch.equal(dE, again), "two runs differ"
    untouched = np.setdiff1d(np.arange(V), ids)
    assert torch.equal(dE[dev(untouched)], start[dev(untouched)])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,V,D,kind", [
    (1, 1, 1, "uniform"), (1, 50304, 64, "zipf"), (2, 1, 24, "uniform"),   # a key of one bit, one token
    (31, 5, 40, "uniform"), (257, 300, 1001, "zipf"),                      # odd width: scalar columns
    (1000, 40, 512, "uniform"),                                           # every run crosses chunks
    (2500, 900, 20, "zipf"), (2300, 30, 1001, "zipf"),                  # units of 4 columns; odd width
    (3001, 70000, 136, "zipf"),                                           # three digits of key
    (5000, 300, 2056, "zipf"), (9999, 2, 72, "uniform"),
    (20000, 50304, 256, "zipf"),
])
def test_backward(mole, T, V, D, kind, dtype):
    rng = np.random.default_rng(T * 7 + V)
    _check_backward(mole, rng, T, V, D, dtype, inputs.draw_ids(rng, T, V, kind))


@pytest.mark.parametrize("T", [1, 15, 16, 17, 32, 33, 1024, 1025, 2048, 2049, 4096, 40000])
def test_backward_one_id(mole, T):
    # all tokens one id: a single run over every chunk
    rng = np.random.default_rng(T)
    _check_backward(mole, rng, T, 9, 64, F32, np.full(T, 4, np.int32))


def test_backward_runs_that_end_on_chunk_borders(mole):
    # runs of exactly 16 and 32 tokens: nothing crosses, every chunk is one run
    rng = np.random.default_rng(3)
    ids = np.repeat(np.arange(40), 16).astype(np.int32)
    _check_backward(mole, rng, ids.size, 50, 64, F32, rng.permutation(ids))
    ids = np.repeat(np.arange(21), 32).astype(np.int32)
    _check_backward(mole, rng, ids.size, 21, 64, BF16, rng.permutation(ids))


@pytest.mark.parametrize("T,V,D", [(256, 30, 33), (257, 30, 33), (258, 2, 17), (511, 60, 100), (777, 4, 2368),
                                   (1024, 900, 2369), (1023, 1, 15), (300, 200, 16)])
def test_backward_small_batches(mole, T, V, D):
    # one launch: shares of every length, runs across many shares, strips of both widths
    rng = np.random.default_rng(T)
    _check_backward(mole, rng, T, V, D, BF16, rng.integers(0, V, T).astype(np.int32))
    _check_backward(mole, rng, T, V, D, F32, np.sort(rng.integers(-1, V, T)).astype(np.int32))


def test_backward_bad_ids(mole):
    rng = np.random.default_rng(4)
    T, V, D = 777, 60, 96
    ids = inputs.uniform_ids(rng, T, V)
    ids[::5] = -1
    ids[3::50] = V
    ids[4::70] = 2 ** 31 - 1
    _check_backward(mole, rng, T, V, D, F32, ids)
    _check_backward(mole, rng, T, V, D, BF16, np.full(T, -7, np.int32))  # none left


def test_backward_bad_tokens_do_not_spread(mole):
    # NaN and infinite rows of tokens with bad ids reach nothing
    rng = np.random.default_rng(5)
    T, V, D = 200, 30, 64
    ids = inputs.uniform_ids(rng, T, V)
    ids[:50] = -1
    dout = _rand(rng, T, D)
    dout[:25] = float("nan")
    dout[25:50] = float("inf")
    dE = torch.zeros(V, D, device="cuda")
    mole.mole_embed_backward(dev(ids), dout, dE)
    assert mole.mole_check() == 5
    want, bound = ref.embed_backward(ids[50:], ref.f64(dout)[50:], np.zeros((V, D)), 1.0, V)
    ref.assert_within(ref.f64(dE), want, bound)


def test_backward_from_unaligned_rows(mole):
    rng = np.random.default_rng(6)
    T, V, D = 90, 20, 64
    ids = inputs.zipf_ids(rng, T, V)
    dout = _rand(rng, T * D + 1, dtype=BF16)[1:].view(T, D)
    _check_backward(mole, rng, T, V, D, BF16, ids, dout=dout)
    buf = torch.zeros(V * D + 2, device="cuda")
    mole.mole_embed_backward(dev(ids), dout, buf[1:-1].view(V, D))
    assert mole.mole_check() == 0
    want, bound = ref.embed_backward(ids, ref.f64(dout), np.zeros((V, D)), 1.0, V)
    ref.assert_within(ref.f64(buf[1:-1]).reshape(V, D), want, bound)
    assert float(buf[0]) == 0.0 and float(buf[-1]) == 0.0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("offset", [0, 1, 2, 3])
@pytest.mark.parametrize("T,V,D", [(1501, 90, 1), (1100, 400, 3), (2049, 37, 67), (1027, 9, 131), (1301, 700, 1613),
                                   (1025, 2000, 514), (4097, 60, 34)])
def test_backward_single_columns(mole, T, V, D, offset, dtype):
    # rows that are no vector ones, from every place of a tensor in 4 elements: all
    # columns, the first and the last of the tensor among them, and no other's
    rng = np.random.default_rng(D)
    buf = torch.full((offset + T * D + 1,), float("nan"), dtype=dtype, device="cuda")
    dout = buf[offset:offset + T * D].view(T, D)
    dout.copy_(_rand(rng, T, D, dtype=dtype))
    _check_backward(mole, rng, T, V, D, dtype, rng.integers(0, V, T).astype(np.int32), dout=dout)


def test_backward_large_batch_and_vocabulary(mole):
    # 200000 tokens over 2^24 + ids (four digits of key), checked by torch in fp64
    rng = np.random.default_rng(7)
    T, V, D = 200000, (1 << 24) + 5, 8
    ids = inputs.uniform_ids(rng, T, V)
    ids[:5000] = V - 1
    dout = _rand(rng, T, D)
    dE = torch.zeros(V, D, device="cuda")
    mole.mole_embed_backward(dev(ids), dout, dE)
    assert mole.mole_check() == 0
    want = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, dev(ids), dout.double())
    mag = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, dev(ids), dout.double().abs())
    assert bool(((dE.double() - want).abs() <= 5004 * ref.U * mag).all())


@pytest.mark.parametrize("T,V,D", [(8_000_000, 3, 4), (3_000_000, 1000, 8), (300_000, 70, 1030)])
def test_backward_very_large_batches(mole, T, V, D):
    # narrow rows (many chunks per CTA) and chunks of many tokens, checked by torch in fp64
    ids = torch.randint(0, V, (T,), dtype=torch.int32, device="cuda")
    dout = torch.randn(T, D, device="cuda").to(BF16)
    dE = torch.zeros(V, D, device="cuda")
    mole.mole_embed_backward(ids, dout, dE)
    assert mole.mole_check() == 0
    want = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, ids, dout.double())
    mag = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, ids, dout.double().abs())
    count = torch.bincount(ids.long(), minlength=V)[:, None]
    assert bool(((dE.double() - want).abs() <= (count + 4) * ref.U * mag).all())


def test_backward_on_a_stream_and_in_a_graph(mole):
    rng = np.random.default_rng(8)
    T, V, D = 3000, 500, 128
    ids, dout = dev(inputs.zipf_ids(rng, T, V)), _rand(rng, T, D)
    want = mole.mole_embed_backward(ids, dout, torch.zeros(V, D, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mole.mole_embed_backward(ids, dout, torch.zeros(V, D, device="cuda"), stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    # captured once, replayed on new inputs in the same buffers
    dE, out = torch.zeros(V, D, device="cuda"), torch.empty(T, D, device="cuda")
    E = _rand(rng, V, D)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mole.mole_embed_forward(ids, E, 2.0, out=out)
        mole.mole_embed_backward(ids, dout, dE)
    for seed in (1, 2):
        rng = np.random.default_rng(seed)
        ids.copy_(dev(inputs.zipf_ids(rng, T, V)))
        dout.copy_(_rand(rng, T, D))
        dE.zero_()
        graph.replay()
        assert torch.equal(out, E[ids.long()] * 2.0)
        assert torch.equal(dE, mole.mole_embed_backward(ids, dout, torch.zeros(V, D, device="cuda")))
    assert mole.mole_check() == 0


def test_empty_batch(mole):
    E = torch.ones(4, 8, device="cuda")
    ids = torch.empty(0, dtype=torch.int32, device="cuda")
    assert mole.mole_embed_forward(ids, E).shape == (0, 8)
    dE = torch.ones(4, 8, device="cuda")
    mole.mole_embed_backward(ids, torch.empty(0, 8, device="cuda"), dE)
    assert mole.mole_check() == 0 and bool((dE == 1).all())


def _check_between_rows(mole, ids, dout, V, scale=1.3):
    """The gradient into rows 1 .. V of a buffer, by torch in fp64: what the
    batch does not hold, the row before the first and the one behind the last
    (that of key V) stay as they were; two runs agree."""
    T, D = dout.shape
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    buf = torch.randn(V + 2, D, generator=g, device="cuda")
    start, again = buf.clone(), buf.clone()
    d_ids = dev(ids)
    mole.mole_embed_backward(d_ids, dout, buf[1:-1], scale)
    mole.mole_embed_backward(d_ids, dout, again[1:-1], scale)
    ok = (d_ids >= 0) & (d_ids < V)
    assert mole.mole_check() == (0 if bool(ok.all()) else 5)
    assert torch.equal(buf, again), "two runs differ"
    rows, terms = d_ids[ok].long() + 1, dout[ok].double() * float(np.float32(scale))
    want, mag = start.double().index_add_(0, rows, terms), start.double().abs().index_add_(0, rows, terms.abs())
    count = torch.bincount(rows, minlength=V + 2)[:, None]
    bound = torch.where(count > 0, (count + 4) * ref.U * mag, 0.0)
    assert bool(((buf.double() - want).abs() <= bound).all())


# Batches of every form of the sort (one CTA, the cluster with 1 and 4 tiles a
# warp, through global memory) with ids outside [0, V); their key V takes one
# digit more than the ids of V = 2^8 and 2^16.
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [72, 67])
@pytest.mark.parametrize("V", [200, 256, 65536])
@pytest.mark.parametrize("T", [1025, 1500, 5000, 20000, 70000])
def test_backward_bad_ids_in_large_batches(mole, T, V, D, dtype):
    rng = np.random.default_rng(T + V)
    dout = _rand(rng, T, D, dtype=dtype)
    ids = inputs.zipf_ids(rng, T, V).copy()
    ids[rng.random(T) < 0.3] = V                     # a run of many chunks behind the last row's
    ids[rng.random(T) < 0.05] = -1
    ids[rng.random(T) < 0.05] = 2 ** 31 - 1
    ids[rng.random(T) < 0.05] = V - 1                # (the run that borders on it)
    ids[7] = -2 ** 31
    dout[dev((ids < 0) | (ids >= V))] = float("nan")  # reaches nothing
    _check_between_rows(mole, ids, dout, V)
    few = inputs.zipf_ids(rng, T, V).copy()
    few[T // 2] = V                                  # one
    _check_between_rows(mole, few, dout.nan_to_num(), V)
    _check_between_rows(mole, np.full(T, -7, np.int32), torch.full_like(dout, float("nan")), V)  # none left


def _runs(lengths, rng):
    """Tokens in random order whose ids sort into runs of these lengths."""
    return rng.permutation(np.repeat(np.arange(len(lengths)), lengths)).astype(np.int32)


# Runs of less than a chunk, of exactly one or two and a token more or less, that
# begin at every place of a chunk (8 tokens at these sizes).
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [64, 67])
@pytest.mark.parametrize("length", [1, 7, 8, 9, 15, 16, 17, 23, 24, 25])
def test_backward_runs_at_chunk_borders(mole, length, D, dtype):
    rng = np.random.default_rng(length)
    for offset in range(8):
        lengths = [offset] * (offset > 0) + [length] * (2100 // length + 1)
        ids = _runs(lengths, rng)
        _check_between_rows(mole, ids, _rand(rng, ids.size, D, dtype=dtype), len(lengths))


# The same with longer chunks (23 tokens at 40000 x 1024, several groups a CTA and
# one), and with runs of all of these lengths side by side.
@pytest.mark.parametrize("T,D,chunk", [(9000, 64, 8), (9000, 67, 8), (40000, 1024, 23), (40000, 1021, 23)])
def test_backward_mixed_runs_at_chunk_borders(mole, T, D, chunk):
    rng = np.random.default_rng(D)
    for dtype in (F32, BF16):
        near = [k * chunk + d for k in range(6) for d in (-1, 0, 1) if k * chunk + d > 0]
        lengths = []
        while sum(lengths) < T:
            lengths.append(int(rng.choice(near)))
        lengths[-1] -= sum(lengths) - T
        assert lengths[-1] > 0
        ids = _runs(lengths, rng)
        assert ids.size == T
        _check_between_rows(mole, ids, _rand(rng, T, D, dtype=dtype), len(lengths))
        ids[ids == len(lengths) - 1] = len(lengths) + 5  # the last run: ids outside the table
        _check_between_rows(mole, ids, _rand(rng, T, D, dtype=dtype), len(lengths) - 1)


def test_backward_beyond_2_31_elements(mole):
    # a gradient of 2^31 + elements: the same bits as with the rows put together
    rng = np.random.default_rng(9)
    T, V, D = 3000, 1048600, 2056
    few = np.sort(rng.choice(V, 300, replace=False))
    few[0], few[-1] = 0, V - 1
    small = rng.integers(0, 300, T).astype(np.int32)
    small[:2] = 0, 299
    dout = _rand(rng, T, D)
    want = mole.mole_embed_backward(dev(small), dout, torch.ones(300, D, device="cuda"), 1.5)
    dE = torch.ones(V, D, device="cuda")
    mole.mole_embed_backward(dev(few[small].astype(np.int32)), dout, dE, 1.5)
    assert mole.mole_check() == 0
    rows = dev(few)
    assert torch.equal(dE[rows], want)
    dE[rows] = 1.0
    assert float(dE.min()) == 1.0 and float(dE.max()) == 1.0
    del dE, want, dout
    # rows of dout behind 2^31 elements: the last tokens are all that is not zero
    T, V, D, last = 1048600, 50, 2056, 64
    dout = torch.zeros(T, D, dtype=BF16, device="cuda")
    dout[-last:] = _rand(rng, last, D, dtype=BF16)
    ids = torch.randint(0, V, (T,), dtype=torch.int32, device="cuda")
    dE = torch.zeros(V, D, device="cuda")
    mole.mole_embed_backward(ids, dout, dE)
    assert mole.mole_check() == 0
    # (adding zeros rounds nothing)
    want, bound = ref.embed_backward(ids[-last:].cpu().numpy(), ref.f64(dout[-last:]), np.zeros((V, D)), 1.0, V)
    ref.assert_within(ref.f64(dE), want, bound)

"""The AdamW step (mole_adamw_step) against the plain fp64 step; bounds count
the roundings (train_ops_ref).  An 8-bit state is off by at most half a step of
e4m3 (2^-4 of the value; half of 2^-9 scales below the smallest normal code),
and a root of v that is not zero is at least 2^-9 scales."""
import numpy as np
import pytest
import torch

import train_ops_ref as ref

pytestmark = pytest.mark.gpu

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8, step=3)


def _blocks(n):
    return (n + 127) // 128


def _state8(rng, n, std, root):
    """Codes and scales of n values spread over several decades."""
    w = rng.standard_normal(n) * std * 10.0 ** rng.uniform(-4, 0, n)
    w = np.abs(w) if root else w
    pad = np.zeros(_blocks(n) * 128)
    pad[:n] = w
    b = torch.from_numpy(pad.astype(np.float32)).view(-1, 128)
    scale = (b.abs().amax(1) / 448.0).clamp_min(2.0 ** -120)
    return (b / scale[:, None]).to(E4M3).view(-1)[:n].clone().cuda(), scale.cuda()


def _tensor(rng, n, param, grad, state, shape=None):
    t = {}
    p = torch.from_numpy((rng.standard_normal(n) * 0.02).astype(np.float32)).cuda()
    t["p"] = p.clone() if param == "f32" else p.to(BF16)
    t["w"] = p.clone() if param == "master" else None
    g = (rng.standard_normal(n) * 1e-3 * 10.0 ** rng.uniform(-3, 0, n)).astype(np.float32)
    t["g"] = torch.from_numpy(g).to(grad).cuda()
    if state == 8:
        (t["m"], t["sm"]), (t["v"], t["sv"]) = _state8(rng, n, 1e-3, False), _state8(rng, n, 1e-3, True)
    else:
        t["m"] = torch.from_numpy((rng.standard_normal(n) * 1e-3).astype(np.float32)).cuda()
        t["v"] = torch.from_numpy((rng.standard_normal(n) * 1e-3).astype(np.float32) ** 2).cuda()
        t["sm"] = t["sv"] = None
    return t


def _moments(t):
    if t["sm"] is None:
        return ref.f64(t["m"]), ref.f64(t["v"])
    n = t["p"].numel()
    spread = lambda s: np.repeat(ref.f64(s), 128)[:n]  # noqa: E731
    return ref.f64(t["m"].float()) * spread(t["sm"]), (ref.f64(t["v"].float()) * spread(t["sv"])) ** 2


def _step(mole, ts, decay, stream=None, **kw):
    col = lambda k: [t[k] for t in ts]  # noqa: E731
    eight = ts[0]["sm"] is not None
    mole.mole_adamw_step(col("p"), col("g"), col("m"), col("v"), masters=col("w"),
                         m_scales=col("sm") if eight else None, v_scales=col("sv") if eight else None,
                         weight_decay=decay, stream=stream, **{**HYPER, **kw})


def _expect(t, decay, factor=1.0, **kw):
    h = {**HYPER, **kw}
    m, v = _moments(t)
    p = ref.f64(t["w"] if t["w"] is not None else t["p"])
    return ref.adamw(p, factor * ref.f64(t["g"]), m, v, h["lr"], h["beta1"], h["beta2"], h["eps"], h["step"],
                     float(np.float32(decay)))


def _check(t, want):
    p, m, v, bp, bm, bv = want
    ref.assert_within(ref.f64(t["p"]), p, bp + ref.HALF[t["p"].dtype] * (np.abs(p) + bp), "param")
    if t["w"] is not None:
        ref.assert_within(ref.f64(t["w"]), p, bp + ref.U * np.abs(p), "master")
        assert torch.equal(t["p"], t["w"].to(BF16))
    if t["sm"] is None:
        ref.assert_within(ref.f64(t["m"]), m, bm, "m")
        ref.assert_within(ref.f64(t["v"]), v, bv, "v")
        return
    n = p.size
    root, broot = np.sqrt(v), 8 * ref.U * np.sqrt(v)
    for name, w, b, codes, scales, tiny in (("m", m, bm, t["m"], t["sm"], 2.0 ** -10),
                                            ("sqrt(v)", root, broot, t["v"], t["sv"], 2.0 ** -9)):
        pad = np.zeros(_blocks(n) * 128)
        pad[:n] = np.abs(w)
        s = np.maximum(pad.reshape(-1, 128).max(1) / 448, 2.0 ** -120)
        pad[:n] = b
        bs = pad.reshape(-1, 128).max(1) / 448 + 3 * ref.U * s
        ref.assert_within(ref.f64(scales), s, bs, name + " scale")
        got = ref.f64(codes.float())
        s_at, got_s = np.repeat(s, 128)[:n], np.repeat(ref.f64(scales), 128)[:n]
        # half a step of the code, and what w and the scale are off by
        bound = np.maximum(2.0 ** -4 * np.abs(w), tiny * s_at) * (1 + 2.0 ** -8) + 2 * b + np.abs(w) * 16 * ref.U
        ref.assert_within(got * got_s, w, bound, name)
        if name != "m":
            assert (got[w > 0] > 0).all(), "a second moment fell to zero"


@pytest.mark.parametrize("state", [32, 8])
@pytest.mark.parametrize("param,grad", [("f32", F32), ("f32", BF16), ("master", F32), ("master", BF16), ("bf16", F32),
                                        ("bf16", BF16)])
def test_step(mole, param, grad, state):
    rng = np.random.default_rng(state + len(param))
    sizes = [1, 2, 7, 8, 127, 128, 129, 1000, 2047, 2048, 2049, 4097, 30000]
    ts = [_tensor(rng, n, param, grad, state) for n in sizes]
    decay = [0.1 * (i % 3) for i in range(len(ts))]
    want = [_expect(t, d) for t, d in zip(ts, decay)]
    _step(mole, ts, decay)
    assert mole.mole_check() == 0
    for t, w in zip(ts, want):
        _check(t, w)


@pytest.mark.parametrize("state", [32, 8])
def test_many_tensors_and_mixed_types(mole, state):
    # more than one launch's tensors; empty ones among them
    rng = np.random.default_rng(3)
    kinds = [("f32", F32), ("master", BF16), ("bf16", F32)]
    ts = [_tensor(rng, int(n), *kinds[i % 3], state) for i, n in enumerate(rng.integers(0, 3000, 150))]
    want = [_expect(t, 0.01) for t in ts]
    _step(mole, ts, 0.01)
    assert mole.mole_check() == 0
    for t, w in zip(ts, want):
        if t["p"].numel():
            _check(t, w)


@pytest.mark.parametrize("state", [32, 8])
def test_views_inside_buffers(mole, state):
    # unaligned tensors, and the elements around them left as they were
    rng = np.random.default_rng(4)
    n = 1003
    t = _tensor(rng, n, "master", F32, state)
    want = _expect(t, 0.1)
    buffers = {}
    for k, x in t.items():
        if x is None:
            continue
        buf = torch.zeros(x.numel() + 2, dtype=F32, device="cuda").to(x.dtype)
        buf.view(torch.uint8).fill_(0x31)
        buf[1:-1] = x
        buffers[k] = (buf, buf.clone())
        t[k] = buf[1:-1]
    _step(mole, [t], 0.1)
    assert mole.mole_check() == 0
    _check(t, want)
    for k, (buf, before) in buffers.items():
        b, a = buf.view(torch.uint8), before.view(torch.uint8)
        e = buf.element_size()
        assert torch.equal(b[:e], a[:e]) and torch.equal(b[-e:], a[-e:]), k


@pytest.mark.parametrize("state", [32, 8])
def test_steps_from_zero_states(mole, state):
    # the usual start: all states (and scales) zero; several steps follow the
    # fp64 step on the states that the device holds
    rng = np.random.default_rng(5)
    t = _tensor(rng, 5000, "master", F32, state)
    for k in ("m", "v", "sm", "sv"):
        if t[k] is not None:
            t[k].view(torch.uint8).zero_()
    for step in (1, 2, 3):
        t["g"].copy_(torch.from_numpy((rng.standard_normal(5000) * 1e-2).astype(np.float32)))
        want = _expect(t, 0.0, step=step)
        _step(mole, [t], 0.0, step=step)
        assert mole.mole_check() == 0
        _check(t, want)


@pytest.mark.parametrize("state", [32, 8])
def test_zero_gradients(mole, state):
    # nothing moves but the decay; zero states stay zero
    rng = np.random.default_rng(6)
    t = _tensor(rng, 700, "f32", F32, state)
    for k in ("m", "v", "g"):
        t[k].view(torch.uint8).zero_()
    p = t["p"].clone()
    _step(mole, [t], 0.0)
    assert mole.mole_check() == 0 and torch.equal(t["p"], p)
    assert not t["m"].float().any() and not t["v"].float().any()


def test_gradients_that_are_not_finite(mole):
    rng = np.random.default_rng(7)
    for state, reach in ((32, 1), (8, 128)):
        t = _tensor(rng, 512, "f32", F32, state)
        t["g"][200] = float("inf")
        t["g"][400] = float("nan")
        _step(mole, [t], 0.0)
        assert mole.mole_check() == 0
        spoilt = torch.zeros(512, dtype=torch.bool, device="cuda")
        for i in (200, 400):
            spoilt[i // reach * reach:i // reach * reach + reach] = True
        m, v = (torch.from_numpy(x).cuda() for x in _moments(t))
        for s in (m, v):
            assert torch.isfinite(s[~spoilt]).all() and not torch.isfinite(s[[200, 400]]).any()
        # the weights are updated from the states in fp32: only the two are lost
        lost = ~torch.isfinite(t["p"])
        assert lost[400] and not lost[torch.arange(512, device="cuda") % 200 != 0].any()


@pytest.mark.parametrize("state", [32, 8])
def test_device_step_rate_and_factor_in_a_graph(mole, state):
    rng = np.random.default_rng(8)
    t = _tensor(rng, 3000, "master", F32, state)
    host = {k: None if x is None else x.clone() for k, x in t.items()}
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    lr = torch.tensor([0.0], device="cuda")
    factor = torch.tensor([1.0], device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(mole, [t], 0.1, step=step, lr_dev=lr, grad_scale=factor)
    for k, rate, fac in ((1, 1e-3, 1.0), (2, 5e-4, 0.25), (1000, 2e-3, 0.5)):
        step.fill_(k)
        lr.fill_(rate)
        factor.fill_(fac)
        graph.replay()
        want = _expect(host, 0.1, factor=fac, step=k, lr=float(np.float32(rate)))
        _step(mole, [host], 0.1, step=k, lr=float(np.float32(rate)), grad_scale=factor)
        assert mole.mole_check() == 0
        _check(host, want)
        for name in t:
            if t[name] is not None:
                assert torch.equal(t[name].view(torch.uint8), host[name].view(torch.uint8)), (name, k)


def test_on_a_stream(mole):
    rng = np.random.default_rng(9)
    t = _tensor(rng, 3000, "f32", F32, 32)
    want = _expect(t, 0.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    _step(mole, [t], 0.0, stream=side)
    side.synchronize()
    _check(t, want)


def test_large_tensor(mole):
    # element offsets beyond 2^31 bytes in every array, checked at both ends by torch in fp64
    n = (1 << 29) + 77
    p = torch.zeros(n, device="cuda")
    g = torch.full((n,), 1e-3, device="cuda")
    m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    mole.mole_adamw_step([p], [g], [m], [v], lr=0.1, beta1=0.9, beta2=0.99, eps=0.0, step=1)
    assert mole.mole_check() == 0
    for x, want in ((p, -0.1), (m, 1e-4), (v, 1e-8)):
        lo, hi = float(x.min()), float(x.max())
        assert abs(lo - want) <= 32 * ref.U * abs(want) and abs(hi - want) <= 32 * ref.U * abs(want)


@pytest.mark.parametrize("eps", [0.0, 1e-50, 1e-40, 2.0 ** -126, 1e-30])
@pytest.mark.parametrize("param", ["f32", "master", "bf16"])
@pytest.mark.parametrize("state", [32, 8])
def test_zero_moments_with_an_eps_near_zero(mole, param, state, eps):
    # zero states and, for every other run of elements, no gradient (the rows of
    # an embedding that a batch does not hold): nothing but the decay moves them
    rng = np.random.default_rng(10)
    n = 5003
    t = _tensor(rng, n, param, F32, state)
    for k in ("m", "v", "sm", "sv"):
        if t[k] is not None:
            t[k].view(torch.uint8).zero_()
    still = np.arange(n) // 50 % 2 == 0
    t["g"][torch.from_numpy(still).cuda()] = 0.0
    t["g"][torch.from_numpy(~still).cuda()] += 1e-6
    host = {k: None if x is None else x.clone() for k, x in t.items()}
    _step(mole, [t], 0.1, eps=eps, step=1)
    assert mole.mole_check() == 0
    with np.errstate(divide="ignore", invalid="ignore"):
        want = [np.array(x) for x in _expect(host, 0.1, eps=eps, step=1)]
    p0 = ref.f64(host["w"] if host["w"] is not None else host["p"])
    # the decay of a weight whose step is zero: three roundings
    decayed = p0 - HYPER["lr"] * float(np.float32(0.1)) * p0
    want[0] = np.where(still, decayed, want[0])
    want[3] = np.where(still, 4 * ref.U * np.abs(p0), want[3])
    _check(t, want)

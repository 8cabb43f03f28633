"""The operators around a layer in a training step, without a GPU: what their
entry points refuse, their workspace sizes, and the fp64 forms that the GPU
tests compare with (their gradients against differences)."""
import ctypes

import numpy as np
import pytest
import torch

import train_ops_ref as ref

P = 0x100000      # a fake, aligned, never dereferenced address
F32, BF16 = 0, 1
NO_DEVICE = 8


@pytest.fixture(autouse=True)
def _no_gpu_call():
    if torch.cuda.is_available():
        pytest.skip("valid arguments would be launched with fake addresses")


def test_embed_refusals(mole):
    f = mole.lib.mole_embed_forward
    ok = dict(ids=P, T=5, E=P, V=10, D=7, scale=1.0, dt_E=BF16, out=P, dt_out=F32)
    call = lambda **kw: f(*{**ok, **kw}.values(), None)  # noqa: E731
    assert call() == NO_DEVICE
    for kw in (dict(T=-1), dict(V=0), dict(D=0), dict(dt_E=2), dict(dt_out=-1), dict(ids=None), dict(E=None),
               dict(out=None)):
        assert call(**kw) == 1, kw
    for kw in (dict(T=2 ** 31), dict(V=2 ** 31), dict(D=2 ** 20 + 1)):
        assert call(**kw) == 3, kw
    for kw in (dict(ids=P + 2), dict(E=P + 1), dict(out=P + 2)):
        assert call(**kw) == 2, kw
    assert call(E=P + 2) == NO_DEVICE              # a bf16 row may start anywhere
    assert call(T=0, ids=None, E=None, out=None) == 0

    size = mole.mole_embed_backward_workspace
    assert size(0, 64) == 0 and size(5, 0) == 0 and size(2 ** 31, 64) == 0
    # two sorted copies, and two rows of partial sums per chunk of 16 tokens or more
    assert size(16384, 2048) >= 2 * 8 * 16384 + 2 * 4 * 2048 * 16384 // 256
    assert size(16384, 2048) <= 2 * 8 * 16384 + 2 * 4 * 2048 * 16384 // 16 + 768
    b = mole.lib.mole_embed_backward
    ws = size(5, 7)
    ok = dict(ids=P, T=5, dout=P, dt=BF16, V=10, D=7, scale=1.0, dE=P, ws=P, ws_bytes=ws)
    call = lambda **kw: b(*{**ok, **kw}.values(), None)  # noqa: E731
    assert call() == NO_DEVICE
    for kw in (dict(T=-1), dict(V=0), dict(D=-3), dict(dt=7), dict(ids=None), dict(dout=None), dict(dE=None)):
        assert call(**kw) == 1, kw
    assert call(T=2 ** 31) == 3
    for kw in (dict(ids=P + 1), dict(dout=P + 1), dict(dE=P + 2), dict(ws=P + 8)):
        assert call(**kw) == 2, kw
    assert call(ws=None) == 4 and call(ws_bytes=ws - 1) == 4
    assert call(T=0, ids=None, dout=None, dE=None, ws=None, ws_bytes=0) == 0


def test_block_norm_refusals(mole):
    f = mole.lib.mole_block_norm_forward
    ok = dict(x=P, dt_x=F32, f=P, dt_f=BF16, w_post=P, gate=P, res_scale=1.0, w_pre=P, eps=1e-6, T=5, D=7, x_out=P,
              h=P, dt_h=BF16)
    call = lambda **kw: f(*{**ok, **kw}.values(), None)  # noqa: E731
    assert call() == NO_DEVICE
    for kw in (dict(T=-1), dict(D=0), dict(dt_x=2), dict(dt_f=2), dict(dt_h=2), dict(eps=0.0), dict(eps=-1.0),
               dict(eps=float("nan")), dict(x=None), dict(x_out=None, h=None), dict(w_pre=None), dict(f=None),
               dict(f=None, w_post=None)):
        assert call(**kw) == 1, kw
    for kw in (dict(T=2 ** 31), dict(D=8193)):
        assert call(**kw) == 3, kw
    for kw in (dict(x=P + 2), dict(f=P + 1), dict(w_post=P + 2), dict(gate=P + 1), dict(w_pre=P + 2),
               dict(x_out=P + 2), dict(h=P + 1)):
        assert call(**kw) == 2, kw
    for kw in (dict(h=None, w_pre=None), dict(x_out=None), dict(f=None, w_post=None, gate=None), dict(w_post=None),
               dict(gate=None), dict(D=8192)):
        assert call(**kw) == NO_DEVICE, kw
    assert call(T=0) == 0

    size = mole.mole_block_norm_backward_workspace
    assert size(0, 64) == 0 and size(5, 0) == 0 and size(5, 8193) == 0
    assert size(5, 64) > 0 and size(1 << 20, 2048) <= 2 * 148 * 16 * 2048 * 4
    b = mole.lib.mole_block_norm_backward
    ws = size(5, 7)
    ok = dict(x=P, dt_x=F32, f=P, dt_f=BF16, w_post=P, gate=P, res_scale=1.0, w_pre=P, eps=1e-6, T=5, D=7, dx_out=P,
              dh=P, dx=P, df=P, dgate=P, dw_post=P, dw_pre=P, ws=P, ws_bytes=ws)
    call = lambda **kw: b(*{**ok, **kw}.values(), None)  # noqa: E731
    assert call() == NO_DEVICE
    for kw in (dict(T=-1), dict(D=0), dict(dt_x=2), dict(dt_f=3), dict(eps=0.0), dict(dx_out=None, dh=None),
               dict(dx=None, df=None, dgate=None, dw_post=None, dw_pre=None), dict(w_pre=None), dict(x=None),
               dict(dh=None), dict(f=None), dict(f=None, w_post=None, dw_post=None), dict(w_post=None)):
        assert call(**kw) == 1, kw
    for kw in (dict(T=2 ** 31), dict(D=8193)):
        assert call(**kw) == 3, kw
    for k in ("w_post", "gate", "w_pre", "dx_out", "dh", "dx", "df", "dgate", "dw_post", "dw_pre", "x"):
        assert call(**{k: P + 2}) == 2, k
    assert call(f=P + 1) == 2 and call(ws=P + 8) == 2
    assert call(ws=None) == 4 and call(ws_bytes=ws - 1) == 4
    assert call(ws=None, ws_bytes=0, dw_post=None, dw_pre=None) == NO_DEVICE
    assert call(T=0) == 0


def _adam(mole, n, state8=0, **kw):
    t = (mole.AdamWTensor * n)()
    for i in range(n):
        base = P + (i << 24)
        t[i].param, t[i].grad, t[i].m, t[i].v = base, base + (1 << 20), base + (2 << 20), base + (3 << 20)
        t[i].n, t[i].dt_param, t[i].dt_grad = 1000, BF16, F32
        if state8:
            t[i].m_scale, t[i].v_scale = base + (4 << 20), base + (5 << 20)
    cfg = mole.AdamWConfig(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, step=1, state8=state8)
    for k, v in kw.items():
        setattr(cfg, k, v)
    return t, cfg


def test_adamw_refusals(mole):
    def call(t, cfg, n=None):
        return mole.lib.mole_adamw_step(t, len(t) if n is None else n, ctypes.addressof(cfg), None)

    assert call(*_adam(mole, 3)) == NO_DEVICE and call(*_adam(mole, 3, 1)) == NO_DEVICE
    t, cfg = _adam(mole, 1)
    assert call(t, cfg, 0) == 0 and call(t, cfg, -1) == 1
    assert mole.lib.mole_adamw_step(None, 1, ctypes.addressof(cfg), None) == 1
    assert mole.lib.mole_adamw_step(t, 1, None, None) == 1
    for kw in (dict(step=0), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(eps=-1.0),
               dict(eps=float("nan")), dict(state8=2)):
        t, cfg = _adam(mole, 1)
        for k, v in kw.items():
            setattr(cfg, k, v)
        assert call(t, cfg) == 1, kw
    assert call(*_adam(mole, 1, step=0, step_dev=P + (9 << 20))) == NO_DEVICE
    assert call(*_adam(mole, 1, step_dev=P + 4 + (9 << 20))) == 2
    assert call(*_adam(mole, 1, lr_dev=P + 2 + (9 << 20))) == 2
    assert call(*_adam(mole, 1, grad_scale_dev=P + 2 + (9 << 20))) == 2
    for field, value, status in (("n", -1, 1), ("n", 2 ** 41, 3), ("dt_param", 2, 1), ("dt_grad", -1, 1),
                                 ("param", None, 1), ("grad", None, 1), ("m", None, 1), ("v", None, 1),
                                 ("param", P + 1, 2), ("grad", P + 2 + (1 << 20), 2), ("m", P + 2 + (2 << 20), 2),
                                 ("master", P + 2 + (7 << 20), 2), ("m_scale", P + (7 << 20), 1)):
        t, cfg = _adam(mole, 2)
        setattr(t[1], field, value)
        assert call(t, cfg) == status, field
    t, cfg = _adam(mole, 1)
    t[0].dt_param, t[0].master = F32, P + (7 << 20)          # an fp32 param has no master
    assert call(t, cfg) == 1
    t, cfg = _adam(mole, 2, 1)
    t[1].v_scale = None
    assert call(t, cfg) == 1
    # an empty tensor's pointers are not looked at
    t, cfg = _adam(mole, 2)
    t[1].n, t[1].param, t[1].m = 0, None, None
    assert call(t, cfg) == NO_DEVICE


def test_adamw_refuses_overlaps(mole):
    def call(change, state8=0):
        t, cfg = _adam(mole, 3, state8)
        change(t, cfg)
        return mole.lib.mole_adamw_step(t, 3, ctypes.addressof(cfg), None)

    assert call(lambda t, c: setattr(t[2], "param", t[0].param)) == 1             # the same tensor twice
    assert call(lambda t, c: setattr(t[2], "param", t[0].param + 1998)) == 1      # one element
    assert call(lambda t, c: setattr(t[2], "param", t[0].param + 2000)) == NO_DEVICE
    assert call(lambda t, c: setattr(t[1], "m", t[1].v)) == 1
    assert call(lambda t, c: setattr(t[1], "grad", t[2].m + 4)) == 1              # a gradient in written memory
    assert call(lambda t, c: setattr(t[1], "grad", t[0].grad)) == NO_DEVICE       # a shared gradient is only read
    assert call(lambda t, c: setattr(t[1], "v_scale", t[1].m_scale + 4 * 7), 1) == 1
    assert call(lambda t, c: setattr(t[1], "v_scale", t[1].m_scale + 4 * 8), 1) == NO_DEVICE
    assert call(lambda t, c: setattr(c, "lr_dev", t[0].v + 8)) == 1


def test_binding_refusals(mole):
    """The binding looks at shapes, types and devices before anything is launched."""
    x, w = torch.zeros(4, 8), torch.zeros(8)
    ids = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: mole.mole_embed_forward(ids, x), lambda: mole.mole_embed_backward(ids, x, x),
                 lambda: mole.mole_block_norm_forward(x, w_pre=w),
                 lambda: mole.mole_block_norm_backward(x, x, x, w_pre=w),
                 lambda: mole.mole_adamw_step([w], [w], [w], [w])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="lengths"):
        mole.mole_adamw_step([w, w], [w], [w, w], [w, w])
    mole.mole_adamw_step([], [], [], [])
    codes = torch.zeros(8, dtype=torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="scales"):
        mole.mole_adamw_step([w], [w], [codes], [codes])
    with pytest.raises(ValueError, match="scales"):
        mole.mole_adamw_step([w], [w], [w], [w], m_scales=[w], v_scales=[w])


def _differences(f, x, eps=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        y = x.copy()
        y[i] += eps
        up = f(y)
        y[i] -= 2 * eps
        g[i] = (up - f(y)) / (2 * eps)
    return g


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_norm_form_against_differences(post, gated):
    rng = np.random.default_rng(1)
    T, D = 3, 5
    x, f, cx, ch = (rng.standard_normal((T, D)) for _ in range(4))
    w_post, w_pre = (rng.standard_normal(D) if post else None), rng.standard_normal(D)
    gate = rng.standard_normal(T) if gated else None

    def loss(x, f, w_post, gate, w_pre):
        xo, h, _, _ = ref.norm_forward(x, f, w_post, gate, 0.7, w_pre, 1e-3)
        return (xo * cx).sum() + (h * ch).sum()

    xo = ref.norm_forward(x, f, w_post, gate, 0.7, w_pre, 1e-3)[0]
    got = ref.norm_backward(xo, f, w_post, gate, 0.7, w_pre, 1e-3, cx, ch)
    args = dict(x=x, f=f, w_post=w_post, gate=gate, w_pre=w_pre)
    for name, arg in (("dx", "x"), ("df", "f"), ("dgate", "gate"), ("dw_post", "w_post"), ("dw_pre", "w_pre")):
        if args[arg] is None:
            continue
        want = _differences(lambda y, arg=arg: loss(**{**args, arg: y}), args[arg])
        np.testing.assert_allclose(got[name][0], want, rtol=1e-6, atol=1e-7, err_msg=name)


def test_embedding_form_against_differences():
    rng = np.random.default_rng(2)
    T, V, D = 9, 4, 3
    ids = np.array([0, 2, 2, 3, 0, 2, -1, 4, 2], np.int32)
    E, c = rng.standard_normal((V, D)), rng.standard_normal((T, D))
    ok = (ids >= 0) & (ids < V)
    want = _differences(lambda y: (1.5 * y[ids[ok]] * c[ok]).sum(), E)
    got, _ = ref.embed_backward(ids, c, np.zeros((V, D)), 1.5, V)
    np.testing.assert_allclose(got, want, rtol=1e-7, atol=1e-9)


def test_adamw_form_against_torch():
    rng = np.random.default_rng(3)
    p = torch.nn.Parameter(torch.from_numpy(rng.standard_normal(50)))
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(0.9, 0.95), eps=1e-6, weight_decay=0.1)
    q, m, v = p.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for step in (1, 2, 3):
        g = rng.standard_normal(50)
        p.grad = torch.from_numpy(g)
        opt.step()
        q, m, v = ref.adamw(q, g, m, v, 1e-2, 0.9, 0.95, 1e-6, step, 0.1)[:3]
        np.testing.assert_allclose(q, p.detach().numpy(), rtol=1e-12)


def test_adamw_eps_range(mole):
    for eps, status in ((0.0, NO_DEVICE), (1e-50, NO_DEVICE), (2.0 ** 125, NO_DEVICE), (2.0 ** 125 * 1.001, 1),
                        (1e300, 1), (float("inf"), 1)):
        t, cfg = _adam(mole, 1, eps=eps)
        assert mole.lib.mole_adamw_step(t, 1, ctypes.addressof(cfg), None) == status, eps


def test_embed_workspace_of_the_shortest_chunks(mole):
    # chunks of 8 tokens: two fp32 rows of partial sums each, T D bytes in all
    for T, D in ((2100, 64), (9000, 67), (14000, 1024)):
        size = mole.mole_embed_backward_workspace(T, D)
        chunks = (T + 7) // 8
        least = 2 * 8 * T + 16 + 8 * chunks + 2 * 4 * D * chunks
        assert least <= size <= least + 4 * 255, (T, D)

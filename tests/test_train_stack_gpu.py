"""A training step of a small model made of the library's calls: embedding,
norm, one MoLE layer, norm with gate and residual, and back, then the AdamW
step on every weight.  The loss is <x1, cx> + <h1, ch> for fixed cx, ch.

Each call has its own tests against fp64; here the whole chain is compared with
the chain of the fp64 forms (the layer's part by the oracle, at the device's own
bf16 inputs and precision points), in the 2-norm of each gradient: the layer's
bound is test_train_gpu's GRAD_RTOL (its bf16 GEMM operands), and what the
other calls add are fp32 roundings, far below it.
"""
import numpy as np
import pytest
import torch

import train_ops_ref as ref
from helpers import dev, host_bits
from mixture_lookup_experts_b200 import inputs

pytestmark = pytest.mark.gpu

GRAD_RTOL = 1e-3
EPS = 1e-6


def _rel(got, want):
    return float(np.linalg.norm(got - want) / np.linalg.norm(want))


@pytest.mark.parametrize("T,V,D,N,Dr", [(1200, 500, 128, 8, 192), (90, 2000, 64, 4, 128)])
def test_training_step(mole, oracle_mod, T, V, D, N, Dr):
    rng = np.random.default_rng(T)
    ids = inputs.zipf_ids(rng, T, V)
    E, W1, W2 = (inputs.normal(rng, s, sd, "bf16") for s, sd in (((V, D), 0.5), ((N, D, Dr), 0.05), ((N, Dr, D), 0.05)))
    Wr = inputs.normal(rng, (D, N), 0.1, "bf16")
    w = [torch.from_numpy((1 + 0.1 * rng.standard_normal(D)).astype(np.float32)).cuda() for _ in range(3)]
    w_in, w_post, w_pre = w
    gate = torch.sigmoid(torch.from_numpy(rng.standard_normal(T).astype(np.float32))).cuda()
    cx, ch = (torch.from_numpy(rng.standard_normal((T, D)).astype(np.float32)).cuda() for _ in range(2))
    scale, res = float(np.sqrt(D)), 0.9
    d_ids, dE_, dW1_, dW2_, dWr_ = dev(ids), dev(E), dev(W1), dev(W2), dev(Wr)
    zeros = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    grads = dict(E=zeros(V, D), W1=zeros(N, D, Dr), W2=zeros(N, Dr, D), Wr=zeros(D, N), w_in=zeros(D),
                 w_post=zeros(D), w_pre=zeros(D))

    # forward
    groups = mole.mole_token_groups_build(d_ids, V, N)
    x0 = mole.mole_embed_forward(d_ids, dE_, scale, out_dtype=torch.float32)
    _, h0 = mole.mole_block_norm_forward(x0, w_pre=w_in, eps=EPS)
    f, cache, U = mole.mole_train_forward(d_ids, groups, h0, dWr_, dE_, dW1_, dW2_)
    x1, h1 = mole.mole_block_norm_forward(x0, f, w_post, gate, res, w_pre, EPS, h_dtype=torch.float32)
    # backward
    dx, df, dgate = mole.mole_block_norm_backward(x1, cx, ch, f, w_post, gate, res, w_pre, EPS,
                                                  dw_post=grads["w_post"], dw_pre=grads["w_pre"])
    dh0 = zeros(T, D)
    mole.mole_train_backward(d_ids, groups, h0, dWr_, dE_, dW1_, dW2_, df, cache, U, dh=dh0, dWr=grads["Wr"],
                             dE=grads["E"], dW1=grads["W1"], dW2=grads["W2"])
    dx0, _, _ = mole.mole_block_norm_backward(x0, dx, dh0, w_pre=w_in, eps=EPS, dw_pre=grads["w_in"])
    mole.mole_embed_backward(d_ids, dx0, grads["E"], scale)
    assert mole.mole_check() == 0

    # the same in fp64, the layer by the oracle on the device's h0
    r32 = float(np.float32(res))
    e32 = float(np.float32(EPS))
    X0 = float(np.float32(scale)) * ref.f64(dE_)[ids]
    F = ref.f64(f)
    X1, H1, _, _ = ref.norm_forward(X0, F, ref.f64(w_post), ref.f64(gate), r32, ref.f64(w_pre), e32)
    assert _rel(ref.f64(x1), X1) < 1e-6 and _rel(ref.f64(h1), H1) < 1e-6
    back = ref.norm_backward(X1, F, ref.f64(w_post), ref.f64(gate), r32, ref.f64(w_pre), e32, ref.f64(cx), ref.f64(ch))
    _, layer = oracle_mod.train_step(ids, host_bits(h0), Wr, E, W1, W2, "gelu", back["df"][0].astype(np.float32),
                                     round_ops=True)
    inner = ref.norm_backward(X0, None, None, None, 1.0, ref.f64(w_in), e32, back["dx"][0], layer["dh"])
    dE = layer["dE"].copy()
    np.add.at(dE, ids, float(np.float32(scale)) * inner["dx"][0])
    want = dict(E=dE, W1=layer["dW1"], W2=layer["dW2"], Wr=layer["dWr"], w_in=inner["dw_pre"][0],
                w_post=back["dw_post"][0], w_pre=back["dw_pre"][0])
    assert _rel(ref.f64(dgate), back["dgate"][0]) < GRAD_RTOL
    for k, g in grads.items():
        assert _rel(ref.f64(g), want[k]) < GRAD_RTOL, k

    # the step: bf16 weights with fp32 masters and 8-bit states, fp32 weights without
    weights = dict(E=dE_, W1=dW1_, W2=dW2_, Wr=dWr_)
    masters = {k: t.float() for k, t in weights.items()}
    blocks = {k: (t.numel() + 127) // 128 for k, t in weights.items()}
    m8, v8 = ({k: torch.zeros_like(t, dtype=torch.float8_e4m3fn) for k, t in weights.items()} for _ in range(2))
    s8 = [[zeros(n) for n in blocks.values()] for _ in range(2)]
    before = {k: ref.f64(t) for k, t in masters.items()}
    mole.mole_adamw_step(weights.values(), [grads[k] for k in weights], m8.values(), v8.values(),
                         masters=masters.values(), m_scales=s8[0], v_scales=s8[1], lr=1e-3, step=1)
    small = dict(w_in=w_in, w_post=w_post, w_pre=w_pre)
    before |= {k: ref.f64(t) for k, t in small.items()}
    mole.mole_adamw_step(small.values(), [grads[k] for k in small], [zeros(D) for _ in small],
                         [zeros(D) for _ in small], lr=1e-3, step=1)
    assert mole.mole_check() == 0
    for k, p in {**masters, **small}.items():
        n = before[k].shape
        q, _, _, bound, _, _ = ref.adamw(before[k], ref.f64(grads[k]), np.zeros(n), np.zeros(n), 1e-3, 0.9, 0.999,
                                         1e-8, 1, 0.0)
        ref.assert_within(ref.f64(p), q, bound, k)
        if k in weights:
            assert torch.equal(weights[k], p.to(torch.bfloat16))
    # ids that the batch does not hold keep their rows
    rest = dev(np.setdiff1d(np.arange(V), ids))
    assert torch.equal(masters["E"][rest].double().cpu(), torch.from_numpy(before["E"])[rest.cpu()])


def test_calls_from_two_threads_on_two_streams(mole):
    """The same calls at the same time, of different sizes, each thread with
    its stream: the results are those of the calls one by one."""
    import threading
    sizes = [(3000, 512), (1500, 2048)]
    V = 700

    def make(T, D):
        g = torch.Generator(device="cuda")
        g.manual_seed(T)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        ids = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
        return dict(ids=ids, x=rnd(T, D), f=rnd(T, D), c=rnd(T, D), w=rnd(D), E=rnd(V, D))

    def run(d, stream):
        T, D = d["x"].shape
        with torch.cuda.stream(stream):
            dE, dw, p, m, v = (torch.zeros(s, device="cuda") for s in ((V, D), (D,), (V, D), (V, D), (V, D)))
            out = mole.mole_embed_forward(d["ids"], d["E"], 2.0)
            x1, h = mole.mole_block_norm_forward(d["x"], d["f"], d["w"], None, 0.5, d["w"])
            dx, df, _ = mole.mole_block_norm_backward(x1, d["c"], d["c"], d["f"], d["w"], None, 0.5, d["w"], dw_pre=dw,
                                                      dw_post=dw.clone())
            mole.mole_embed_backward(d["ids"], dx, dE)
            mole.mole_adamw_step([p], [dE], [m], [v])
        return out, x1, h, dx, df, dw, dE, p

    data = [make(*s) for s in sizes]
    torch.cuda.synchronize()
    want = [run(d, torch.cuda.current_stream()) for d in data]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            for _ in range(30):
                got[i] = run(data[i], stream)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert mole.mole_check() == 0
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_norm_backward_before_kernels_that_start_early(mole):
    """Without weight gradients the backward is one kernel; the library's other
    kernels behind it (a row prefetch, a combine: both may start early) still
    find its results."""
    T, V, D, N = 20000, 300, 512, 8
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, f, c, w = rnd(T, D), rnd(T, D), rnd(T, D), rnd(D)
    lut, Wr = rnd(V, N, D).to(torch.bfloat16), rnd(D, N)
    lut32 = lut.float()
    ids = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    _, df, _ = mole.mole_block_norm_backward(x, c, c, f, w, None, 1.0, w)
    torch.cuda.synchronize()
    want = mole.mole_lookup_combine(ids, df, Wr, lut32)
    torch.cuda.synchronize()
    for _ in range(5):
        out = torch.zeros_like(df)
        mole.mole_block_norm_backward(x, c, c, f, w, None, 1.0, w, df=out)
        mole.mole_prefetch_rows(ids, [lut])
        got = mole.mole_lookup_combine(ids, out, Wr, lut32)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    assert mole.mole_check() == 0


def test_streams_by_handle(mole):
    """A stream given by its handle (0: the default stream, as the other calls
    take it) gets the kernels behind what it holds already; so does a torch
    stream."""
    T, V, D = 3000, 400, 256
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    ids = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    E, X, F, C, w = rnd(V, D), rnd(T, D), rnd(T, D), rnd(T, D), rnd(D)

    def run(stream):
        dE, dw, p, m, v = (torch.zeros(s, device="cuda") for s in ((V, D), (D,), (V, D), (V, D), (V, D)))
        x = torch.zeros_like(X)
        torch.cuda._sleep(20_000_000)  # (some 10 ms: what follows is not there before)
        x.copy_(X)
        out = mole.mole_embed_forward(ids, E, 2.0, stream=stream)
        x1, h = mole.mole_block_norm_forward(x, F, w, None, 0.5, w, stream=stream)
        dx, df, _ = mole.mole_block_norm_backward(x1, C, C, F, w, None, 0.5, w, dw_pre=dw, stream=stream)
        mole.mole_embed_backward(ids, dx, dE, stream=stream)
        mole.mole_adamw_step([p], [dE], [m], [v], stream=stream)
        return [t.clone() for t in (out, x1, h, dx, df, dw, dE, p)]

    dev0 = E.device
    for handle in (0, 1, torch.cuda.default_stream().cuda_stream):
        with mole._on_stream(handle, dev0):
            assert torch.cuda.current_stream() == torch.cuda.default_stream()
    with pytest.raises(ValueError, match="per-thread"):
        run(2)
    want = run(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for current, stream in ((torch.cuda.default_stream(), 0), (torch.cuda.default_stream(), 1), (side, side),
                            (side, side.cuda_stream)):
        torch.cuda.synchronize()
        with torch.cuda.stream(current):
            got = run(stream)
        torch.cuda.synchronize()
        assert mole.mole_check() == 0
        for a, b in zip(want, got):
            assert torch.equal(a, b), stream


def test_capture_with_the_streams_handle(mole):
    """Calls captured with the capturing stream's handle, workspaces made in the
    capture: a replay gives the results of the calls one by one."""
    T, V, D = 3000, 400, 256
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    ids = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    E, X, F, C, w = rnd(V, D), rnd(T, D), rnd(T, D), rnd(T, D), rnd(D)

    def run(sums, stream):
        dE, dw, p, m, v = sums
        out = mole.mole_embed_forward(ids, E, 2.0, stream=stream)
        x1, h = mole.mole_block_norm_forward(X, F, w, None, 0.5, w, stream=stream)
        dx, df, _ = mole.mole_block_norm_backward(x1, C, C, F, w, None, 0.5, w, dw_pre=dw, stream=stream)
        mole.mole_embed_backward(ids, dx, dE, stream=stream)
        mole.mole_adamw_step([p], [dE], [m], [v], stream=stream)
        return out, x1, h, dx, df

    make = lambda: [torch.zeros(s, device="cuda") for s in ((V, D), (D,), (V, D), (V, D), (V, D))]  # noqa: E731
    sums, once = make(), make()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(sums, torch.cuda.current_stream().cuda_stream)
    want = run(once, None)
    for _ in range(2):
        for t in sums:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((*want, *once), (*got, *sums)):
            assert torch.equal(a, b)
    assert mole.mole_check() == 0
